// ssm_internal.h -- host-side interface between the C ABI layer of the
// state-space operators (ssm_capi.cu) and their kernel launchers.
#pragma once

#include "wkv_internal.h"
#include "wkv_ssm.h"

namespace wkv {

// Address of the current device's error word (capi.cu).
wkv_status device_error_word(unsigned** out);

// For each of up to kMost planes that has an output: out[c] = the sum of
// part[rows][cols] (float or double) over its rows, in a fixed order. One launch.
template <class P>
struct SumRows {
  static constexpr int kMost = 5;
  struct Plane {
    const P* part;
    int64_t cols;
    float* out;
  } plane[kMost];
  int planes;
  int64_t rows;
  void add(const P* part, int64_t cols, float* out) {
    if (out) plane[planes++] = {part, cols, out};
  }
};
template <class P>
wkv_status launch_sum_rows(const SumRows<P>& s, cudaStream_t stream, const char** why);

// ---- short causal convolution ------------------------------------------------
struct ConvArgs {
  int64_t B, T, C;  // slots: B = S, T unused
  int dtype, W, silu;
  const void* x;
  const float* weight;
  const float* bias;
  const void* x_prev;
  void* y;
  const void* gy;
  void* gx;
  float* gweight;
  float* gbias;
  void* gx_prev;
  float* part;
  int64_t n_tokens;
  const int32_t* cu;
  void* state;
};
// Launch shape: channel blocks, and each sequence cut into nrun runs of Lt tokens.
struct ConvShape {
  int ncb, nrun, Lt;
};
ConvShape conv_bwd_shape(int64_t B, int64_t T, int64_t C);
wkv_status launch_conv_forward(const ConvArgs& a, cudaStream_t stream, const char** why);
wkv_status launch_conv_backward(const ConvArgs& a, cudaStream_t stream, const char** why);
wkv_status launch_conv_chunk_step(const ConvArgs& a, cudaStream_t stream, unsigned* err, const char** why);
wkv_status launch_conv_decode_step(const ConvArgs& a, cudaStream_t stream, const char** why);

// ---- per-head norm with rotation ------------------------------------------------
struct NormArgs {
  int64_t tokens, T;  // tokens = B * T
  int Hq, Hk, K, R, dtype, interleaved;
  const void* q;
  const void* k;
  const float* wq;
  const float* wk;
  float eps;
  const float* inv_freq;
  const int32_t* positions;
  int64_t pos_offset;
  void* q_out;  // backward: gq
  void* k_out;  // backward: gk
  const void* gq;
  const void* gk;
  float* gwq;
  float* gwk;
  float* part;
};
// CTAs of the backward kernel (each leaves one row of weight-gradient partial sums).
int64_t norm_bwd_blocks(int64_t tokens, int64_t Hq, int64_t Hk, int64_t K);
wkv_status launch_norm_rotate(const NormArgs& a, cudaStream_t stream, const char** why);
wkv_status launch_norm_rotate_backward(const NormArgs& a, cudaStream_t stream, const char** why);

// ---- selective scan -------------------------------------------------------------
struct ScanArgs {
  int64_t B, T, C, N, G;  // slots: B = S, T unused
  int dtype;
  const void* x;
  const void* dt;
  const float* A;
  const void* Bm;
  const void* Cm;
  const float* D;
  const void* z;
  const float* dt_bias;
  int softplus;
  const float* init_state;
  void* y;
  float* final_state;
  float* ckpt;
  float* carry;  // of the cut sequences: [sequence][nseg][C][N] states, then [sequence][nseg][C] sums of d
  int64_t n_tokens;
  const int32_t* cu;  // slots, else null
};
struct ScanBwdArgs {
  ScanArgs f;  // f.ckpt: the checkpoints (read); f.carry: pieces of the reverse walk
  const void* gy;
  const float* g_final;
  void* gx;
  void* gdt;
  float* gA;
  void* gB;
  void* gC;
  float* gD;
  void* gz;
  float* gdt_bias;
  float* g_init;
  float* part_bc;  // [2][blocks per group][B*T][G*N]
  double* part_a;  // [pieces of all sequences][C][N]
  double* part_d;  // [2][pieces of all sequences][C]: gD, gdt_bias
};
// State sizes the kernels are built for.
inline int scan_padded_states(int64_t N) { return N <= 8 ? 8 : N <= 16 ? 16 : N <= 32 ? 32 : 64; }
// Channels per CTA, by the padded state size.
constexpr int scan_cta_channels(int states) { return states <= 8 ? 64 : states <= 32 ? 32 : 16; }
// CTAs that cover one group's channels.
inline int64_t scan_group_blocks(int64_t C, int64_t N, int64_t G) {
  return ceil_div(C / std::max<int64_t>(G, 1), scan_cta_channels(scan_padded_states(N)));
}
// How a launch is cut along T: the first `whole` sequences are not, the others
// are, into nseg pieces, each but the last of seg_tiles * WKV_SCAN_CKPT_LEN
// tokens. nseg is 1 where none is cut.
struct ScanCut {
  int64_t whole;
  int nseg, seg_tiles;
  int64_t rows(int64_t B) const { return whole + (B - whole) * nseg; }  // pieces of all sequences
};
ScanCut scan_fwd_cut(int64_t B, int64_t T, int64_t C, int64_t N, int64_t G);
ScanCut scan_bwd_cut(int64_t B, int64_t T, int64_t C, int64_t N, int64_t G);
inline int64_t scan_carry_floats(int64_t B, int64_t C, int64_t N, const ScanCut& cut) {
  return (B - cut.whole) * cut.nseg * C * (N + 1);
}
wkv_status launch_scan_forward(const ScanArgs& a, cudaStream_t stream, const char** why);
wkv_status launch_scan_chunk_step(const ScanArgs& a, cudaStream_t stream, unsigned* err, const char** why);
wkv_status launch_scan_decode_step(const ScanArgs& a, cudaStream_t stream, const char** why);
wkv_status launch_scan_backward(const ScanBwdArgs& a, cudaStream_t stream, const char** why);

}  // namespace wkv
