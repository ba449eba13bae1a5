// ssm_capi.cu -- the C ABI of the state-space operators (include/wkv_ssm.h):
// argument checks on the host, then the launchers. Nothing here allocates or
// synchronises.
#include <cuda_runtime.h>

#include "ssm_internal.h"

#define WKV_EXPORT extern "C" __attribute__((visibility("default")))

namespace wkv {
namespace {

wkv_status fail(wkv_status s, const char* why) {
  set_last_error(why);
  return s;
}
wkv_status ended(wkv_status s, const char* why) { return s == WKV_OK ? s : fail(s, why); }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

#define REQUIRE_PTR(p, name)                                                             \
  do {                                                                                   \
    if (!(p)) return fail(WKV_ERR_INVALID_ARG, name " is NULL");                         \
    if (!aligned16(p)) return fail(WKV_ERR_INVALID_ARG, name " is not 16-byte aligned"); \
  } while (0)
#define OPTIONAL_PTR(p, name)                                                                   \
  do {                                                                                          \
    if ((p) && !aligned16(p)) return fail(WKV_ERR_INVALID_ARG, name " is not 16-byte aligned"); \
  } while (0)

// B * T * C activations of `dtype`. The product bound keeps every offset and
// launch grid in range.
wkv_status check_act(int64_t B, int64_t T, int64_t C, int dtype) {
  if (B < 0 || T < 0 || C < 0) return fail(WKV_ERR_INVALID_ARG, "negative size");
  if (dtype != WKV_F32 && dtype != WKV_BF16) return fail(WKV_ERR_INVALID_ARG, "unknown dtype");
  if ((dtype == WKV_F32 && C % 4) || (dtype == WKV_BF16 && C % 8))
    return fail(WKV_ERR_UNSUPPORTED, "C must be a multiple of 4 (f32) or 8 (bf16)");
  if (T > INT32_MAX || B > INT32_MAX) return fail(WKV_ERR_UNSUPPORTED, "size above 2^31-1");
  if (C > (1 << 26)) return fail(WKV_ERR_UNSUPPORTED, "C above 2^26");
  constexpr int64_t kMost = (int64_t)1 << 40;
  if (B > 0 && C > 0 && (B > kMost / C || (T > 0 && B * C > kMost / T)))
    return fail(WKV_ERR_UNSUPPORTED, "problem above 2^40 elements");
  if (B * ceil_div(C, 32) > (1 << 26)) return fail(WKV_ERR_UNSUPPORTED, "B * C too large for one launch");
  return WKV_OK;
}

wkv_status check_conv(int64_t B, int64_t T, int64_t C, int dtype, int64_t W) {
  if (wkv_status s = check_act(B, T, C, dtype)) return s;
  if (W < 2 || W > 4) return fail(WKV_ERR_UNSUPPORTED, "W must be 2, 3 or 4");
  return WKV_OK;
}

cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

wkv_status zero(void* p, size_t bytes, void* stream) {
  if (!p || bytes == 0) return WKV_OK;
  return cudaMemsetAsync(p, 0, bytes, as_stream(stream)) == cudaSuccess ? WKV_OK
                                                                         : fail(WKV_ERR_CUDA, "cudaMemsetAsync failed");
}
size_t elem_bytes(int dtype) { return dtype == WKV_BF16 ? 2 : 4; }

}  // namespace
}  // namespace wkv

using namespace wkv;

// ---------------------------------------------------------------------------
// short causal convolution
// ---------------------------------------------------------------------------

WKV_EXPORT wkv_status wkv_conv_forward(int64_t B, int64_t T, int64_t C, int dtype, int64_t W, int silu, const void* x,
                                       const float* weight, const float* bias, const void* x_prev, void* y,
                                       void* stream) {
  if (wkv_status s = check_conv(B, T, C, dtype, W)) return s;
  if (B == 0 || T == 0 || C == 0) return WKV_OK;
  REQUIRE_PTR(x, "x");
  REQUIRE_PTR(weight, "weight");
  OPTIONAL_PTR(bias, "bias");
  OPTIONAL_PTR(x_prev, "x_prev");
  REQUIRE_PTR(y, "y");
  ConvArgs a{};
  a.B = B, a.T = T, a.C = C, a.dtype = dtype, a.W = (int)W, a.silu = silu != 0;
  a.x = x, a.weight = weight, a.bias = bias, a.x_prev = x_prev, a.y = y;
  const char* why = "";
  return ended(launch_conv_forward(a, as_stream(stream), &why), why);
}

WKV_EXPORT size_t wkv_conv_backward_workspace_bytes(int64_t B, int64_t T, int64_t C, int dtype, int64_t W) {
  if (B <= 0 || T <= 0 || C <= 0 || W < 2 || W > 4 || (dtype != WKV_F32 && dtype != WKV_BF16)) return 0;
  return (size_t)(W + 1) * (size_t)B * (size_t)conv_bwd_shape(B, T, C).nrun * (size_t)C * sizeof(float);
}

WKV_EXPORT wkv_status wkv_conv_backward(int64_t B, int64_t T, int64_t C, int dtype, int64_t W, int silu, const void* x,
                                        const float* weight, const float* bias, const void* x_prev, const void* gy,
                                        void* gx, float* gweight, float* gbias, void* gx_prev, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  if (wkv_status s = check_conv(B, T, C, dtype, W)) return s;
  if (C == 0) return WKV_OK;
  REQUIRE_PTR(gweight, "gweight");
  OPTIONAL_PTR(gbias, "gbias");
  OPTIONAL_PTR(gx_prev, "gx_prev");
  if (B == 0 || T == 0) {
    // nothing flows back
    if (wkv_status s = zero(gweight, (size_t)W * C * sizeof(float), stream)) return s;
    if (wkv_status s = zero(gbias, (size_t)C * sizeof(float), stream)) return s;
    return zero(gx_prev, (size_t)B * (W - 1) * C * elem_bytes(dtype), stream);
  }
  REQUIRE_PTR(x, "x");
  REQUIRE_PTR(weight, "weight");
  OPTIONAL_PTR(bias, "bias");
  OPTIONAL_PTR(x_prev, "x_prev");
  REQUIRE_PTR(gy, "gy");
  REQUIRE_PTR(gx, "gx");
  REQUIRE_PTR(workspace, "workspace");
  if (workspace_bytes < wkv_conv_backward_workspace_bytes(B, T, C, dtype, W))
    return fail(WKV_ERR_INVALID_ARG, "workspace_bytes below wkv_conv_backward_workspace_bytes()");
  ConvArgs a{};
  a.B = B, a.T = T, a.C = C, a.dtype = dtype, a.W = (int)W, a.silu = silu != 0;
  a.x = x, a.weight = weight, a.bias = bias, a.x_prev = x_prev;
  a.gy = gy, a.gx = gx, a.gweight = gweight, a.gbias = gbias, a.gx_prev = gx_prev, a.part = static_cast<float*>(workspace);
  const char* why = "";
  return ended(launch_conv_backward(a, as_stream(stream), &why), why);
}

WKV_EXPORT wkv_status wkv_conv_chunk_step(int64_t S, int64_t C, int dtype, int64_t W, int silu, const void* x,
                                          const float* weight, const float* bias, void* y, int64_t n_tokens,
                                          const int32_t* cu_tokens, void* state, void* stream) {
  if (n_tokens < 0) return fail(WKV_ERR_INVALID_ARG, "negative n_tokens");
  if (wkv_status s = check_conv(S, 1, C, dtype, W)) return s;
  if (wkv_status s = check_conv(1, n_tokens, C, dtype, W)) return s;
  if (S == 0 || C == 0) return WKV_OK;
  REQUIRE_PTR(weight, "weight");
  OPTIONAL_PTR(bias, "bias");
  REQUIRE_PTR(cu_tokens, "cu_tokens");
  REQUIRE_PTR(state, "state");
  if (n_tokens > 0) {
    REQUIRE_PTR(x, "x");
    REQUIRE_PTR(y, "y");
  }
  unsigned* err = nullptr;
  if (wkv_status s = device_error_word(&err)) return s;
  ConvArgs a{};
  a.B = S, a.C = C, a.dtype = dtype, a.W = (int)W, a.silu = silu != 0;
  a.x = x, a.weight = weight, a.bias = bias, a.y = y, a.n_tokens = n_tokens, a.cu = cu_tokens, a.state = state;
  const char* why = "";
  return ended(launch_conv_chunk_step(a, as_stream(stream), err, &why), why);
}

WKV_EXPORT wkv_status wkv_conv_decode_step(int64_t S, int64_t C, int dtype, int64_t W, int silu, const void* x,
                                           const float* weight, const float* bias, void* y, void* state,
                                           void* stream) {
  if (wkv_status s = check_conv(S, 1, C, dtype, W)) return s;
  if (S == 0 || C == 0) return WKV_OK;
  REQUIRE_PTR(x, "x");
  REQUIRE_PTR(weight, "weight");
  OPTIONAL_PTR(bias, "bias");
  REQUIRE_PTR(y, "y");
  REQUIRE_PTR(state, "state");
  ConvArgs a{};
  a.B = S, a.C = C, a.dtype = dtype, a.W = (int)W, a.silu = silu != 0;
  a.x = x, a.weight = weight, a.bias = bias, a.y = y, a.state = state;
  const char* why = "";
  return ended(launch_conv_decode_step(a, as_stream(stream), &why), why);
}

// ---------------------------------------------------------------------------
// per-head norm with position rotation
// ---------------------------------------------------------------------------

static wkv_status check_norm(int64_t B, int64_t T, int64_t Hq, int64_t Hk, int64_t K, int64_t R, int dtype, float eps,
                             const int32_t* positions, int64_t pos_offset, int interleaved) {
  if (B < 0 || T < 0 || Hq < 0 || Hk < 0 || K < 0 || R < 0) return fail(WKV_ERR_INVALID_ARG, "negative size");
  if (dtype != WKV_F32 && dtype != WKV_BF16) return fail(WKV_ERR_INVALID_ARG, "unknown dtype");
  if (!(eps >= 0.f)) return fail(WKV_ERR_INVALID_ARG, "eps must be >= 0");
  if (K < 8 || K > 256 || K % 8) return fail(WKV_ERR_UNSUPPORTED, "K must be a multiple of 8 in 8..256");
  if (R > K) return fail(WKV_ERR_INVALID_ARG, "R above K");
  if (R % (interleaved ? 2 : 16))
    return fail(WKV_ERR_UNSUPPORTED, "R must be a multiple of 16 (of 2 if interleaved)");
  constexpr int64_t kMost = (int64_t)1 << 40;
  if (T > INT32_MAX || B > INT32_MAX || Hq > 65535 || Hk > 65535) return fail(WKV_ERR_UNSUPPORTED, "size out of range");
  if (B * T > INT32_MAX || B * T > kMost / std::max<int64_t>(1, (Hq + Hk) * K))
    return fail(WKV_ERR_UNSUPPORTED, "B * T above 2^31-1 or problem above 2^40 elements");
  constexpr int64_t kFar = (int64_t)1 << 53;  // positions that float64 holds
  if (R > 0 && !positions && (pos_offset < -kFar || pos_offset > kFar - T))
    return fail(WKV_ERR_UNSUPPORTED, "pos_offset + t beyond 2^53");
  return WKV_OK;
}

WKV_EXPORT wkv_status wkv_norm_rotate(int64_t B, int64_t T, int64_t Hq, int64_t Hk, int64_t K, int64_t R, int dtype,
                                      const void* q, const void* k, const float* q_weight, const float* k_weight,
                                      float eps, const float* inv_freq, const int32_t* positions, int64_t pos_offset,
                                      int interleaved, void* q_out, void* k_out, void* stream) {
  if (wkv_status s = check_norm(B, T, Hq, Hk, K, R, dtype, eps, positions, pos_offset, interleaved)) return s;
  if (B == 0 || T == 0 || Hq + Hk == 0) return WKV_OK;
  if (Hq > 0) {
    REQUIRE_PTR(q, "q");
    REQUIRE_PTR(q_out, "q_out");
    OPTIONAL_PTR(q_weight, "q_weight");
  }
  if (Hk > 0) {
    REQUIRE_PTR(k, "k");
    REQUIRE_PTR(k_out, "k_out");
    OPTIONAL_PTR(k_weight, "k_weight");
  }
  if (R > 0) {
    REQUIRE_PTR(inv_freq, "inv_freq");
    OPTIONAL_PTR(positions, "positions");
  }
  NormArgs a{};
  a.tokens = B * T, a.T = T, a.Hq = (int)Hq, a.Hk = (int)Hk, a.K = (int)K, a.R = (int)R, a.dtype = dtype;
  a.interleaved = interleaved != 0, a.q = q, a.k = k, a.wq = Hq > 0 ? q_weight : nullptr;
  a.wk = Hk > 0 ? k_weight : nullptr;
  a.eps = eps, a.inv_freq = inv_freq, a.positions = positions, a.pos_offset = pos_offset;
  a.q_out = q_out, a.k_out = k_out;
  const char* why = "";
  return ended(launch_norm_rotate(a, as_stream(stream), &why), why);
}

WKV_EXPORT size_t wkv_norm_rotate_backward_workspace_bytes(int64_t B, int64_t T, int64_t Hq, int64_t Hk, int64_t K) {
  if (B <= 0 || T <= 0 || Hq < 0 || Hk < 0 || Hq + Hk <= 0 || K < 8 || K > 256 || K % 8 || B > INT32_MAX ||
      T > INT32_MAX || B * T > INT32_MAX)
    return 0;
  return 2 * (size_t)norm_bwd_blocks(B * T, Hq, Hk, K) * (size_t)K * sizeof(float);
}

WKV_EXPORT wkv_status wkv_norm_rotate_backward(int64_t B, int64_t T, int64_t Hq, int64_t Hk, int64_t K, int64_t R,
                                               int dtype, const void* q, const void* k, const void* gq_out,
                                               const void* gk_out, const float* q_weight, const float* k_weight,
                                               float eps, const float* inv_freq, const int32_t* positions,
                                               int64_t pos_offset, int interleaved, void* gq, void* gk,
                                               float* gq_weight, float* gk_weight, void* workspace,
                                               size_t workspace_bytes, void* stream) {
  if (wkv_status s = check_norm(B, T, Hq, Hk, K, R, dtype, eps, positions, pos_offset, interleaved)) return s;
  OPTIONAL_PTR(gq_weight, "gq_weight");
  OPTIONAL_PTR(gk_weight, "gk_weight");
  const bool none = B == 0 || T == 0;
  if (none || Hq == 0) {
    if (wkv_status s = zero(gq_weight, (size_t)K * sizeof(float), stream)) return s;
    gq_weight = nullptr;
  }
  if (none || Hk == 0) {
    if (wkv_status s = zero(gk_weight, (size_t)K * sizeof(float), stream)) return s;
    gk_weight = nullptr;
  }
  if (none || Hq + Hk == 0) return WKV_OK;
  if (Hq > 0) {
    REQUIRE_PTR(q, "q");
    REQUIRE_PTR(gq_out, "gq_out");
    REQUIRE_PTR(gq, "gq");
    OPTIONAL_PTR(q_weight, "q_weight");
  }
  if (Hk > 0) {
    REQUIRE_PTR(k, "k");
    REQUIRE_PTR(gk_out, "gk_out");
    REQUIRE_PTR(gk, "gk");
    OPTIONAL_PTR(k_weight, "k_weight");
  }
  if (R > 0) {
    REQUIRE_PTR(inv_freq, "inv_freq");
    OPTIONAL_PTR(positions, "positions");
  }
  REQUIRE_PTR(workspace, "workspace");
  if (workspace_bytes < wkv_norm_rotate_backward_workspace_bytes(B, T, Hq, Hk, K))
    return fail(WKV_ERR_INVALID_ARG, "workspace_bytes below wkv_norm_rotate_backward_workspace_bytes()");
  NormArgs a{};
  a.tokens = B * T, a.T = T, a.Hq = (int)Hq, a.Hk = (int)Hk, a.K = (int)K, a.R = (int)R, a.dtype = dtype;
  a.interleaved = interleaved != 0, a.q = q, a.k = k, a.gq = gq_out, a.gk = gk_out;
  a.wq = Hq > 0 ? q_weight : nullptr, a.wk = Hk > 0 ? k_weight : nullptr;
  a.eps = eps, a.inv_freq = inv_freq, a.positions = positions, a.pos_offset = pos_offset;
  a.q_out = gq, a.k_out = gk, a.gwq = gq_weight, a.gwk = gk_weight, a.part = static_cast<float*>(workspace);
  const char* why = "";
  return ended(launch_norm_rotate_backward(a, as_stream(stream), &why), why);
}

// ---------------------------------------------------------------------------
// selective scan
// ---------------------------------------------------------------------------

static wkv_status check_scan(int64_t B, int64_t T, int64_t C, int64_t N, int64_t G, int dtype) {
  if (N < 0 || G < 0) return fail(WKV_ERR_INVALID_ARG, "negative size");
  if (wkv_status s = check_act(B, T, C, dtype)) return s;
  if (N < 4 || N > 64 || N % 4) return fail(WKV_ERR_UNSUPPORTED, "N must be a multiple of 4 in 4..64");
  if (G < 1) return fail(WKV_ERR_INVALID_ARG, "G must be at least 1");
  if (C % G) return fail(WKV_ERR_INVALID_ARG, "C must be a multiple of G");
  const int64_t unit = dtype == WKV_BF16 ? 8 : 4;
  if ((C / G) % unit) return fail(WKV_ERR_UNSUPPORTED, "C / G must be a multiple of 4 (f32) or 8 (bf16)");
  if (B > 0 && C > 0 && ceil_div(std::max<int64_t>(T, 1), WKV_SCAN_CKPT_LEN) > ((int64_t)1 << 40) / N / (B * C))
    return fail(WKV_ERR_UNSUPPORTED, "state checkpoints above 2^40 elements");
  if (B > 0 && T > 0 && B * T > ((int64_t)1 << 40) / (G * N))
    return fail(WKV_ERR_UNSUPPORTED, "B and C above 2^40 elements");
  return WKV_OK;
}

static void set_scan(ScanArgs& a, int64_t B, int64_t T, int64_t C, int64_t N, int64_t G, int dtype, const void* x,
                     const void* dt, const float* A, const void* Bm, const void* Cm, const float* D, const void* z,
                     const float* dt_bias, int softplus) {
  a.B = B, a.T = T, a.C = C, a.N = N, a.G = G, a.dtype = dtype;
  a.x = x, a.dt = dt, a.A = A, a.Bm = Bm, a.Cm = Cm, a.D = D, a.z = z, a.dt_bias = dt_bias, a.softplus = softplus != 0;
}

static size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

static bool scan_sizes_ok(int64_t B, int64_t T, int64_t C, int64_t N, int64_t G) {
  return B > 0 && T > 0 && C > 0 && N >= 4 && N <= 64 && N % 4 == 0 && G >= 1 && C % G == 0;
}

WKV_EXPORT size_t wkv_scan_ckpt_floats(int64_t B, int64_t T, int64_t C, int64_t N) {
  if (B <= 0 || T <= 0 || C <= 0 || N <= 0) return 0;
  return (size_t)B * (size_t)ceil_div(T, WKV_SCAN_CKPT_LEN) * (size_t)C * (size_t)N;
}

WKV_EXPORT size_t wkv_scan_forward_workspace_bytes(int64_t B, int64_t T, int64_t C, int64_t N, int64_t G) {
  if (!scan_sizes_ok(B, T, C, N, G)) return 0;
  return (size_t)scan_carry_floats(B, C, N, scan_fwd_cut(B, T, C, N, G)) * sizeof(float);
}

// The backward's workspace: partial sums, the pieces of the reverse walk,
// then (without ckpt) the regenerated checkpoints and their forward's pieces.
struct ScanBwdSpace {
  size_t bc, a, d, carry, ckpt, fwd, total;
};
static ScanBwdSpace scan_bwd_space(int64_t B, int64_t T, int64_t C, int64_t N, int64_t G, bool has_ckpt) {
  ScanBwdSpace w{};
  const ScanCut cut = scan_bwd_cut(B, T, C, N, G);
  size_t at = 0;
  auto take = [&](size_t floats) {
    const size_t here = at;
    at += round256(floats * sizeof(float));
    return here;
  };
  w.bc = take(2 * (size_t)scan_group_blocks(C, N, G) * B * T * G * N);
  w.a = take(2 * (size_t)cut.rows(B) * C * N);  // float64
  w.d = take(2 * 2 * (size_t)cut.rows(B) * C);
  w.carry = take((size_t)scan_carry_floats(B, C, N, cut));
  if (!has_ckpt) {
    w.ckpt = take(wkv_scan_ckpt_floats(B, T, C, N));
    w.fwd = take((size_t)scan_carry_floats(B, C, N, scan_fwd_cut(B, T, C, N, G)));
  }
  w.total = at;
  return w;
}

WKV_EXPORT size_t wkv_scan_backward_workspace_bytes(int64_t B, int64_t T, int64_t C, int64_t N, int64_t G,
                                                    int has_ckpt) {
  if (!scan_sizes_ok(B, T, C, N, G)) return 0;
  return scan_bwd_space(B, T, C, N, G, has_ckpt != 0).total;
}

WKV_EXPORT wkv_status wkv_scan_forward(int64_t B, int64_t T, int64_t C, int64_t N, int64_t G, int dtype, const void* x,
                                       const void* dt, const float* A, const void* Bm, const void* Cm, const float* D,
                                       const void* z, const float* dt_bias, int dt_softplus, const float* init_state,
                                       void* y, float* final_state, float* ckpt, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  if (wkv_status s = check_scan(B, T, C, N, G, dtype)) return s;
  if (B == 0 || C == 0) return WKV_OK;
  OPTIONAL_PTR(init_state, "init_state");
  OPTIONAL_PTR(final_state, "final_state");
  OPTIONAL_PTR(y, "y");
  OPTIONAL_PTR(ckpt, "ckpt");
  if (T == 0) {
    // no token: the final state is the initial one
    if (!final_state || final_state == init_state) return WKV_OK;
    const size_t bytes = (size_t)B * C * N * sizeof(float);
    if (!init_state) return zero(final_state, bytes, stream);
    return cudaMemcpyAsync(final_state, init_state, bytes, cudaMemcpyDeviceToDevice, as_stream(stream)) == cudaSuccess
               ? WKV_OK
               : fail(WKV_ERR_CUDA, "copy of init_state failed");
  }
  if (!y && !ckpt && !final_state) return fail(WKV_ERR_INVALID_ARG, "y, final_state and ckpt are all NULL");
  REQUIRE_PTR(x, "x");
  REQUIRE_PTR(dt, "dt");
  REQUIRE_PTR(A, "A");
  REQUIRE_PTR(Bm, "Bm");
  REQUIRE_PTR(Cm, "Cm");
  OPTIONAL_PTR(D, "D");
  OPTIONAL_PTR(z, "z");
  OPTIONAL_PTR(dt_bias, "dt_bias");
  const size_t need = wkv_scan_forward_workspace_bytes(B, T, C, N, G);
  if (need > 0) REQUIRE_PTR(workspace, "workspace");
  if (workspace_bytes < need)
    return fail(WKV_ERR_INVALID_ARG, "workspace_bytes below wkv_scan_forward_workspace_bytes()");
  ScanArgs a{};
  set_scan(a, B, T, C, N, G, dtype, x, dt, A, Bm, Cm, D, z, dt_bias, dt_softplus);
  a.init_state = init_state, a.y = y, a.final_state = final_state, a.ckpt = ckpt;
  a.carry = static_cast<float*>(workspace);
  const char* why = "";
  return ended(launch_scan_forward(a, as_stream(stream), &why), why);
}

WKV_EXPORT wkv_status wkv_scan_backward(int64_t B, int64_t T, int64_t C, int64_t N, int64_t G, int dtype, const void* x,
                                        const void* dt, const float* A, const void* Bm, const void* Cm, const float* D,
                                        const void* z, const float* dt_bias, int dt_softplus, const float* init_state,
                                        const void* gy, const float* g_final, const float* ckpt, void* gx, void* gdt,
                                        float* gA, void* gB, void* gC, float* gD, void* gz, float* gdt_bias,
                                        float* g_init, void* workspace, size_t workspace_bytes, void* stream) {
  if (wkv_status s = check_scan(B, T, C, N, G, dtype)) return s;
  if (C == 0) return WKV_OK;
  REQUIRE_PTR(gA, "gA");
  OPTIONAL_PTR(gD, "gD");
  OPTIONAL_PTR(gdt_bias, "gdt_bias");
  OPTIONAL_PTR(g_init, "g_init");
  OPTIONAL_PTR(g_final, "g_final");
  OPTIONAL_PTR(init_state, "init_state");
  if (B == 0 || T == 0) {
    // nothing flows through time: the parameter gradients are zero, g_init = g_final
    if (wkv_status s = zero(gA, (size_t)C * N * sizeof(float), stream)) return s;
    if (wkv_status s = zero(gD, (size_t)C * sizeof(float), stream)) return s;
    if (wkv_status s = zero(gdt_bias, (size_t)C * sizeof(float), stream)) return s;
    const size_t bytes = (size_t)B * C * N * sizeof(float);
    if (!g_init || bytes == 0 || g_init == g_final) return WKV_OK;
    if (!g_final) return zero(g_init, bytes, stream);
    return cudaMemcpyAsync(g_init, g_final, bytes, cudaMemcpyDeviceToDevice, as_stream(stream)) == cudaSuccess
               ? WKV_OK
               : fail(WKV_ERR_CUDA, "copy of g_final failed");
  }
  REQUIRE_PTR(x, "x");
  REQUIRE_PTR(dt, "dt");
  REQUIRE_PTR(A, "A");
  REQUIRE_PTR(Bm, "Bm");
  REQUIRE_PTR(Cm, "Cm");
  OPTIONAL_PTR(D, "D");
  OPTIONAL_PTR(z, "z");
  OPTIONAL_PTR(dt_bias, "dt_bias");
  REQUIRE_PTR(gy, "gy");
  OPTIONAL_PTR(ckpt, "ckpt");
  REQUIRE_PTR(gx, "gx");
  REQUIRE_PTR(gdt, "gdt");
  REQUIRE_PTR(gB, "gB");
  REQUIRE_PTR(gC, "gC");
  if (z) REQUIRE_PTR(gz, "gz");
  REQUIRE_PTR(workspace, "workspace");
  const ScanBwdSpace w = scan_bwd_space(B, T, C, N, G, ckpt != nullptr);
  if (workspace_bytes < w.total)
    return fail(WKV_ERR_INVALID_ARG, "workspace_bytes below wkv_scan_backward_workspace_bytes()");
  char* base = static_cast<char*>(workspace);
  auto at = [&](size_t off) { return reinterpret_cast<float*>(base + off); };
  ScanBwdArgs b{};
  set_scan(b.f, B, T, C, N, G, dtype, x, dt, A, Bm, Cm, D, z, dt_bias, dt_softplus);
  b.f.init_state = init_state;
  const char* why = "";
  if (!ckpt) {
    ScanArgs f = b.f;
    f.ckpt = at(w.ckpt), f.carry = at(w.fwd);
    if (wkv_status s = launch_scan_forward(f, as_stream(stream), &why)) return fail(s, why);
    b.f.ckpt = f.ckpt;
  } else {
    b.f.ckpt = const_cast<float*>(ckpt);
  }
  b.f.carry = at(w.carry);
  b.gy = gy, b.g_final = g_final, b.gx = gx, b.gdt = gdt, b.gA = gA, b.gB = gB, b.gC = gC, b.gD = gD, b.gz = z ? gz : nullptr;
  b.gdt_bias = gdt_bias, b.g_init = g_init;
  b.part_bc = at(w.bc);
  b.part_a = reinterpret_cast<double*>(base + w.a), b.part_d = reinterpret_cast<double*>(base + w.d);
  return ended(launch_scan_backward(b, as_stream(stream), &why), why);
}

WKV_EXPORT wkv_status wkv_scan_chunk_step(int64_t S, int64_t C, int64_t N, int64_t G, int dtype, const void* x,
                                          const void* dt, const float* A, const void* Bm, const void* Cm,
                                          const float* D, const void* z, const float* dt_bias, int dt_softplus, void* y,
                                          int64_t n_tokens, const int32_t* cu_tokens, float* state, void* stream) {
  if (n_tokens < 0) return fail(WKV_ERR_INVALID_ARG, "negative n_tokens");
  if (wkv_status s = check_scan(S, 1, C, N, G, dtype)) return s;
  if (wkv_status s = check_scan(1, n_tokens, C, N, G, dtype)) return s;
  if (S == 0 || C == 0) return WKV_OK;
  REQUIRE_PTR(cu_tokens, "cu_tokens");
  REQUIRE_PTR(state, "state");
  REQUIRE_PTR(A, "A");
  OPTIONAL_PTR(D, "D");
  OPTIONAL_PTR(z, "z");
  OPTIONAL_PTR(dt_bias, "dt_bias");
  if (n_tokens > 0) {
    REQUIRE_PTR(x, "x");
    REQUIRE_PTR(dt, "dt");
    REQUIRE_PTR(Bm, "Bm");
    REQUIRE_PTR(Cm, "Cm");
    REQUIRE_PTR(y, "y");
  }
  unsigned* err = nullptr;
  if (wkv_status s = device_error_word(&err)) return s;
  ScanArgs a{};
  set_scan(a, S, 0, C, N, G, dtype, x, dt, A, Bm, Cm, D, z, dt_bias, dt_softplus);
  a.init_state = state, a.final_state = state, a.y = y, a.n_tokens = n_tokens, a.cu = cu_tokens;
  const char* why = "";
  return ended(launch_scan_chunk_step(a, as_stream(stream), err, &why), why);
}

WKV_EXPORT wkv_status wkv_scan_decode_step(int64_t S, int64_t C, int64_t N, int64_t G, int dtype, const void* x,
                                           const void* dt, const float* A, const void* Bm, const void* Cm,
                                           const float* D, const void* z, const float* dt_bias, int dt_softplus,
                                           void* y, float* state, void* stream) {
  if (wkv_status s = check_scan(S, 1, C, N, G, dtype)) return s;
  if (S == 0 || C == 0) return WKV_OK;
  REQUIRE_PTR(x, "x");
  REQUIRE_PTR(dt, "dt");
  REQUIRE_PTR(A, "A");
  REQUIRE_PTR(Bm, "Bm");
  REQUIRE_PTR(Cm, "Cm");
  OPTIONAL_PTR(D, "D");
  OPTIONAL_PTR(z, "z");
  OPTIONAL_PTR(dt_bias, "dt_bias");
  REQUIRE_PTR(y, "y");
  REQUIRE_PTR(state, "state");
  ScanArgs a{};
  set_scan(a, S, 1, C, N, G, dtype, x, dt, A, Bm, Cm, D, z, dt_bias, dt_softplus);
  a.init_state = state, a.final_state = state, a.y = y;
  const char* why = "";
  return ended(launch_scan_decode_step(a, as_stream(stream), &why), why);
}
