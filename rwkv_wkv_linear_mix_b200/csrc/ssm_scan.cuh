// ssm_scan.cuh -- what the kernels of the selective scan share: the launch
// geometry, where a CTA works, and the loads of a tile of tokens.
//
// A thread carries S = 2 or 4 states of each of 2 adjacent channels; LPC lanes
// side by side share the pair, so that S LPC >= N. The states above N are zero
// and stay zero: their B and C are zero, and their lanes take d x and gs for
// zero (an infinite d x of the channel times B = 0 would be NaN). A CTA covers
// CB channels of one group, so that B and C are one row of numbers per token
// for all of them, and walks its tokens in tiles of 16.
//
// Packed pairs hold one state of both channels. Sums over lanes are taken in
// halving steps, and a lane's order of channels and states is chosen so that
// the first steps need no selects: lane bit 0 swaps the two channels, so that
// the second one's sums are always the ones to give away, and (backward) the
// bits above the lane group permute the states likewise. B and C, d and the
// rest lie in shared memory in each order.
#pragma once

#include <float.h>

#include "ssm_device.cuh"

namespace wkv {

constexpr int kScanTile = WKV_SCAN_CKPT_LEN;  // tokens per tile

// S: states per thread.
template <class E, int LPC_, int S_>
struct ScanGeom {
  static constexpr int LPC = LPC_, S = S_;
  static constexpr int NP = S * LPC;                  // padded states
  static constexpr int CB = scan_cta_channels(NP);   // channels per CTA
  static constexpr int HB = CB / 2;                   // channel pairs per CTA
  static constexpr int THREADS = HB * LPC;
  static constexpr int PT = kScanTile * HB / THREADS; // channel pairs a thread converts per tile
  static constexpr int ROWS = THREADS / HB;           // tokens apart
  static constexpr int VN = 16 / (int)sizeof(E);      // channels per 16-byte copy
  static constexpr int VPR = CB / VN;                 // such copies per token
  static constexpr int BPR = NP / 4;                  // 4-state copies of B or C per token
  static_assert(THREADS % 32 == 0 && kScanTile % ROWS == 0, "whole rows");
};

struct ScanParams {
  int64_t B, T, C, N, G, Cg;  // Cg = C / G
  int nbg, nseg;              // CTAs per group; pieces of a cut sequence
  int64_t seg_tokens;
  int softplus;
  const void *x, *dt, *Bm, *Cm, *z;
  const float *A, *D, *dt_bias, *init_state;
  void* y;
  float *final_state, *ckpt, *carry;
  int64_t final_step;  // floats between the final states of two sequences
  const int32_t* cu;
  int64_t n_tokens;
  unsigned* err;
  // backward
  const void* gy;
  const float* g_final;
  void *gx, *gdt, *gz;
  float *g_init, *part_bc;
  double *part_a, *part_d;
  // sequences that are not cut; pieces of all
  int64_t whole, rows;
};

// Where a CTA works: sequence b, piece seg up to its last, of all pieces the
// row-th, group g, channels c0 .. cend-1 (at most CB of them), block blk of
// the group. The pieces of cut sequences come after the whole sequences; MIXED:
// a launch may have both (the forward cuts all or none).
struct ScanPlace {
  int64_t b, c0, cend, row;
  int g, blk, seg, last;
};
template <int CB, bool MIXED>
__device__ __forceinline__ ScanPlace scan_place(const ScanParams& p) {
  ScanPlace w;
  const unsigned ncb = (unsigned)(p.G * p.nbg);
  const unsigned cb = blockIdx.x % ncb, row = blockIdx.x / ncb, whole = MIXED ? (unsigned)p.whole : 0;
  w.row = row;
  if (MIXED && row < whole) {
    w.seg = w.last = 0;
    w.b = row;
  } else {
    w.seg = (int)((row - whole) % (unsigned)p.nseg);
    w.last = p.nseg - 1;
    w.b = whole + (row - whole) / (unsigned)p.nseg;
  }
  w.g = (int)(cb / (unsigned)p.nbg);
  w.blk = (int)(cb % (unsigned)p.nbg);
  w.c0 = w.g * p.Cg + (int64_t)w.blk * CB;
  w.cend = min((w.g + 1) * p.Cg, w.c0 + CB);
  return w;
}

// A tile of tokens as stored: NT activations, B and C, with zeros past the
// sequence, the group's channels and the N states.
template <class E, class Geo, int NT>
struct ScanRaw {
  E act[NT][kScanTile][Geo::CB];
  E bc[2][kScanTile][Geo::NP];

  // B or C into float32 rows [16][V][NP], row m of a token with state n at n ^ m
  template <int V>
  __device__ __forceinline__ void put_bc(int which, float* table) const {
#pragma unroll
    for (int i = 0; i < (kScanTile * Geo::BPR + Geo::THREADS - 1) / Geo::THREADS; ++i) {
      const int k = (int)threadIdx.x + i * Geo::THREADS;
      if (k < kScanTile * Geo::BPR) {
        Pack<E, 4> v;
        v.load(&bc[which][0][0] + 4 * k);
        float f[4];
        v.get(f);
#pragma unroll
        for (int m = 0; m < V; ++m)
          *reinterpret_cast<float4*>(table + (k / Geo::BPR * V + m) * Geo::NP + k % Geo::BPR * 4) =
              make_float4(f[m], f[1 ^ m], f[2 ^ m], f[3 ^ m]);
      }
    }
  }
};

// The copies of a tile that a thread issues: what to read, where to and which
// token, worked out once and moved on tile by tile (worked out anew for each
// tile they were 8 % of the forward's instructions).
template <class E, class Geo, int NT>
struct ScanCopies {
  static constexpr int ACTS = kScanTile * Geo::VPR, PA = (NT * ACTS + Geo::THREADS - 1) / Geo::THREADS;
  static constexpr int BCS = kScanTile * Geo::BPR, PB = (2 * BCS + Geo::THREADS - 1) / Geo::THREADS;
  static constexpr int kNone = 1 << 20;  // no token: zeros
  const E *a[PA], *b[PB];
  uint32_t a_to[PA], b_to[PB];
  int a_t[PA], b_t[PB];

  // From the tile whose first token is row `row` of the tensors; a tensor may be null.
  __device__ __forceinline__ void init(ScanRaw<E, Geo, NT>& raw, const void* const (&act)[NT], const void* const (&bc)[2],
                                       int64_t row, int64_t C, int64_t c0, int channels, int64_t GN, int64_t gN, int N) {
#pragma unroll
    for (int i = 0; i < PA; ++i) {
      const int k = (int)threadIdx.x + i * Geo::THREADS, w = k / ACTS % NT, t = k % ACTS / Geo::VPR,
                col = k % Geo::VPR * Geo::VN;
      const void* from = act[0];
#pragma unroll
      for (int j = 1; j < NT; ++j) from = w == j ? act[j] : from;
      a_t[i] = from && col < channels ? t : kNone;
      a[i] = static_cast<const E*>(from) + (row + t) * C + c0 + col;
      a_to[i] = smem_u32(&raw.act[w][t][col]);
    }
#pragma unroll
    for (int i = 0; i < PB; ++i) {
      const int k = (int)threadIdx.x + i * Geo::THREADS, w = k / BCS % 2, t = k % BCS / Geo::BPR, n = k % Geo::BPR * 4;
      const void* from = w ? bc[1] : bc[0];
      b_t[i] = from && n < N ? t : kNone;
      b[i] = static_cast<const E*>(from) + (row + t) * GN + gN + n;
      b_to[i] = smem_u32(&raw.bc[w][t][n]);
    }
  }
  // The tile with `left` tokens, into the raw tile `offset` bytes after the first.
  __device__ __forceinline__ void issue(uint32_t offset, int left) const {
#pragma unroll
    for (int i = 0; i < PA; ++i)
      if ((NT * ACTS) % Geo::THREADS == 0 || (int)threadIdx.x + i * Geo::THREADS < NT * ACTS)
        copy_async<16>(a_to[i] + offset, a[i], a_t[i] < left);
#pragma unroll
    for (int i = 0; i < PB; ++i)
      if ((2 * BCS) % Geo::THREADS == 0 || (int)threadIdx.x + i * Geo::THREADS < 2 * BCS)
        copy_async<4 * (int)sizeof(E)>(b_to[i] + offset, b[i], b_t[i] < left);
    copy_async_commit();
  }
  // On by so many rows of the activations and of B and C, in elements.
  __device__ __forceinline__ void step(int64_t by_a, int64_t by_b) {
#pragma unroll
    for (int i = 0; i < PA; ++i) a[i] += by_a;
#pragma unroll
    for (int i = 0; i < PB; ++i) b[i] += by_b;
  }
};

// S states of a pair of channels: n[j] holds a state of the lane's first and
// second channel. (Storing numbers twice in shared memory to spare the moves
// that double them does not pay: a load costs a cycle per register it fills,
// whatever the lanes share.)
template <int S>
struct States {
  float2 n[S];
};
// A row of S numbers of a table, each for both channels.
template <int S>
struct Row {
  float n[S];
};
template <int S>
__device__ __forceinline__ Row<S> ld_row(const float* p) {
  Row<S> r;
  if constexpr (S == 2) {
    const float2 f = *reinterpret_cast<const float2*>(p);
    r.n[0] = f.x, r.n[1] = f.y;
  } else {
    const float4 f = *reinterpret_cast<const float4*>(p);
    r.n[0] = f.x, r.n[1] = f.y, r.n[2] = f.z, r.n[3] = f.w;
  }
  return r;
}
// The order of a lane: its first channel is swap (0 or 1) of the pair, its
// register j holds state j ^ perm of its S.
struct LaneOrder {
  int swap, perm;
};
// From / to [channel][N] rows; p: the lane's states of the pair's channel 0.
template <int S>
__device__ __forceinline__ States<S> ld_states(const float* p, int64_t N, bool there, LaneOrder o) {
  States<S> r;
  const float* a = p + (o.swap ? N : 0);
  const float* b = p + (o.swap ? 0 : N);
#pragma unroll
  for (int j = 0; j < S; ++j) r.n[j] = there ? make_float2(a[j ^ o.perm], b[j ^ o.perm]) : splat2(0.f);
  return r;
}
template <int S>
__device__ __forceinline__ void st_states(float* p, int64_t N, const States<S>& s, LaneOrder o) {
  float* a = p + (o.swap ? N : 0);
  float* b = p + (o.swap ? 0 : N);
#pragma unroll
  for (int j = 0; j < S; ++j) {
    a[j ^ o.perm] = s.n[j].x;
    b[j ^ o.perm] = s.n[j].y;
  }
}
// The same for a lane in natural state order, as wide accesses.
template <int S>
__device__ __forceinline__ States<S> ld_states_wide(const float* p, int64_t N, bool there) {
  States<S> r;
  Row<S> a = {}, b = {};
  if (there) {
    a = ld_row<S>(p);
    b = ld_row<S>(p + N);
  }
#pragma unroll
  for (int j = 0; j < S; ++j) r.n[j] = make_float2(a.n[j], b.n[j]);
  return r;
}
template <int S>
__device__ __forceinline__ void st_states_wide(float* p, int64_t N, const States<S>& s, int swap) {
  float* a = p + (swap ? N : 0);
  float* b = p + (swap ? 0 : N);
  if constexpr (S == 2) {
    *reinterpret_cast<float2*>(a) = make_float2(s.n[0].x, s.n[1].x);
    *reinterpret_cast<float2*>(b) = make_float2(s.n[0].y, s.n[1].y);
  } else {
    *reinterpret_cast<float4*>(a) = make_float4(s.n[0].x, s.n[1].x, s.n[2].x, s.n[3].x);
    *reinterpret_cast<float4*>(b) = make_float4(s.n[0].y, s.n[1].y, s.n[2].y, s.n[3].y);
  }
}
// A log2 e, so that a decay is one exponential. Kept finite: d = 0, which
// passes over the tokens behind the last, must give a decay of 1 for any rate.
__device__ __forceinline__ float scan_rate(float A) {
  const float r = __fmul_rn(A, kLog2e);
  return r < -FLT_MAX ? -FLT_MAX : r;
}
template <int S>
__device__ __forceinline__ States<S> scan_rates(const States<S>& A) {
  States<S> r;
#pragma unroll
  for (int j = 0; j < S; ++j) r.n[j] = make_float2(scan_rate(A.n[j].x), scan_rate(A.n[j].y));
  return r;
}

// A pair's d x or gs for a lane of states; zero for one without. Kernels are
// built apart for N that leaves no such lane (PAD false), since the selects
// cost 2 to 5 % of N=12 (B=4 T=2048 C=2048 bf16: forward 198 -> 202 us,
// backward 474 -> 496; N=24: 324 -> 326, 828 -> 813).
template <bool PAD>
__device__ __forceinline__ float2 scan_taken(float x, float y, bool states) {
  return !PAD || states ? make_float2(x, y) : splat2(0.f);
}

// The step sizes d of a pair of channels from what is stored.
__device__ __forceinline__ float2 scan_step_size2(float2 dt, float2 bias, bool softplus) {
  const float2 raw = add2(dt, bias);
  return softplus ? softplus2(raw) : raw;
}
// The decays of the states over step sizes d (A2 = A log2 e). ex2.approx is low
// on average, which a state adds up over the tokens it remembers; the exponent's
// multiply-add makes up for it at no cost. Mean relative error measured against
// float64 (2^20 exponents a range), without and with it: [-0.01, -0.001]
// -1.7e-8 and 3e-9, [-0.1, -0.01] -2.0e-8 and 1e-9, [-0.5, -0.1] -2.0e-8 and
// 2e-9, below that the exponent's own rounding is larger. Above -0.001, where a
// state remembers more than 1,400 tokens, the mean is smaller by itself
// (-5e-9 to -1e-8), and 1.0e-8 to 1.5e-8 with it.
constexpr float kEx2Low = 3.0e-8f;
template <int S>
__device__ __forceinline__ States<S> scan_decay(float2 d, const States<S>& A2) {
  States<S> r;
#pragma unroll
  for (int j = 0; j < S; ++j) r.n[j] = ex2_2(fma2(d, A2.n[j], splat2(kEx2Low)));
  return r;
}
// h <- a h + dx B
template <int S>
__device__ __forceinline__ void scan_absorb(States<S>& h, const States<S>& a, float2 dx, const Row<S>& Bv) {
#pragma unroll
  for (int j = 0; j < S; ++j) h.n[j] = fma2(a.n[j], h.n[j], mul2(dx, splat2(Bv.n[j])));
}
// The sums over the lane's states of a b, of both channels: each two states by
// one multiply-add, then these in pairs, and on in the lane exchanges, so
// that the sum does not depend on how many states a lane holds.
template <int S>
__device__ __forceinline__ float2 scan_dot(const States<S>& a, const States<S>& b) {
  const float2 s = fma2(a.n[1], b.n[1], mul2(a.n[0], b.n[0]));
  if constexpr (S == 4) return add2(s, fma2(a.n[3], b.n[3], mul2(a.n[2], b.n[2])));
  return s;
}
template <int S>
__device__ __forceinline__ float2 scan_dot(const States<S>& a, const Row<S>& b) {
  States<S> r;
#pragma unroll
  for (int j = 0; j < S; ++j) r.n[j] = splat2(b.n[j]);
  return scan_dot<S>(a, r);
}
// h <- e^{d A} h + s, the fold of a piece's end state s; d is the sum of the
// piece's step sizes. The decay is taken in two halves, each kept within
// 2^-126 .. 2^127, and never formed whole: what the walk does token by token
// then holds where it would leave float32. Nothing stays nothing under growth
// past it, a little grows to what it does, an infinity stays one under a decay
// that comes to 0. (A decay below 2^-252 counts as that: what it leaves of a
// number is below 5e-38.) The backward of 1,024 pieces takes 181 us for 169
// (B=1 T=65536 C=16), of eight pieces the same.
template <int S>
__device__ __forceinline__ void scan_fold(States<S>& h, float2 d, const States<S>& A2, const States<S>& s) {
  const float2 half = mul2(d, splat2(0.5f));
#pragma unroll
  for (int j = 0; j < S; ++j) {
    const float2 x = fma2(half, A2.n[j], splat2(kEx2Low));
    const float2 q = ex2_2(make_float2(fminf(fmaxf(x.x, -126.f), 127.f), fminf(fmaxf(x.y, -126.f), 127.f)));
    h.n[j] = fma2(mul2(h.n[j], q), q, s.n[j]);
  }
}
// One number per token of 4 tokens for each of the two channels, summed over
// the LPC lanes of the pair: the lane ends with its first channel's sums of
// tokens pair_sum_first<LPC>(g) .. , kPairSums<LPC> of them (16 lanes: the
// upper 8 have copies).
template <int LPC>
constexpr int kPairSums = LPC >= 8 ? 1 : 8 / LPC;
template <int LPC>
__device__ __forceinline__ int pair_sum_first(int g) {
  return reduce_scatter_first<4, LPC / 2>(g / 2);
}
// The first step, for one token; then the rest, for four.
__device__ __forceinline__ float pair_give(float2 s) { return __fadd_rn(s.x, __shfl_xor_sync(0xffffffffu, s.y, 1)); }
template <int LPC>
__device__ __forceinline__ void pair_sums(float (&v)[4], float (&out)[kPairSums<LPC>], int lane) {
  reduce_scatter<4, LPC / 2, 2>(v, lane);
#pragma unroll
  for (int t = 0; t < kPairSums<LPC>; ++t) out[t] = v[t];
}

// Host: the sequences from `whole` on in at most nseg pieces of the same length
// (4 tiles or more), but for the last, which takes what is left.
inline ScanCut scan_cut(int64_t B, int64_t whole, int64_t nseg, int64_t T) {
  const int64_t tiles = std::max<int64_t>(1, ceil_div(T, kScanTile));
  const int64_t per = ceil_div(tiles, std::max<int64_t>(1, std::min(nseg, tiles / 4)));
  const int64_t n = ceil_div(tiles, per);
  return ScanCut{n > 1 ? whole : B, (int)n, (int)per};
}
// A launch with `ctas` CTAs per sequence. With fewer than `few` in all, every
// sequence is cut for about eight per SM, which is what an SM holds (four: 205
// against 176 us at B=1 T=8191 C=1536); else none is, since the carry pass costs
// most of a second walk.
inline ScanCut scan_cut_few(int64_t B, int64_t ctas, int64_t T, int64_t few) {
  const int64_t all = std::max<int64_t>(1, B * ctas);
  return all < few ? scan_cut(B, 0, ceil_div(148 * 8, all), T) : scan_cut(B, B, 1, T);
}

// Host: the parameters a launch has in common.
inline ScanParams scan_params(const ScanArgs& a, const ScanCut& cut) {
  ScanParams p{};
  p.B = a.B, p.T = a.T, p.C = a.C, p.N = a.N, p.G = a.G, p.Cg = a.C / a.G;
  p.nbg = (int)scan_group_blocks(a.C, a.N, a.G);
  p.nseg = cut.nseg;
  p.whole = cut.whole, p.rows = cut.rows(a.B);
  p.seg_tokens = (int64_t)cut.seg_tiles * kScanTile;
  p.softplus = a.softplus;
  p.x = a.x, p.dt = a.dt, p.Bm = a.Bm, p.Cm = a.Cm, p.z = a.z;
  p.A = a.A, p.D = a.D, p.dt_bias = a.dt_bias, p.init_state = a.init_state;
  p.y = a.y, p.final_state = a.final_state, p.ckpt = a.ckpt, p.carry = a.carry;
  p.final_step = a.C * a.N;
  p.cu = a.cu, p.n_tokens = a.n_tokens;
  return p;
}

}  // namespace wkv
