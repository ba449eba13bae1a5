// ssm_norm.cu -- root-mean-square norm of every head of the queries and keys
// and the rotation by position, in one pass, and its backward:
//
//     r = 1 / sqrt(mean(x^2) + eps),  v = x r w,  (v_a, v_b) turned by p f_i
//     gn = the output gradient turned back,  gw = sum gn x r,
//     gx = r (gn w - x r^2 mean(gn w x))
//
// A stream of short rows (token, head): 8 elements per lane, K / 8 lanes
// (rounded up to a power of two) per row, sums by lane exchange. A group of
// lanes keeps its token and walks over heads, the loads of several heads in
// flight, so that the token's sines and cosines stay in registers. They are
// worked out once per token by the CTA: positions reach 2^53, so the angle
// p * f is reduced to half a turn in two float64 parts, and only then evaluated
// in float32, with what the rounding of the half turn leaves added on.
// Halves of a pair i, i + R/2 lie in lanes R/16 apart and are exchanged by
// shuffle.
#include "ssm_device.cuh"

namespace wkv {

namespace {

constexpr int kNormThreads = 256;
constexpr int kNormV = 8;  // elements per lane
constexpr int kNormU = 4;     // heads whose loads are issued together (forward)
constexpr int kNormBwdU = 4;  // (backward)
constexpr int kNormChain = 256;  // float32 additions in a row to a weight gradient (of a token's heads, if those are more)

struct NormRows {
  int64_t tokens, T;
  int Hq, Hk, K, R;
  int gpt;  // groups of lanes per token (a power of two)
  float eps, inv_K;
  const float* inv_freq;
  const int32_t* positions;
  int64_t pos_offset;
};
// Floats of a token's row of cosines (or sines), kept 16-byte aligned.
__host__ __device__ __forceinline__ int norm_row(int R) { return (R / 2 + 3) & ~3; }

// cos and sin of the tokens [t0, t0 + n) into tables of rows.
__device__ __forceinline__ void norm_angles(const NormRows& a, int64_t t0, int n, float* cs, float* sn) {
  const int half = a.R / 2, row = norm_row(a.R);
  for (int i = threadIdx.x; i < n * half; i += kNormThreads) {
    const int t = i / half, f = i - t * half;
    const int64_t tok = t0 + t;
    const int64_t p = a.positions ? (int64_t)a.positions[tok] : a.pos_offset + tok % a.T;
    // p f and 1 / 2 pi in two parts each, so that the turns less the whole
    // ones are right in 64 bits, then half turns in two float32 parts
    constexpr double kInv = 0.15915494309189535, kInvLow = -9.839338337591243e-18;
    const double pd = (double)p, fd = (double)a.inv_freq[f];
    const double angle = pd * fd, angle_low = fma(pd, fd, -angle), turns = angle * kInv;
    const double low = fma(angle_low, kInv, fma(angle, kInvLow, fma(angle, kInv, -turns)));
    const double half = 2.0 * ((turns - rint(turns)) + (low - rint(low)));  // from 2^53 turns on low has whole ones
    const float h = (float)half, rest = __fmul_rn((float)(half - (double)h), 3.14159274f);
    float s, c;
    sincospif(h, &s, &c);
    // turned on by the rest, below 2^-24
    const float s1 = __fmaf_rn(c, rest, s);
    c = __fmaf_rn(-s, rest, c);
    s = s1;
    cs[t * row + f] = c;
    sn[t * row + f] = s;
  }
}

// What a lane needs to turn its 8 elements (entries 8 l .. of a head).
template <bool IL>
struct NormTurn {
  static constexpr int NF = IL ? kNormV / 2 : kNormV;
  float c[NF], s[NF];  // s: with the sign of the other half's term
  int src;             // lane of the other half of the pairs
  int turned;          // how many of the NF factors apply (entries from R on are left as they are)
  // cs, sn: the token's rows, read only if `there`
  __device__ __forceinline__ void load(const float* cs, const float* sn, bool there, int l, int row_lane0, int R) {
    const int lanes = R / (2 * kNormV);  // lanes that hold the first half
    const bool lo = l < lanes, in = l < 2 * lanes;
    turned = !there ? 0 : IL ? min(max(R / 2 - l * NF, 0), NF) : in ? NF : 0;
    src = row_lane0 + (lo ? l + lanes : in ? l - lanes : l);
    const int f0 = IL ? l * NF : (lo ? l : l - lanes) * kNormV;
#pragma unroll
    for (int i = 0; i < NF; ++i) c[i] = 1.f, s[i] = 0.f;
    if (turned) {
#pragma unroll
      for (int i = 0; i < NF; i += 4) {
        const float4 a = *reinterpret_cast<const float4*>(cs + f0 + i), b = *reinterpret_cast<const float4*>(sn + f0 + i);
        c[i] = a.x, c[i + 1] = a.y, c[i + 2] = a.z, c[i + 3] = a.w;
        s[i] = b.x, s[i + 1] = b.y, s[i + 2] = b.z, s[i + 3] = b.w;
      }
      if (!IL && lo) {
#pragma unroll
        for (int i = 0; i < NF; ++i) s[i] = -s[i];
      }
    }
  }
  // By the angle, or (BACK) by minus the angle. All 32 lanes call it.
  template <bool BACK>
  __device__ __forceinline__ void turn(float (&v)[kNormV]) const {
    if constexpr (IL) {
#pragma unroll
      for (int m = 0; m < NF; ++m) {
        if (m < turned) {
          const float ss = BACK ? -s[m] : s[m], x = v[2 * m], y = v[2 * m + 1];
          v[2 * m] = __fmaf_rn(x, c[m], -__fmul_rn(y, ss));
          v[2 * m + 1] = __fmaf_rn(x, ss, __fmul_rn(y, c[m]));
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < kNormV; ++i) {
        const float other = __shfl_sync(0xffffffffu, v[i], src);
        if (turned) v[i] = __fmaf_rn(v[i], c[i], __fmul_rn(other, BACK ? -s[i] : s[i]));
      }
    }
  }
};

template <int LR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int m = 1; m < LR; m *= 2) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, m));
  return v;
}

// The heads of one tensor for a group of lanes: hsub, hsub + gpt, ..; the
// whole warp runs as many steps as any of its groups needs.
template <class E, int LR, bool IL>
__device__ __forceinline__ void norm_heads(const NormRows& a, const E* in, E* out, int H, int64_t tok, bool there, int hsub,
                                           int l, const float* weight, const NormTurn<IL>& turn) {
  const bool on = there && l * kNormV < a.K;
  float w[kNormV];
  ld_param<kNormV>(weight && on ? weight + l * kNormV : nullptr, w, 1.f);
  const int64_t base = tok * H * a.K + l * kNormV;
  for (int h0 = hsub, step = 0; step < H; step += kNormU * a.gpt, h0 += kNormU * a.gpt) {
    Pack<E, kNormV> p[kNormU];
#pragma unroll
    for (int u = 0; u < kNormU; ++u) {
      p[u].zero();
      if (on && h0 + u * a.gpt < H) p[u].load(in + base + (int64_t)(h0 + u * a.gpt) * a.K);
    }
#pragma unroll
    for (int u = 0; u < kNormU; ++u) {
      if (step + u * a.gpt >= H) break;  // no group has such a head
      float v[kNormV], ss = 0.f;
      p[u].get(v);
#pragma unroll
      for (int i = 0; i < kNormV; ++i) ss = __fmaf_rn(v[i], v[i], ss);
      const float rs = rsqrtf(__fmaf_rn(row_sum<LR>(ss), a.inv_K, a.eps));
#pragma unroll
      for (int i = 0; i < kNormV; ++i) v[i] = __fmul_rn(__fmul_rn(v[i], rs), w[i]);
      if (a.R) turn.template turn<false>(v);
      if (on && h0 + u * a.gpt < H) {
        p[u].set(v);
        p[u].store(out + base + (int64_t)(h0 + u * a.gpt) * a.K);
      }
    }
  }
}

// LR lanes per row.
template <class E, int LR, bool IL>
__global__ void __launch_bounds__(kNormThreads) norm_rotate_kernel(NormRows a, const E* q, const E* k,
                                                                   const float* __restrict__ wq,
                                                                   const float* __restrict__ wk, E* q_out, E* k_out) {
  extern __shared__ float4 tab4[];
  constexpr int RP = kNormThreads / LR;  // groups of lanes
  const int ntok = RP / a.gpt, row = norm_row(a.R);
  float* cs = reinterpret_cast<float*>(tab4);
  float* sn = cs + ntok * row;
  const int64_t t0 = (int64_t)blockIdx.x * ntok;
  const int l = threadIdx.x % LR, grp = threadIdx.x / LR, t = grp / a.gpt, hsub = grp % a.gpt;
  const int64_t left = a.tokens - t0;
  NormTurn<IL> turn;
  if (a.R) {
    norm_angles(a, t0, (int)min((int64_t)ntok, left), cs, sn);
    __syncthreads();
    turn.load(cs + t * row, sn + t * row, t < left, l, (threadIdx.x % 32) / LR * LR, a.R);
  }
  norm_heads<E, LR, IL>(a, q, q_out, a.Hq, t0 + t, t < left, hsub, l, wq, turn);
  norm_heads<E, LR, IL>(a, k, k_out, a.Hk, t0 + t, t < left, hsub, l, wk, turn);
}

// The same for the backward; gw: the lane's sums of the weight gradient.
template <class E, int LR, bool IL>
__device__ __forceinline__ void norm_heads_bwd(const NormRows& a, const E* in, const E* gout, E* gin, int H, int64_t tok,
                                               bool there, int hsub, int l, const float (&w)[kNormV],
                                               const NormTurn<IL>& turn, float (&gw)[kNormV]) {
  const bool on = there && l * kNormV < a.K;
  const int64_t base = tok * H * a.K + l * kNormV;
  for (int h0 = hsub, step = 0; step < H; step += kNormBwdU * a.gpt, h0 += kNormBwdU * a.gpt) {
    Pack<E, kNormV> px[kNormBwdU], pg[kNormBwdU];
#pragma unroll
    for (int u = 0; u < kNormBwdU; ++u) {
      px[u].zero();
      pg[u].zero();
      if (on && h0 + u * a.gpt < H) {
        px[u].load(in + base + (int64_t)(h0 + u * a.gpt) * a.K);
        pg[u].load(gout + base + (int64_t)(h0 + u * a.gpt) * a.K);
      }
    }
#pragma unroll
    for (int u = 0; u < kNormBwdU; ++u) {
      if (step + u * a.gpt >= H) break;
      float x[kNormV], g[kNormV], ss = 0.f, dot = 0.f;
      px[u].get(x);
      pg[u].get(g);
      if (a.R) turn.template turn<true>(g);
#pragma unroll
      for (int i = 0; i < kNormV; ++i) {
        ss = __fmaf_rn(x[i], x[i], ss);
        dot = __fmaf_rn(__fmul_rn(g[i], w[i]), x[i], dot);
      }
      ss = row_sum<LR>(ss);
      dot = row_sum<LR>(dot);
      const bool live = on && h0 + u * a.gpt < H;
      // where there is no head nothing may reach the weight sums (eps may be 0)
      const float rs = live ? rsqrtf(__fmaf_rn(ss, a.inv_K, a.eps)) : 0.f;
      const float m = __fmul_rn(__fmul_rn(rs, rs), __fmul_rn(dot, a.inv_K));
#pragma unroll
      for (int i = 0; i < kNormV; ++i) {
        gw[i] = __fmaf_rn(g[i], __fmul_rn(x[i], rs), gw[i]);
        g[i] = __fmul_rn(rs, __fmaf_rn(-x[i], m, __fmul_rn(g[i], w[i])));
      }
      if (live) {
        pg[u].set(g);
        pg[u].store(gin + base + (int64_t)(h0 + u * a.gpt) * a.K);
      }
    }
  }
}

// part: [2][gridDim.x][K] partial weight gradients (q, k).
template <class E, int LR, bool IL>
__global__ void __launch_bounds__(kNormThreads, 2) norm_rotate_bwd_kernel(NormRows a, const E* __restrict__ q,
                                                                       const E* __restrict__ k, const E* gqo,
                                                                       const E* gko, const float* __restrict__ wq,
                                                                       const float* __restrict__ wk, E* gq, E* gk,
                                                                       float* __restrict__ part) {
  extern __shared__ float4 tab4[];
  __shared__ float sums[kNormThreads * kNormV];
  constexpr int RP = kNormThreads / LR;
  const int ntok = RP / a.gpt, row = norm_row(a.R);
  float* cs = reinterpret_cast<float*>(tab4);
  float* sn = cs + ntok * row;
  const int l = threadIdx.x % LR, grp = threadIdx.x / LR, t = grp / a.gpt, hsub = grp % a.gpt;
  const bool on = l * kNormV < a.K;
  float w[2][kNormV], gw[2][kNormV];
  ld_param<kNormV>(wq && on ? wq + l * kNormV : nullptr, w[0], 1.f);
  ld_param<kNormV>(wk && on ? wk + l * kNormV : nullptr, w[1], 1.f);
#pragma unroll
  for (int i = 0; i < kNormV; ++i) gw[0][i] = gw[1][i] = 0.f;
  for (int64_t t0 = (int64_t)blockIdx.x * ntok; t0 < a.tokens; t0 += (int64_t)gridDim.x * ntok) {
    const int64_t left = a.tokens - t0;
    NormTurn<IL> turn;
    if (a.R) {
      __syncthreads();  // the tables of the step before are done with
      norm_angles(a, t0, (int)min((int64_t)ntok, left), cs, sn);
      __syncthreads();
      turn.load(cs + t * row, sn + t * row, t < left, l, (threadIdx.x % 32) / LR * LR, a.R);
    }
    norm_heads_bwd<E, LR, IL>(a, q, gqo, gq, a.Hq, t0 + t, t < left, hsub, l, w[0], turn, gw[0]);
    norm_heads_bwd<E, LR, IL>(a, k, gko, gk, a.Hk, t0 + t, t < left, hsub, l, w[1], turn, gw[1]);
  }
  // the CTA's sums: thread i < K adds element i of its RP groups (8 or more),
  // in eight chains of at most 32
  static_assert(RP % 8 == 0 && RP <= 256, "eight chains");
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kNormV; ++i) sums[threadIdx.x * kNormV + i] = gw[j][i];
    __syncthreads();
    if ((int)threadIdx.x < a.K) {
      float v[8] = {};
      for (int i = 0; i < RP; i += 8)
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = __fadd_rn(v[u], sums[(i + u) * LR * kNormV + threadIdx.x]);
#pragma unroll
      for (int n = 4; n > 0; n /= 2)
#pragma unroll
        for (int u = 0; u < n; ++u) v[u] = __fadd_rn(v[u], v[u + n]);
      part[((int64_t)j * gridDim.x + blockIdx.x) * a.K + threadIdx.x] = v[0];
    }
  }
}

int norm_lanes(int64_t K) { return K <= 8 ? 1 : K <= 16 ? 2 : K <= 32 ? 4 : K <= 64 ? 8 : K <= 128 ? 16 : 32; }

// Groups of lanes per token: one for every 16 heads, whose work pays for the
// group's share of the angles (one for every 8: 107 against 103 us at 32 + 32
// heads of 64, 32,768 tokens), more where there are few tokens, so that they
// spread over the SMs.
int norm_gpt(int64_t tokens, int64_t H, int64_t K) {
  const int64_t groups = kNormThreads / norm_lanes(K);
  int gpt = 1;
  while (gpt < groups && (gpt * 16 < H || (gpt < H && tokens * gpt < 148 * 2 * groups))) gpt *= 2;
  return gpt;
}

NormRows norm_rows(const NormArgs& a) {
  NormRows r;
  r.tokens = a.tokens;
  r.T = std::max<int64_t>(1, a.T);
  r.Hq = a.Hq;
  r.Hk = a.Hk;
  r.K = a.K;
  r.R = a.R;
  r.gpt = norm_gpt(a.tokens, a.Hq + a.Hk, a.K);
  r.eps = a.eps;
  r.inv_K = 1.f / (float)a.K;
  r.inv_freq = a.inv_freq;
  r.positions = a.positions;
  r.pos_offset = a.pos_offset;
  return r;
}

template <class E, int LR, bool IL>
wkv_status run_norm(const NormArgs& a, bool bwd, cudaStream_t st, const char** why) {
  const NormRows r = norm_rows(a);
  const int64_t ntok = kNormThreads / LR / r.gpt;
  const size_t smem = r.R ? 2 * (size_t)ntok * norm_row(r.R) * sizeof(float) : 0;
  if (!bwd) {
    norm_rotate_kernel<E, LR, IL><<<(unsigned)ceil_div(r.tokens, ntok), kNormThreads, smem, st>>>(
        r, static_cast<const E*>(a.q), static_cast<const E*>(a.k), a.wq, a.wk, static_cast<E*>(a.q_out),
        static_cast<E*>(a.k_out));
  } else {
    norm_rotate_bwd_kernel<E, LR, IL>
        <<<(unsigned)norm_bwd_blocks(r.tokens, r.Hq, r.Hk, r.K), kNormThreads, smem, st>>>(
            r, static_cast<const E*>(a.q), static_cast<const E*>(a.k), static_cast<const E*>(a.gq),
            static_cast<const E*>(a.gk), a.wq, a.wk, static_cast<E*>(a.q_out), static_cast<E*>(a.k_out), a.part);
  }
  if (cudaGetLastError() != cudaSuccess) {
    *why = "norm_rotate kernel launch failed";
    return WKV_ERR_CUDA;
  }
  return WKV_OK;
}

template <class E, bool IL>
wkv_status norm_lanes_dispatch(const NormArgs& a, bool bwd, cudaStream_t st, const char** why) {
  switch (norm_lanes(a.K)) {
    case 1: return run_norm<E, 1, IL>(a, bwd, st, why);
    case 2: return run_norm<E, 2, IL>(a, bwd, st, why);
    case 4: return run_norm<E, 4, IL>(a, bwd, st, why);
    case 8: return run_norm<E, 8, IL>(a, bwd, st, why);
    case 16: return run_norm<E, 16, IL>(a, bwd, st, why);
    default: return run_norm<E, 32, IL>(a, bwd, st, why);
  }
}
wkv_status norm_dispatch(const NormArgs& a, bool bwd, cudaStream_t st, const char** why) {
  if (a.dtype == WKV_BF16)
    return a.interleaved ? norm_lanes_dispatch<__nv_bfloat16, true>(a, bwd, st, why)
                         : norm_lanes_dispatch<__nv_bfloat16, false>(a, bwd, st, why);
  return a.interleaved ? norm_lanes_dispatch<float, true>(a, bwd, st, why)
                       : norm_lanes_dispatch<float, false>(a, bwd, st, why);
}

}  // namespace

// Two CTAs per SM, and as many as it takes for a group of lanes to add up no
// more than kNormChain heads of its tokens.
int64_t norm_bwd_blocks(int64_t tokens, int64_t Hq, int64_t Hk, int64_t K) {
  const int64_t gpt = norm_gpt(tokens, Hq + Hk, K), ntok = kNormThreads / norm_lanes(K) / gpt;
  const int64_t steps = ceil_div(tokens, ntok), heads = ceil_div(std::max(Hq, Hk), gpt);  // of a token in one chain
  return std::min(steps, std::max<int64_t>(148 * 2, ceil_div(steps, std::max<int64_t>(1, kNormChain / heads))));
}

wkv_status launch_norm_rotate(const NormArgs& a, cudaStream_t stream, const char** why) {
  return norm_dispatch(a, false, stream, why);
}

wkv_status launch_norm_rotate_backward(const NormArgs& a, cudaStream_t stream, const char** why) {
  if (wkv_status s = norm_dispatch(a, true, stream, why)) return s;
  SumRows<float> sums{};
  sums.rows = norm_bwd_blocks(a.tokens, a.Hq, a.Hk, a.K);
  sums.add(a.part, a.K, a.gwq);
  sums.add(a.part + sums.rows * a.K, a.K, a.gwk);
  return launch_sum_rows(sums, stream, why);
}

}  // namespace wkv
