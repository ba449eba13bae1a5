// ssm_norm.cu -- root-mean-square norm of every head of the queries and keys
// and the rotation by position, in one pass, and its backward:
//
//     r = 1 / sqrt(mean(x^2) + eps),  v = x r w,  (v_a, v_b) turned by p f_i
//     gn = the output gradient turned back,  gw = sum gn x r,
//     gx = r (gn w - x r^2 mean(gn w x))
//
// A stream of short rows (token, head): 8 elements per lane, K / 8 lanes
// (rounded up to a power of two) per row, sums by lane exchange. The rows of
// kNormTokens tokens or so go to one CTA, which first works the tokens'
// sines and cosines out once for all their heads: angles p * f reach 2^31
// turns, so they are reduced to half a turn in float64 and only then
// evaluated in float32. Halves of a pair i, i + R/2 lie in lanes R/16 apart
// and are exchanged by shuffle.
#include "ssm_device.cuh"

namespace wkv {

namespace {

constexpr int kNormThreads = 256;
constexpr int kNormV = 8;         // elements per lane
constexpr int kNormMaxTokens = 16;  // tokens per CTA, at most

struct NormRows {
  int64_t tokens, T;
  int Hq, Hk, K, R, tok_cta;  // tok_cta: tokens per CTA and step
  float eps, inv_K;
  const float* inv_freq;
  const int32_t* positions;
  int64_t pos_offset;
};

// cos and sin of the tokens [t0, t0 + n) into [t][R/2] tables.
__device__ __forceinline__ void norm_angles(const NormRows& a, int64_t t0, int n, float* cs, float* sn) {
  const int half = a.R / 2;
  for (int i = threadIdx.x; i < n * half; i += kNormThreads) {
    const int t = i / half, f = i - t * half;
    const int64_t tok = t0 + t;
    const int64_t p = a.positions ? (int64_t)a.positions[tok] : a.pos_offset + tok % a.T;
    // p f / 2 pi, less its whole turns
    double turn = (double)p * ((double)a.inv_freq[f] * 0.15915494309189535);
    turn -= rint(turn);
    float s, c;
    sincospif((float)(2.0 * turn), &s, &c);
    cs[i] = c;
    sn[i] = s;
  }
}

// Turns the 8 elements at e0 = 8 * l of a row (forward: by the angle; BACK:
// by minus the angle). c, s: the token's tables.
template <bool IL, bool BACK>
__device__ __forceinline__ void norm_turn(float (&v)[kNormV], int l, int row_lane0, int R, const float* c, const float* s) {
  const int e0 = l * kNormV;
  if constexpr (IL) {
#pragma unroll
    for (int m = 0; m < kNormV / 2; ++m) {
      if (e0 + 2 * m < R) {
        const float cc = c[e0 / 2 + m], ss = BACK ? -s[e0 / 2 + m] : s[e0 / 2 + m];
        const float a = v[2 * m], b = v[2 * m + 1];
        v[2 * m] = __fmaf_rn(a, cc, -__fmul_rn(b, ss));
        v[2 * m + 1] = __fmaf_rn(a, ss, __fmul_rn(b, cc));
      }
    }
  } else {
    const int lanes = R / (2 * kNormV);  // lanes that hold the first half
    const bool lo = l < lanes, in = l < 2 * lanes;
    const int src = row_lane0 + (lo ? l + lanes : in ? l - lanes : l);
    const int f0 = (lo ? l : l - lanes) * kNormV;
#pragma unroll
    for (int i = 0; i < kNormV; ++i) {
      const float other = __shfl_sync(0xffffffffu, v[i], src);
      if (in) {
        const float cc = c[f0 + i];
        const float ss = (lo != BACK) ? -s[f0 + i] : s[f0 + i];
        v[i] = __fmaf_rn(v[i], cc, __fmul_rn(other, ss));
      }
    }
  }
}

template <int LR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int m = 1; m < LR; m *= 2) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, m));
  return v;
}

// LR lanes per row.
template <class E, int LR, bool IL>
__global__ void __launch_bounds__(kNormThreads) norm_rotate_kernel(NormRows a, const E* q, const E* k,
                                                                   const float* __restrict__ wq,
                                                                   const float* __restrict__ wk, E* q_out, E* k_out) {
  extern __shared__ float tab[];  // cos, then sin: [tok_cta][R/2]
  const int64_t t0 = (int64_t)blockIdx.x * a.tok_cta;
  const int nt = (int)min((int64_t)a.tok_cta, a.tokens - t0);
  float* cs = tab;
  float* sn = tab + a.tok_cta * (a.R / 2);
  const int l = threadIdx.x % LR, row_lane0 = (threadIdx.x % 32) / LR * LR;
  const bool on = l * kNormV < a.K;
  float w[2][kNormV];
  ld_param<kNormV>(wq && on ? wq + l * kNormV : nullptr, w[0], 1.f);
  ld_param<kNormV>(wk && on ? wk + l * kNormV : nullptr, w[1], 1.f);
  norm_angles(a, t0, nt, cs, sn);
  __syncthreads();
  const int H = a.Hq + a.Hk, rows = nt * H;
  constexpr int RP = kNormThreads / LR;  // rows per pass
  for (int r0 = 0; r0 < rows; r0 += RP) {  // whole warps stay: the rows' lanes exchange values
    const int r = r0 + threadIdx.x / LR;
    const bool have = r < rows && on;
    const int t = r / H, h = r - t * H;
    const bool key = h >= a.Hq;
    const int64_t off = key ? ((t0 + t) * a.Hk + (h - a.Hq)) * (int64_t)a.K : ((t0 + t) * a.Hq + h) * (int64_t)a.K;
    Pack<E, kNormV> p;
    p.zero();
    if (have) p.load((key ? k : q) + off + l * kNormV);
    float v[kNormV];
    p.get(v);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < kNormV; ++i) ss = __fmaf_rn(v[i], v[i], ss);
    ss = row_sum<LR>(ss);
    const float rs = rsqrtf(__fmaf_rn(ss, a.inv_K, a.eps));
#pragma unroll
    for (int i = 0; i < kNormV; ++i) v[i] = __fmul_rn(__fmul_rn(v[i], rs), key ? w[1][i] : w[0][i]);
    if (a.R) {
      const int tt = min(t, nt - 1) * (a.R / 2);
      norm_turn<IL, false>(v, l, row_lane0, a.R, cs + tt, sn + tt);
    }
    if (have) {
      p.set(v);
      p.store((key ? k_out : q_out) + off + l * kNormV);
    }
  }
}

// part: [2][gridDim.x][K] partial weight gradients (q, k).
template <class E, int LR, bool IL>
__global__ void __launch_bounds__(kNormThreads) norm_rotate_bwd_kernel(NormRows a, const E* __restrict__ q,
                                                                       const E* __restrict__ k, const E* gqo,
                                                                       const E* gko, const float* __restrict__ wq,
                                                                       const float* __restrict__ wk, E* gq, E* gk,
                                                                       float* __restrict__ part) {
  extern __shared__ float tab[];
  __shared__ float sums[kNormThreads * kNormV];
  float* cs = tab;
  float* sn = tab + a.tok_cta * (a.R / 2);
  const int l = threadIdx.x % LR, row_lane0 = (threadIdx.x % 32) / LR * LR;
  const bool on = l * kNormV < a.K;
  float w[2][kNormV], gw[2][kNormV];
  ld_param<kNormV>(wq && on ? wq + l * kNormV : nullptr, w[0], 1.f);
  ld_param<kNormV>(wk && on ? wk + l * kNormV : nullptr, w[1], 1.f);
#pragma unroll
  for (int i = 0; i < kNormV; ++i) gw[0][i] = gw[1][i] = 0.f;
  const int H = a.Hq + a.Hk;
  constexpr int RP = kNormThreads / LR;
  for (int64_t t0 = (int64_t)blockIdx.x * a.tok_cta; t0 < a.tokens; t0 += (int64_t)gridDim.x * a.tok_cta) {
    const int nt = (int)min((int64_t)a.tok_cta, a.tokens - t0);
    __syncthreads();  // the tables of the step before are done with
    norm_angles(a, t0, nt, cs, sn);
    __syncthreads();
    const int rows = nt * H;
    for (int r0 = 0; r0 < rows; r0 += RP) {
      const int r = r0 + threadIdx.x / LR;
      const bool have = r < rows && on;
      const int t = r / H, h = r - t * H;
      const bool key = h >= a.Hq;
      const int64_t off = key ? ((t0 + t) * a.Hk + (h - a.Hq)) * (int64_t)a.K : ((t0 + t) * a.Hq + h) * (int64_t)a.K;
      Pack<E, kNormV> px, pg;
      px.zero();
      pg.zero();
      if (have) {
        px.load((key ? k : q) + off + l * kNormV);
        pg.load((key ? gko : gqo) + off + l * kNormV);
      }
      float x[kNormV], g[kNormV];
      px.get(x);
      pg.get(g);
      if (a.R) {
        const int tt = min(t, nt - 1) * (a.R / 2);
        norm_turn<IL, true>(g, l, row_lane0, a.R, cs + tt, sn + tt);
      }
      float ss = 0.f, dot = 0.f;
#pragma unroll
      for (int i = 0; i < kNormV; ++i) {
        ss = __fmaf_rn(x[i], x[i], ss);
        dot = __fmaf_rn(__fmul_rn(g[i], key ? w[1][i] : w[0][i]), x[i], dot);
      }
      ss = row_sum<LR>(ss);
      dot = row_sum<LR>(dot);
      const float rs = rsqrtf(__fmaf_rn(ss, a.inv_K, a.eps));
      const float m = __fmul_rn(__fmul_rn(rs, rs), __fmul_rn(dot, a.inv_K));
      float o[kNormV];
#pragma unroll
      for (int i = 0; i < kNormV; ++i) {
        const float gx = __fmul_rn(g[i], __fmul_rn(x[i], rs));
        if (have) {
          if (key)
            gw[1][i] = __fadd_rn(gw[1][i], gx);
          else
            gw[0][i] = __fadd_rn(gw[0][i], gx);
        }
        o[i] = __fmul_rn(rs, __fmaf_rn(-x[i], m, __fmul_rn(g[i], key ? w[1][i] : w[0][i])));
      }
      if (have) {
        pg.set(o);
        pg.store((key ? gk : gq) + off + l * kNormV);
      }
    }
  }
  // the CTA's sums: thread i < LR * 8 adds element i of its RP rows in order
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kNormV; ++i) sums[threadIdx.x * kNormV + i] = gw[j][i];
    __syncthreads();
    if ((int)threadIdx.x < a.K) {
      float s = 0.f;
      for (int i = 0; i < RP; ++i) s = __fadd_rn(s, sums[i * LR * kNormV + threadIdx.x]);
      part[((int64_t)j * gridDim.x + blockIdx.x) * a.K + threadIdx.x] = s;
    }
  }
}

int norm_lanes(int64_t K) { return K <= 8 ? 1 : K <= 16 ? 2 : K <= 32 ? 4 : K <= 64 ? 8 : K <= 128 ? 16 : 32; }

// Tokens per CTA: rows for four passes of its threads.
int norm_tokens(int64_t tokens, int64_t H, int64_t K) {
  const int64_t rows = 4 * kNormThreads / norm_lanes(K);
  const int64_t want = std::min<int64_t>(kNormMaxTokens, ceil_div(rows, std::max<int64_t>(1, H)));
  // few tokens: spread them over the SMs instead
  return (int)std::max<int64_t>(1, std::min(want, tokens / 148));
}

NormRows norm_rows(const NormArgs& a) {
  NormRows r;
  r.tokens = a.tokens;
  r.T = std::max<int64_t>(1, a.T);
  r.Hq = a.Hq;
  r.Hk = a.Hk;
  r.K = a.K;
  r.R = a.R;
  r.tok_cta = norm_tokens(a.tokens, a.Hq + a.Hk, a.K);
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
  const size_t smem = (size_t)r.tok_cta * r.R * sizeof(float);
  if (!bwd) {
    norm_rotate_kernel<E, LR, IL><<<(unsigned)ceil_div(r.tokens, r.tok_cta), kNormThreads, smem, st>>>(
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

int64_t norm_bwd_blocks(int64_t tokens, int64_t Hq, int64_t Hk, int64_t K) {
  return std::min<int64_t>(ceil_div(tokens, norm_tokens(tokens, Hq + Hk, K)), 148 * 4);
}

wkv_status launch_norm_rotate(const NormArgs& a, cudaStream_t stream, const char** why) {
  return norm_dispatch(a, false, stream, why);
}

wkv_status launch_norm_rotate_backward(const NormArgs& a, cudaStream_t stream, const char** why) {
  if (wkv_status s = norm_dispatch(a, true, stream, why)) return s;
  const int64_t rows = norm_bwd_blocks(a.tokens, a.Hq, a.Hk, a.K);
  if (a.gwq)
    if (wkv_status s = launch_sum_rows(a.part, 1, rows, a.K, a.gwq, stream, why)) return s;
  return a.gwk ? launch_sum_rows(a.part + rows * a.K, 1, rows, a.K, a.gwk, stream, why) : WKV_OK;
}

}  // namespace wkv
