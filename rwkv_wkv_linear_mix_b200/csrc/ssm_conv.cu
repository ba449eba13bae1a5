// ssm_conv.cu -- the short causal convolution
//
//     pre_t = bias + sum_j w_j x_{t-W+1+j},   y_t = silu(pre_t) or pre_t
//
// and its backward, with gpre_t = gy_t y'(pre_t):
//
//     gx_t = sum_j w_j gpre_{t+W-1-j},  gw_j = sum gpre_t x_{t-W+1+j},  gbias = sum gpre_t
//
// A pure stream: a thread owns a few channels (forward 16 bytes, backward 4
// channels) over a run of tokens and keeps the last W-1 tokens in registers,
// so that a run reads only W-1 tokens more than it has. Loads of a batch of
// tokens are issued before any of them is used. The backward walks upward
// too: token t's pre-activation gives gpre_t, which completes gx_{t-W+1}; it
// reads W-1 tokens past the end of its run. Parameter gradients leave as one
// partial sum per run, added in a fixed order by a second kernel.
#include "ssm_device.cuh"

namespace wkv {

namespace {

constexpr int kConvThreads = 128;
constexpr int kConvU = 4;     // tokens whose loads are issued together
constexpr int kConvBwdN = 4;  // channels per thread of the backward

template <class E>
constexpr int kConvN = 16 / (int)sizeof(E);  // channels per thread elsewhere

// pre of one token: win[0 .. W-2] the tokens before it (oldest first), cur the token.
template <int W, int N>
__device__ __forceinline__ void conv_pre(const float (&w)[W][N], const float (&bias)[N], const float (&win)[W - 1][N],
                                         const float (&cur)[N], float (&pre)[N]) {
#pragma unroll
  for (int n = 0; n < N; ++n) {
    float s = bias[n];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) s = __fmaf_rn(w[j][n], win[j][n], s);
    pre[n] = __fmaf_rn(w[W - 1][n], cur[n], s);
  }
}
template <int W, int N>
__device__ __forceinline__ void conv_shift(float (&win)[W - 1][N], const float (&cur)[N]) {
#pragma unroll
  for (int n = 0; n < N; ++n) {
#pragma unroll
    for (int j = 0; j + 1 < W - 1; ++j) win[j][n] = win[j + 1][n];
    win[W - 2][n] = cur[n];
  }
}
template <class E, int W, int N>
__device__ __forceinline__ void conv_store(E* y, const float (&pre)[N], bool silu) {
  float o[N];
#pragma unroll
  for (int n = 0; n < N; ++n) o[n] = silu ? __fmul_rn(pre[n], sigmoid_f(pre[n])) : pre[n];
  Pack<E, N> p;
  p.set(o);
  p.store(y);
}
// The W-1 tokens before token t0 of a sequence whose first token is at x and
// whose earlier ones are at prev (null: zeros).
template <class E, int W, int N>
__device__ __forceinline__ void conv_window(const E* x, const E* prev, int64_t t0, int64_t C, float (&win)[W - 1][N]) {
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    const int64_t t = t0 - (W - 1) + j;
    Pack<E, N> p;
    p.zero();
    if (t >= 0)
      p.load(x + t * C);
    else if (prev)
      p.load(prev + (t + W - 1) * C);
    p.get(win[j]);
  }
}

// SLOTS: sequence b is slot b, tokens cu[b] .. cu[b+1] of the packed tensors,
// and x_prev is the slots' state; its tokens are split over the nrun CTAs.
template <class E, int W, bool SLOTS>
__global__ void __launch_bounds__(kConvThreads) conv_fwd_kernel(const E* __restrict__ x, const float* __restrict__ weight,
                                                                const float* __restrict__ bias,
                                                                const E* __restrict__ x_prev, E* __restrict__ y, int64_t T,
                                                                int64_t C, int ncb, int nrun, int64_t Lt, int silu,
                                                                const int32_t* __restrict__ cu, int64_t n_tokens,
                                                                unsigned* err) {
  constexpr int N = kConvN<E>;
  const int cb = (int)(blockIdx.x % ncb);
  const int rest = (int)(blockIdx.x / ncb);
  const int run = rest % nrun;
  const int64_t b = rest / nrun;
  const int64_t c = ((int64_t)cb * kConvThreads + threadIdx.x) * N;
  if (c >= C) return;
  int64_t first = b * T;
  if constexpr (SLOTS) {
    const int64_t beg = cu[b], end = cu[b + 1];
    if (end == beg) return;
    if (end < beg || beg < 0 || end > n_tokens) {
      if (c == 0 && run == 0) record_error(err, WKV_DEVERR_BAD_SLOT);
      return;
    }
    first = beg;
    T = end - beg;
    Lt = (T + nrun - 1) / nrun;
  }
  const int64_t t0 = run * Lt, t1 = t0 + Lt < T ? t0 + Lt : T;
  if (t0 >= t1) return;
  float w[W][N], bi[N], win[W - 1][N];
#pragma unroll
  for (int j = 0; j < W; ++j) ld_param<N>(weight + (int64_t)j * C + c, w[j], 0.f);
  ld_param<N>(bias ? bias + c : nullptr, bi, 0.f);
  const E* xs = x + first * C + c;
  conv_window<E, W, N>(xs, x_prev ? x_prev + b * (W - 1) * C + c : nullptr, t0, C, win);
  const E* xp = xs + t0 * C;
  E* yp = y + (first + t0) * C + c;
  for (int64_t t = t0; t < t1; t += kConvU) {
    Pack<E, N> raw[kConvU];
#pragma unroll
    for (int j = 0; j < kConvU; ++j)
      if (t + j < t1) raw[j].load(xp + j * C);
#pragma unroll
    for (int j = 0; j < kConvU; ++j) {
      if (t + j < t1) {
        float cur[N], pre[N];
        raw[j].get(cur);
        conv_pre<W, N>(w, bi, win, cur, pre);
        conv_store<E, W, N>(yp + j * C, pre, silu);
        conv_shift<W, N>(win, cur);
      }
    }
    xp += kConvU * C;
    yp += kConvU * C;
  }
}

// The slots' new states, once their outputs are written: the last W-1 of the
// old state and the slot's tokens. A thread reads all of its rows first.
template <class E, int W>
__global__ void __launch_bounds__(kConvThreads) conv_state_kernel(const E* __restrict__ x, E* __restrict__ state, int64_t S,
                                                                  int64_t C, const int32_t* __restrict__ cu,
                                                                  int64_t n_tokens) {
  constexpr int N = kConvN<E>;
  const int64_t i = (int64_t)blockIdx.x * kConvThreads + threadIdx.x;
  const int64_t nv = C / N;
  if (i >= S * nv) return;
  const int64_t b = i / nv, c = (i - b * nv) * N;
  const int64_t beg = cu[b], end = cu[b + 1];
  if (end <= beg || beg < 0 || end > n_tokens) return;
  E* st = state + b * (W - 1) * C + c;
  Pack<E, N> rows[W - 1];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    const int64_t t = end - beg - (W - 1) + j;
    if (t >= 0)
      rows[j].load(x + (beg + t) * C + c);
    else
      rows[j].load(st + (t + W - 1) * C);
  }
#pragma unroll
  for (int j = 0; j < W - 1; ++j) rows[j].store(st + j * C);
}

// One token per slot.
template <class E, int W>
__global__ void __launch_bounds__(kConvThreads) conv_decode_kernel(const E* __restrict__ x, const float* __restrict__ weight,
                                                                   const float* __restrict__ bias, E* __restrict__ y,
                                                                   E* __restrict__ state, int64_t S, int64_t C, int silu) {
  constexpr int N = kConvN<E>;
  const int64_t i = (int64_t)blockIdx.x * kConvThreads + threadIdx.x;
  const int64_t nv = C / N;
  if (i >= S * nv) return;
  const int64_t b = i / nv, c = (i - b * nv) * N;
  E* st = state + b * (W - 1) * C + c;
  Pack<E, N> rows[W];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) rows[j].load(st + j * C);
  rows[W - 1].load(x + b * C + c);
  float w[W][N], bi[N], win[W - 1][N], cur[N], pre[N];
#pragma unroll
  for (int j = 0; j < W; ++j) ld_param<N>(weight + (int64_t)j * C + c, w[j], 0.f);
  ld_param<N>(bias ? bias + c : nullptr, bi, 0.f);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) rows[j].get(win[j]);
  rows[W - 1].get(cur);
  conv_pre<W, N>(w, bi, win, cur, pre);
  conv_store<E, W, N>(y + b * C + c, pre, silu);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) rows[j + 1].store(st + j * C);
}

// part: [W + 1][B * nrun][C] partial sums (gw_0 .. gw_{W-1}, gbias).
template <class E, int W>
__global__ void __launch_bounds__(kConvThreads) conv_bwd_kernel(const E* __restrict__ x, const float* __restrict__ weight,
                                                                const float* __restrict__ bias,
                                                                const E* __restrict__ x_prev, const E* __restrict__ gy,
                                                                E* __restrict__ gx, E* __restrict__ gx_prev,
                                                                float* __restrict__ part, int64_t B, int64_t T, int64_t C,
                                                                int ncb, int nrun, int64_t Lt, int silu) {
  constexpr int N = kConvBwdN;
  const int cb = (int)(blockIdx.x % ncb);
  const int rest = (int)(blockIdx.x / ncb);
  const int run = rest % nrun;
  const int64_t b = rest / nrun;
  const int64_t c = ((int64_t)cb * kConvThreads + threadIdx.x) * N;
  if (c >= C) return;
  const int64_t t0 = run * Lt, t1 = t0 + Lt < T ? t0 + Lt : T;
  float w[W][N], bi[N], win[W - 1][N];
#pragma unroll
  for (int j = 0; j < W; ++j) ld_param<N>(weight + (int64_t)j * C + c, w[j], 0.f);
  ld_param<N>(bias ? bias + c : nullptr, bi, 0.f);
  const int64_t row = b * T * C + c;
  conv_window<E, W, N>(x + row, x_prev ? x_prev + b * (W - 1) * C + c : nullptr, t0, C, win);
  float gwin[W - 1][N], gw[W][N], gb[N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    gb[n] = 0.f;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) gwin[j][n] = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) gw[j][n] = 0.f;
  }
  const int64_t stop = t1 + W - 1;  // the last W-1 steps only complete gx
  for (int64_t t = t0; t < stop; t += kConvU) {
    Pack<E, N> xr[kConvU], gr[kConvU];
#pragma unroll
    for (int j = 0; j < kConvU; ++j) {
      xr[j].zero();
      gr[j].zero();
      if (t + j < stop && t + j < T) {
        xr[j].load(x + row + (t + j) * C);
        gr[j].load(gy + row + (t + j) * C);
      }
    }
#pragma unroll
    for (int j = 0; j < kConvU; ++j) {
      if (t + j < stop) {
        float cur[N], g[N], pre[N], o[N];
        xr[j].get(cur);
        gr[j].get(g);
        conv_pre<W, N>(w, bi, win, cur, pre);
        const bool mine = t + j < t1, past = t + j >= T;
#pragma unroll
        for (int n = 0; n < N; ++n) {
          if (silu) {
            // d silu = p (1 + pre (1 - p)), p = sigmoid(pre)
            const float p = sigmoid_f(pre[n]);
            g[n] = __fmul_rn(g[n], __fmul_rn(p, __fmaf_rn(pre[n], __fsub_rn(1.f, p), 1.f)));
          }
          if (mine) {
#pragma unroll
            for (int i = 0; i < W - 1; ++i) gw[i][n] = __fmaf_rn(g[n], win[i][n], gw[i][n]);
            gw[W - 1][n] = __fmaf_rn(g[n], cur[n], gw[W - 1][n]);
            gb[n] = __fadd_rn(gb[n], g[n]);
          }
          if (past) g[n] = 0.f;  // whatever the window holds
          // gx_{t-W+1} = sum_i w_i gpre_{t-i}
          float s = __fmul_rn(w[0][n], g[n]);
#pragma unroll
          for (int i = 1; i < W; ++i) s = __fmaf_rn(w[i][n], gwin[W - 1 - i][n], s);
          o[n] = s;
        }
        const int64_t to = t + j - (W - 1);
        Pack<E, N> q;
        q.set(o);
        if (to >= t0)
          q.store(gx + row + to * C);
        else if (t0 == 0 && gx_prev)
          q.store(gx_prev + (b * (W - 1) + to + W - 1) * C + c);
        conv_shift<W, N>(win, cur);
        conv_shift<W, N>(gwin, g);
      }
    }
  }
  const int64_t rows = B * nrun, prow = b * nrun + run;
#pragma unroll
  for (int j = 0; j < W; ++j)
    *reinterpret_cast<float4*>(part + (j * rows + prow) * C + c) = make_float4(gw[j][0], gw[j][1], gw[j][2], gw[j][3]);
  *reinterpret_cast<float4*>(part + (W * rows + prow) * C + c) = make_float4(gb[0], gb[1], gb[2], gb[3]);
}

ConvShape conv_shape(int64_t B, int64_t T, int64_t C, int vec, int min_run) {
  ConvShape s;
  s.ncb = (int)ceil_div(C, (int64_t)kConvThreads * vec);
  // runs per sequence: enough CTAs for ~16 per SM, runs of at least min_run tokens
  const int64_t want = ceil_div(148 * 16, std::max<int64_t>(1, B * s.ncb));
  const int64_t most = std::max<int64_t>(1, ceil_div(T, min_run));
  const int64_t nrun = std::max<int64_t>(1, std::min(want, most));
  s.Lt = (int)std::max<int64_t>(1, ceil_div(T, nrun));
  s.nrun = (int)std::max<int64_t>(1, ceil_div(T, s.Lt));
  return s;
}

wkv_status launched(const char* what, const char** why) {
  if (cudaGetLastError() == cudaSuccess) return WKV_OK;
  *why = what;
  return WKV_ERR_CUDA;
}

template <class E, int W>
wkv_status run_fwd(const ConvArgs& a, cudaStream_t st, const char** why) {
  const ConvShape s = conv_shape(a.B, a.T, a.C, kConvN<E>, 16);
  conv_fwd_kernel<E, W, false><<<(unsigned)(s.ncb * s.nrun * a.B), kConvThreads, 0, st>>>(
      static_cast<const E*>(a.x), a.weight, a.bias, static_cast<const E*>(a.x_prev), static_cast<E*>(a.y), a.T, a.C, s.ncb,
      s.nrun, s.Lt, a.silu, nullptr, 0, nullptr);
  return launched("conv forward kernel launch failed", why);
}
template <class E, int W>
wkv_status run_chunk(const ConvArgs& a, cudaStream_t st, unsigned* err, const char** why) {
  // the lengths are on the device: the runs are cut for the mean length
  const ConvShape s = conv_shape(a.B, ceil_div(a.n_tokens, a.B), a.C, kConvN<E>, 16);
  conv_fwd_kernel<E, W, true><<<(unsigned)(s.ncb * s.nrun * a.B), kConvThreads, 0, st>>>(
      static_cast<const E*>(a.x), a.weight, a.bias, static_cast<const E*>(a.state), static_cast<E*>(a.y), 0, a.C, s.ncb,
      s.nrun, 0, a.silu, a.cu, a.n_tokens, err);
  if (wkv_status e = launched("conv chunk step kernel launch failed", why)) return e;
  conv_state_kernel<E, W><<<(unsigned)ceil_div(a.B * (a.C / kConvN<E>), kConvThreads), kConvThreads, 0, st>>>(
      static_cast<const E*>(a.x), static_cast<E*>(a.state), a.B, a.C, a.cu, a.n_tokens);
  return launched("conv state kernel launch failed", why);
}
template <class E, int W>
wkv_status run_decode(const ConvArgs& a, cudaStream_t st, const char** why) {
  conv_decode_kernel<E, W><<<(unsigned)ceil_div(a.B * (a.C / kConvN<E>), kConvThreads), kConvThreads, 0, st>>>(
      static_cast<const E*>(a.x), a.weight, a.bias, static_cast<E*>(a.y), static_cast<E*>(a.state), a.B, a.C, a.silu);
  return launched("conv decode kernel launch failed", why);
}
template <class E, int W>
wkv_status run_bwd(const ConvArgs& a, cudaStream_t st, const char** why) {
  const ConvShape s = conv_bwd_shape(a.B, a.T, a.C);
  conv_bwd_kernel<E, W><<<(unsigned)(s.ncb * s.nrun * a.B), kConvThreads, 0, st>>>(
      static_cast<const E*>(a.x), a.weight, a.bias, static_cast<const E*>(a.x_prev), static_cast<const E*>(a.gy),
      static_cast<E*>(a.gx), static_cast<E*>(a.gx_prev), a.part, a.B, a.T, a.C, s.ncb, s.nrun, s.Lt, a.silu);
  if (wkv_status e = launched("conv backward kernel launch failed", why)) return e;
  const int64_t rows = a.B * s.nrun;
  if (wkv_status e = launch_sum_rows(a.part, W, rows, a.C, a.gweight, st, why)) return e;
  return a.gbias ? launch_sum_rows(a.part + W * rows * a.C, 1, rows, a.C, a.gbias, st, why) : WKV_OK;
}

#define WKV_CONV_DISPATCH(CALL)                                                        \
  const bool bf = a.dtype == WKV_BF16;                                                 \
  switch (a.W) {                                                                       \
    case 2: return bf ? CALL(__nv_bfloat16, 2) : CALL(float, 2);                       \
    case 3: return bf ? CALL(__nv_bfloat16, 3) : CALL(float, 3);                       \
    default: return bf ? CALL(__nv_bfloat16, 4) : CALL(float, 4);                      \
  }

}  // namespace

ConvShape conv_bwd_shape(int64_t B, int64_t T, int64_t C) { return conv_shape(B, T, C, kConvBwdN, 32); }

wkv_status launch_conv_forward(const ConvArgs& a, cudaStream_t stream, const char** why) {
#define CALL(E, W) (run_fwd<E, W>(a, stream, why))
  WKV_CONV_DISPATCH(CALL)
#undef CALL
}
wkv_status launch_conv_backward(const ConvArgs& a, cudaStream_t stream, const char** why) {
#define CALL(E, W) (run_bwd<E, W>(a, stream, why))
  WKV_CONV_DISPATCH(CALL)
#undef CALL
}
wkv_status launch_conv_chunk_step(const ConvArgs& a, cudaStream_t stream, unsigned* err, const char** why) {
#define CALL(E, W) (run_chunk<E, W>(a, stream, err, why))
  WKV_CONV_DISPATCH(CALL)
#undef CALL
}
wkv_status launch_conv_decode_step(const ConvArgs& a, cudaStream_t stream, const char** why) {
#define CALL(E, W) (run_decode<E, W>(a, stream, why))
  WKV_CONV_DISPATCH(CALL)
#undef CALL
}

}  // namespace wkv
