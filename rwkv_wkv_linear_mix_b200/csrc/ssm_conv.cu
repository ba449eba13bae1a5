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
// partial sum per run of at most 256 tokens, added in a fixed order and in
// float64 by a second kernel.
#include "ssm_device.cuh"

namespace wkv {

namespace {

constexpr int kConvThreads = 128;
constexpr int kConvU = 4;        // tokens whose loads are issued together, one batch ahead (forward)
constexpr int kConvBwdU = 4;     // (backward)
constexpr int kConvBwdN = 4;     // channels per thread of the backward
constexpr int kConvMinRun = 16;  // tokens of a run that the forward aims at (conv_shape evens runs out, slots have as many)
static_assert(kConvMinRun >= 3, "only the first run of a slot may look before it");
// Tokens whose parameter gradients are added up in one float32 chain (32,768
// like-signed ones lost 4e-4 of the sum; 3e-6 now).
constexpr int kConvMaxRun = 256;
template <class E>
constexpr int kConvN = 16 / (int)sizeof(E);  // channels per thread elsewhere

// pre of one token: win[0 .. W-2] the tokens before it (oldest first), cur the token.
template <int W, int N>
__device__ __forceinline__ void conv_pre(const float2 (&w)[W][N / 2], const float2 (&bias)[N / 2],
                                         const float2 (&win)[W - 1][N / 2], const float2 (&cur)[N / 2],
                                         float2 (&pre)[N / 2]) {
#pragma unroll
  for (int n = 0; n < N / 2; ++n) {
    float2 s = bias[n];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) s = fma2(w[j][n], win[j][n], s);
    pre[n] = fma2(w[W - 1][n], cur[n], s);
  }
}
template <int W, int N>
__device__ __forceinline__ void conv_shift(float2 (&win)[W - 1][N / 2], const float2 (&cur)[N / 2]) {
#pragma unroll
  for (int n = 0; n < N / 2; ++n) {
#pragma unroll
    for (int j = 0; j + 1 < W - 1; ++j) win[j][n] = win[j + 1][n];
    win[W - 2][n] = cur[n];
  }
}
template <class E, int W, int N, bool SILU>
__device__ __forceinline__ void conv_store(E* y, const float2 (&pre)[N / 2]) {
  float2 o[N / 2];
#pragma unroll
  for (int n = 0; n < N / 2; ++n) o[n] = SILU ? mul2(pre[n], sigmoid2(pre[n])) : pre[n];
  set2<E, N>(o).store(y);
}
// The W-1 tokens before token t0 of a sequence whose first token is at x and
// whose earlier ones are at prev (null: zeros).
template <class E, int W, int N>
__device__ __forceinline__ void conv_window(const E* x, const E* prev, int64_t t0, int64_t C,
                                            float2 (&win)[W - 1][N / 2]) {
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    const int64_t t = t0 - (W - 1) + j;
    Pack<E, N> p;
    p.zero();
    if (t >= 0)
      p.load(x + t * C);
    else if (prev)
      p.load(prev + (t + W - 1) * C);
    get2(p, win[j]);
  }
}

// SLOTS: sequence b is slot b, tokens cu[b] .. cu[b+1] of the packed tensors,
// and x_prev is the slots' state (also `state`, to be written); its tokens are
// split over the nrun CTAs,
// kConvMinRun tokens or more to each.
template <class E, int W, bool SILU, bool SLOTS>
__global__ void __launch_bounds__(kConvThreads) conv_fwd_kernel(const E* __restrict__ x, const float* __restrict__ weight,
                                                                const float* __restrict__ bias,
                                                                const E* x_prev, E* state, E* __restrict__ y, int64_t T,
                                                                int64_t C, int ncb, int nrun, int64_t Lt,
                                                                const int32_t* __restrict__ cu, int64_t n_tokens,
                                                                unsigned* err) {
  constexpr int N = kConvN<E>, U = kConvU;
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
    Lt = max((T + nrun - 1) / nrun, (int64_t)kConvMinRun);
  }
  const int64_t t0 = run * Lt;
  if (t0 >= T) return;
  int left = (int)min(Lt, T - t0);  // tokens of the run still to load
  const E* xs = x + first * C + c;
  const E* xp = xs + t0 * C;
  E* yp = y + (first + t0) * C + c;
  Pack<E, N> raw[U];
#pragma unroll
  for (int j = 0; j < U; ++j)
    if (j < left) raw[j].load(xp + j * C);
  float2 w[W][N / 2], bi[N / 2], win[W - 1][N / 2];
#pragma unroll
  for (int j = 0; j < W; ++j) ld_param2<N>(weight + (int64_t)j * C + c, w[j], 0.f);
  ld_param2<N>(bias ? bias + c : nullptr, bi, 0.f);
  conv_window<E, W, N>(xs, x_prev ? x_prev + b * (W - 1) * C + c : nullptr, t0, C, win);
  if (SLOTS && run == 0) {
    // the slot's new state, the last W-1 of the old one and its tokens: the
    // first run alone reads the state (a run has at least W-1 tokens before
    // it), so it may write it while others are at work
    E* st = state + b * (W - 1) * C + c;
    Pack<E, N> rows[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      const int64_t t = T - (W - 1) + j;
      if (t >= 0)
        rows[j].load(xs + t * C);
      else
        rows[j].load(st + (t + W - 1) * C);
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) rows[j].store(st + j * C);
  }
  while (true) {
    Pack<E, N> next[U];
    xp += U * C;
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (U + j < left) next[j].load(xp + j * C);
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (j < left) {
        float2 cur[N / 2], pre[N / 2];
        get2(raw[j], cur);
        conv_pre<W, N>(w, bi, win, cur, pre);
        conv_store<E, W, N, SILU>(yp + j * C, pre);
        conv_shift<W, N>(win, cur);
      }
    }
    left -= U;
    if (left <= 0) break;
    yp += U * C;
#pragma unroll
    for (int j = 0; j < U; ++j) raw[j] = next[j];
  }
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
  float2 w[W][N / 2], bi[N / 2], win[W - 1][N / 2], cur[N / 2], pre[N / 2];
#pragma unroll
  for (int j = 0; j < W; ++j) ld_param2<N>(weight + (int64_t)j * C + c, w[j], 0.f);
  ld_param2<N>(bias ? bias + c : nullptr, bi, 0.f);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) get2(rows[j], win[j]);
  get2(rows[W - 1], cur);
  conv_pre<W, N>(w, bi, win, cur, pre);
  if (silu)
    conv_store<E, W, N, true>(y + b * C + c, pre);
  else
    conv_store<E, W, N, false>(y + b * C + c, pre);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) rows[j + 1].store(st + j * C);
}

// part: [W + 1][B * nrun][C] partial sums (gw_0 .. gw_{W-1}, gbias).
template <class E, int W, bool SILU>
__global__ void __launch_bounds__(kConvThreads, 4) conv_bwd_kernel(const E* __restrict__ x, const float* __restrict__ weight,
                                                                const float* __restrict__ bias,
                                                                const E* __restrict__ x_prev, const E* __restrict__ gy,
                                                                E* __restrict__ gx, E* __restrict__ gx_prev,
                                                                float* __restrict__ part, int64_t B, int64_t T, int64_t C,
                                                                int ncb, int nrun, int64_t Lt) {
  constexpr int N = kConvBwdN, H = N / 2, U = kConvBwdU;
  const int cb = (int)(blockIdx.x % ncb);
  const int rest = (int)(blockIdx.x / ncb);
  const int run = rest % nrun;
  const int64_t b = rest / nrun;
  const int64_t c = ((int64_t)cb * kConvThreads + threadIdx.x) * N;
  if (c >= C) return;
  const int64_t t0 = run * Lt, row = (b * T + t0) * C + c;
  const int n = (int)min(Lt, T - t0);        // tokens of the run
  const int there = (int)min(T - t0, (int64_t)n + W - 1);  // tokens to read: W-1 more complete gx
  const E* xp = x + row;
  const E* gp = gy + row;
  // One batch of loads ahead.
  Pack<E, N> xr[U], gr[U];
  auto fetch = [&](int t, Pack<E, N>(&xo)[U], Pack<E, N>(&go)[U]) {
    if (t + U <= there) {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        xo[j].load(xp + j * C);
        go[j].load(gp + j * C);
      }
    } else {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        xo[j].zero();
        go[j].zero();
        if (t + j < there) {
          xo[j].load(xp + j * C);
          go[j].load(gp + j * C);
        }
      }
    }
    xp += U * C;
    gp += U * C;
  };
  fetch(0, xr, gr);
  float2 w[W][H], bi[H], win[W - 1][H];
#pragma unroll
  for (int j = 0; j < W; ++j) ld_param2<N>(weight + (int64_t)j * C + c, w[j], 0.f);
  ld_param2<N>(bias ? bias + c : nullptr, bi, 0.f);
  conv_window<E, W, N>(x + b * T * C + c, x_prev ? x_prev + b * (W - 1) * C + c : nullptr, t0, C, win);
  float2 gwin[W - 1][H], gw[W][H], gb[H];
#pragma unroll
  for (int i = 0; i < H; ++i) {
    gb[i] = splat2(0.f);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) gwin[j][i] = splat2(0.f);
#pragma unroll
    for (int j = 0; j < W; ++j) gw[j][i] = splat2(0.f);
  }
  E* op = gx + row - (W - 1) * C;  // gx of token t - (W-1)
  // One batch from token t. EDGE: some of its tokens are not the run's own, or
  // complete a gx that is not.
  auto batch = [&](auto edge, int t) {
    constexpr bool EDGE = decltype(edge)::value;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (!EDGE || t + j < n + W - 1) {
        float2 cur[H], g[H], pre[H], o[H];
        get2(xr[j], cur);
        get2(gr[j], g);
        conv_pre<W, N>(w, bi, win, cur, pre);
#pragma unroll
        for (int i = 0; i < H; ++i) {
          if constexpr (SILU) {
            // d silu = p (1 + pre (1 - p)), p = sigmoid(pre)
            const float2 p = sigmoid2(pre[i]);
            g[i] = mul2(g[i], mul2(p, fma2(pre[i], sub2(splat2(1.f), p), splat2(1.f))));
          }
          if (EDGE && t + j >= there) g[i] = splat2(0.f);  // whatever the window holds
          if (!EDGE || t + j < n) {
#pragma unroll
            for (int k = 0; k < W - 1; ++k) gw[k][i] = fma2(g[i], win[k][i], gw[k][i]);
            gw[W - 1][i] = fma2(g[i], cur[i], gw[W - 1][i]);
            gb[i] = add2(gb[i], g[i]);
          }
          // gx_{t-W+1} = sum_k w_k gpre_{t-k}
          float2 s = mul2(w[0][i], g[i]);
#pragma unroll
          for (int k = 1; k < W; ++k) s = fma2(w[k][i], gwin[W - 1 - k][i], s);
          o[i] = s;
        }
        const int to = t + j - (W - 1);  // in the run
        if (!EDGE || to >= 0)
          set2<E, N>(o).store(op + j * C);
        else if (t0 == 0 && gx_prev)
          set2<E, N>(o).store(gx_prev + (b * (W - 1) + to + W - 1) * C + c);
        conv_shift<W, N>(win, cur);
        conv_shift<W, N>(gwin, g);
      }
    }
  };
  for (int t = 0; t < n + W - 1; t += U) {
    Pack<E, N> xn[U], gn[U];
    fetch(t + U, xn, gn);
    if (t >= W - 1 && t + U <= n)
      batch(BoolConst<false>{}, t);
    else
      batch(BoolConst<true>{}, t);
    op += U * C;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      xr[j] = xn[j];
      gr[j] = gn[j];
    }
  }
  const int64_t rows = B * nrun, prow = b * nrun + run;
#pragma unroll
  for (int j = 0; j <= W; ++j) {
    const float2(&v)[H] = j < W ? gw[j < W ? j : 0] : gb;
    set2<float, N>(v).store(part + (j * rows + prow) * C + c);
  }
}

// Runs per sequence: enough for `ctas` CTAs per SM, of about min_run tokens or
// more (evened out, so down to half of that), and of max_run at most.
ConvShape conv_shape(int64_t B, int64_t T, int64_t C, int vec, int min_run, int64_t max_run, int ctas) {
  ConvShape s;
  s.ncb = (int)ceil_div(C, (int64_t)kConvThreads * vec);
  const int64_t want = ceil_div(148 * ctas, std::max<int64_t>(1, B * s.ncb));
  const int64_t most = std::max<int64_t>(1, ceil_div(T, min_run));
  const int64_t nrun = std::max({(int64_t)1, std::min(want, most), ceil_div(T, max_run)});
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
  const ConvShape s = conv_shape(a.B, a.T, a.C, kConvN<E>, kConvMinRun, a.T, 16);
  const auto kernel = a.silu ? conv_fwd_kernel<E, W, true, false> : conv_fwd_kernel<E, W, false, false>;
  kernel<<<(unsigned)(s.ncb * s.nrun * a.B), kConvThreads, 0, st>>>(
      static_cast<const E*>(a.x), a.weight, a.bias, static_cast<const E*>(a.x_prev), nullptr, static_cast<E*>(a.y), a.T, a.C, s.ncb,
      s.nrun, s.Lt, nullptr, 0, nullptr);
  return launched("conv forward kernel launch failed", why);
}
template <class E, int W>
wkv_status run_chunk(const ConvArgs& a, cudaStream_t st, unsigned* err, const char** why) {
  // the lengths are on the device: the runs are cut for the mean length
  const int64_t mean = std::max<int64_t>(1, ceil_div(a.n_tokens, a.B));
  const ConvShape s = conv_shape(a.B, mean, a.C, kConvN<E>, kConvMinRun, mean, 16);
  const auto kernel = a.silu ? conv_fwd_kernel<E, W, true, true> : conv_fwd_kernel<E, W, false, true>;
  kernel<<<(unsigned)(s.ncb * s.nrun * a.B), kConvThreads, 0, st>>>(
      static_cast<const E*>(a.x), a.weight, a.bias, static_cast<const E*>(a.state), static_cast<E*>(a.state),
      static_cast<E*>(a.y), 0, a.C, s.ncb, s.nrun, 0, a.cu, a.n_tokens, err);
  return launched("conv chunk step kernel launch failed", why);
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
  const auto kernel = a.silu ? conv_bwd_kernel<E, W, true> : conv_bwd_kernel<E, W, false>;
  kernel<<<(unsigned)(s.ncb * s.nrun * a.B), kConvThreads, 0, st>>>(
      static_cast<const E*>(a.x), a.weight, a.bias, static_cast<const E*>(a.x_prev), static_cast<const E*>(a.gy),
      static_cast<E*>(a.gx), static_cast<E*>(a.gx_prev), a.part, a.B, a.T, a.C, s.ncb, s.nrun, s.Lt);
  if (wkv_status e = launched("conv backward kernel launch failed", why)) return e;
  SumRows<float> sums{};
  sums.rows = a.B * s.nrun;
  for (int j = 0; j <= W; ++j) sums.add(a.part + j * sums.rows * a.C, a.C, j < W ? a.gweight + j * a.C : a.gbias);
  return launch_sum_rows(sums, st, why);
}

#define WKV_CONV_DISPATCH(CALL)                                                        \
  const bool bf = a.dtype == WKV_BF16;                                                 \
  switch (a.W) {                                                                       \
    case 2: return bf ? CALL(__nv_bfloat16, 2) : CALL(float, 2);                       \
    case 3: return bf ? CALL(__nv_bfloat16, 3) : CALL(float, 3);                       \
    default: return bf ? CALL(__nv_bfloat16, 4) : CALL(float, 4);                      \
  }

}  // namespace

ConvShape conv_bwd_shape(int64_t B, int64_t T, int64_t C) { return conv_shape(B, T, C, kConvBwdN, 32, kConvMaxRun, 16); }

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
