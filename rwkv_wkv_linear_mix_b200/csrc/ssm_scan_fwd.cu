// ssm_scan_fwd.cu -- forward of the selective scan
//
//     d = softplus(dt + bias),  h_t = e^{d A} h_{t-1} + d x B_t,
//     y_t = (C_t . h_t + D x_t) silu(z_t)
//
// over batches, packed slots and single tokens. Per token and channel it
// takes N exponentials and 4 N float32 operations on 8 bytes of bf16
// activations, so it is bound by the special-function unit (16 results per
// clock and SM) and by instruction issue, not by memory.
//
// A tile of 16 tokens is turned once into what the walk needs of each
// channel: (d, d x) and (D x, silu z), with the logistic functions evaluated
// once per element and not per lane; the next tile's loads are in flight
// during the walk. The state stays in registers. The lanes of a channel sum
// C . h for 4 tokens of 2 channels together in halving steps, which leaves
// each lane whole outputs to finish and store.
//
// Cut launches (too few channels to fill the SMs): the carry kernel runs
// every piece but the last from a zero state, keeping its end state and
// its sum of d (the decay of a whole piece is e^{A sum d}); the main kernel
// folds the pieces before its own and runs it.
#include "ssm_scan.cuh"

namespace wkv {

namespace {

enum ScanMode { kScanMain, kScanCarry, kScanSlots };

template <int CB, int NP>
struct ScanBuf {
  float4 dd[kScanTile][CB / 2];  // per channel pair: d0, d0 x0, d1, d1 x1
  float4 eg[kScanTile][CB / 2];  // D0 x0, gate0, D1 x1, gate1
  float B[kScanTile][NP];
  float C[kScanTile][NP];
};

template <class E, int LPC, int MODE>
__global__ void __launch_bounds__(ScanGeom<E, LPC>::THREADS) scan_fwd_kernel(const ScanParams p) {
  using Geo = ScanGeom<E, LPC>;
  constexpr int CB = Geo::CB, NP = Geo::NP, VN = Geo::VN;
  using Buf = ScanBuf<CB, NP>;
  extern __shared__ float4 smem4[];
  Buf* buf = reinterpret_cast<Buf*>(smem4);
  const ScanPlace w = scan_place<CB>(p);
  const int tid = threadIdx.x;
  if (MODE == kScanCarry && w.seg == p.nseg - 1) return;  // nothing follows the last piece
  int64_t first = w.b * p.T, T = p.T;
  if constexpr (MODE == kScanSlots) {
    const int64_t beg = p.cu[w.b], end = p.cu[w.b + 1];
    if (end == beg) return;
    if (end < beg || beg < 0 || end > p.n_tokens) {
      if (tid == 0 && w.c0 == 0) record_error(p.err, WKV_DEVERR_BAD_SLOT);
      return;
    }
    first = beg;
    T = end - beg;
  }
  const int64_t tbeg = w.seg * p.seg_tokens;
  const int64_t tend = MODE == kScanSlots || w.seg == p.nseg - 1 ? T : tbeg + p.seg_tokens;
  const E* xg = static_cast<const E*>(p.x) + first * p.C;
  const E* dtg = static_cast<const E*>(p.dt) + first * p.C;
  const E* zg = p.z ? static_cast<const E*>(p.z) + first * p.C : nullptr;
  E* yg = static_cast<E*>(p.y);
  if (yg) yg += first * p.C;
  const int64_t GN = p.G * p.N, gN = w.g * p.N;
  const E* Bg = static_cast<const E*>(p.Bm) + first * GN;
  const E* Cg = static_cast<const E*>(p.Cm) + first * GN;

  // the thread's channels in the loads, and their parameters
  const int col = tid % Geo::VPR * VN;
  const bool col_on = w.c0 + col < w.cend;
  float bias[VN], Dv[VN];
  ld_param<VN>(p.dt_bias && col_on ? p.dt_bias + w.c0 + col : nullptr, bias, 0.f);
  ld_param<VN>(MODE != kScanCarry && p.D && col_on ? p.D + w.c0 + col : nullptr, Dv, 0.f);

  ScanRows<E, LPC> rx, rdt, rz;
  ScanVecs<E, LPC> rb, rc;
  auto load = [&](int64_t t0) {
    rx.load(xg, t0, tend, p.C, w.c0, w.cend);
    rdt.load(dtg, t0, tend, p.C, w.c0, w.cend);
    rb.load(Bg, t0, tend, GN, gN, p.N);
    if constexpr (MODE != kScanCarry) {
      rc.load(Cg, t0, tend, GN, gN, p.N);
      if (zg) rz.load(zg, t0, tend, p.C, w.c0, w.cend);
    }
  };
  auto convert = [&](Buf& o, int64_t t0) {
    rb.put(&o.B[0][0]);
    if constexpr (MODE != kScanCarry) rc.put(&o.C[0][0]);
#pragma unroll
    for (int i = 0; i < Geo::PT; ++i) {
      const int t = (tid + i * Geo::THREADS) / Geo::VPR;
      if (t < kScanTile) {
        const bool real = t0 + t < tend;
        float x[VN], dt[VN], z[VN];
        rx.v[i].get(x);
        rdt.v[i].get(dt);
        if (MODE != kScanCarry && zg) rz.v[i].get(z);
#pragma unroll
        for (int n = 0; n < VN; n += 2) {
          float d[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            // a token past the end: d = 0 leaves the state as it is
            d[k] = real ? scan_step_size(dt[n + k], bias[n + k], p.softplus) : 0.f;
          }
          o.dd[t][(col + n) / 2] = make_float4(d[0], __fmul_rn(d[0], x[n]), d[1], __fmul_rn(d[1], x[n + 1]));
          if constexpr (MODE != kScanCarry) {
            const float g0 = zg ? __fmul_rn(z[n], sigmoid_f(z[n])) : 1.f;
            const float g1 = zg ? __fmul_rn(z[n + 1], sigmoid_f(z[n + 1])) : 1.f;
            o.eg[t][(col + n) / 2] = make_float4(__fmul_rn(Dv[n], x[n]), g0, __fmul_rn(Dv[n + 1], x[n + 1]), g1);
          }
        }
      }
    }
  };

  // the thread's channel pair and states
  const int pair = tid / LPC, g = tid % LPC;
  const int64_t c = w.c0 + 2 * pair;
  const bool on = c < w.cend && 4 * g < p.N;  // channel counts are even
  State4 A2[2], h[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    A2[k] = scale4(ld_state(p.A + (c + k) * p.N + 4 * g, on), kLog2e);
    h[k] = ld_state(p.init_state + (w.b * p.C + c + k) * p.N + 4 * g, MODE != kScanCarry && on && p.init_state);
  }
  if constexpr (MODE == kScanMain) {
    const float* sums = p.carry + p.B * p.nseg * p.C * p.N;
    for (int j = 0; j < w.seg; ++j) {
      const int64_t row = (w.b * p.nseg + j) * p.C + c;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (on) {
          const State4 s = ld_state(p.carry + (row + k) * p.N + 4 * g, true);
          const State4 a = scan_decay(sums[row + k], A2[k]);
          h[k].q[0] = fma2(a.q[0], h[k].q[0], s.q[0]);
          h[k].q[1] = fma2(a.q[1], h[k].q[1], s.q[1]);
        }
      }
    }
  }
  float sum_d[2] = {0.f, 0.f};
  const int out0 = reduce_scatter_first<8, LPC>(g);

  const int nt = (int)((tend - tbeg + kScanTile - 1) / kScanTile);
  load(tbeg);
  convert(buf[0], tbeg);
  if (nt > 1) load(tbeg + kScanTile);
  __syncthreads();
  for (int i = 0; i < nt; ++i) {
    const int64_t t0 = tbeg + (int64_t)i * kScanTile;
    if (i + 1 < nt) convert(buf[(i + 1) & 1], t0 + kScanTile);
    if (i + 2 < nt) load(t0 + 2 * kScanTile);
    const Buf& o = buf[i & 1];
    if (MODE == kScanMain && p.ckpt && on) {
      const int64_t m = t0 / kScanTile, nck = (p.T + kScanTile - 1) / kScanTile;
#pragma unroll
      for (int k = 0; k < 2; ++k) st_state(p.ckpt + ((w.b * nck + m) * p.C + c + k) * p.N + 4 * g, h[k]);
    }
    float tile_d[2] = {0.f, 0.f};
#pragma unroll
    for (int tg = 0; tg < kScanTile; tg += 4) {
      float out[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 dd = o.dd[tg + j][pair];
        const State4 Bv = lds_state(&o.B[tg + j][4 * g]);
        scan_absorb(h[0], scan_decay(dd.x, A2[0]), dd.y, Bv);
        scan_absorb(h[1], scan_decay(dd.z, A2[1]), dd.w, Bv);
        if constexpr (MODE != kScanCarry) {
          const State4 Cv = lds_state(&o.C[tg + j][4 * g]);
          out[2 * j] = scan_dot(h[0], Cv);
          out[2 * j + 1] = scan_dot(h[1], Cv);
        } else {
          tile_d[0] = __fadd_rn(tile_d[0], dd.x);
          tile_d[1] = __fadd_rn(tile_d[1], dd.z);
        }
      }
      if constexpr (MODE != kScanCarry) {
        reduce_scatter<8, LPC>(out, tid);
        // out[i] is now value out0 + i: token (out0 + i) / 2, channel (out0 + i) % 2
        if constexpr (LPC <= 4) {
#pragma unroll
          for (int v = 0; v < 8 / LPC; v += 2) {
            const int t = tg + (out0 + v) / 2;
            const float4 e = o.eg[t][pair];
            const float2 y = make_float2(__fmul_rn(__fadd_rn(out[v], e.x), e.y), __fmul_rn(__fadd_rn(out[v + 1], e.z), e.w));
            if (yg && t0 + t < tend && c < w.cend) st_pair(yg + (t0 + t) * p.C + c, y);
          }
        } else {
          const int t = tg + out0 / 2, k = out0 % 2;
          const float4 e = o.eg[t][pair];
          const float y = __fmul_rn(__fadd_rn(out[0], k ? e.z : e.x), k ? e.w : e.y);
          if (yg && t0 + t < tend && c < w.cend && g < 8) yg[(t0 + t) * p.C + c + k] = Elem<E>::from_f32(y);
        }
      }
    }
    sum_d[0] = __fadd_rn(sum_d[0], tile_d[0]);
    sum_d[1] = __fadd_rn(sum_d[1], tile_d[1]);
    __syncthreads();
  }
  if constexpr (MODE == kScanCarry) {
    const int64_t row = (w.b * p.nseg + w.seg) * p.C + c;
    float* sums = p.carry + p.B * p.nseg * p.C * p.N;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (on) st_state(p.carry + (row + k) * p.N + 4 * g, h[k]);
      if (on && g == 0) sums[row + k] = sum_d[k];
    }
  } else if (p.final_state && on && (MODE == kScanSlots || w.seg == p.nseg - 1)) {
#pragma unroll
    for (int k = 0; k < 2; ++k) st_state(p.final_state + (w.b * p.C + c + k) * p.N + 4 * g, h[k]);
  }
}

// One token per slot: a stream of the states. The lanes of a channel pair
// each work the token's step size out for themselves.
constexpr int kDecodeThreads = 128;
template <class E, int LPC>
__global__ void __launch_bounds__(kDecodeThreads) scan_decode_kernel(const ScanParams p) {
  const int64_t i = (int64_t)blockIdx.x * kDecodeThreads + threadIdx.x;
  const int64_t np = p.C / 2, all = p.B * np * LPC;
  const int g = (int)(i % LPC);
  const int64_t k0 = min(i, all - 1) / LPC, s = k0 / np, c = (k0 - s * np) * 2;
  const bool on = i < all && 4 * g < p.N;
  const int64_t grp = c / p.Cg;
  const float2 x = ld_pair(static_cast<const E*>(p.x) + s * p.C + c);
  const float2 dt = ld_pair(static_cast<const E*>(p.dt) + s * p.C + c);
  const float2 z = p.z ? ld_pair(static_cast<const E*>(p.z) + s * p.C + c) : splat2(0.f);
  const float2 bias = p.dt_bias ? ld_pair(p.dt_bias + c) : splat2(0.f);
  const float2 D = p.D ? ld_pair(p.D + c) : splat2(0.f);
  float Bf[4] = {0.f, 0.f, 0.f, 0.f}, Cf[4] = {0.f, 0.f, 0.f, 0.f};
  if (on) {
    Pack<E, 4> pb, pc;
    pb.load(static_cast<const E*>(p.Bm) + (s * p.G + grp) * p.N + 4 * g);
    pc.load(static_cast<const E*>(p.Cm) + (s * p.G + grp) * p.N + 4 * g);
    pb.get(Bf);
    pc.get(Cf);
  }
  const State4 Bv = {{make_float2(Bf[0], Bf[1]), make_float2(Bf[2], Bf[3])}};
  const State4 Cv = {{make_float2(Cf[0], Cf[1]), make_float2(Cf[2], Cf[3])}};
  float out[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float* st = p.final_state + (s * p.C + c + k) * p.N + 4 * g;
    State4 h = ld_state(st, on);
    const State4 A2 = scale4(ld_state(p.A + (c + k) * p.N + 4 * g, on), kLog2e);
    const float d = scan_step_size(k ? dt.y : dt.x, k ? bias.y : bias.x, p.softplus);
    scan_absorb(h, scan_decay(d, A2), __fmul_rn(d, k ? x.y : x.x), Bv);
    out[k] = scan_dot(h, Cv);
    if (on) st_state(st, h);
  }
  // one lane bit at a time, as the walk's halving steps do
#pragma unroll
  for (int m = 1; m < LPC; m *= 2) {
    out[0] = __fadd_rn(out[0], __shfl_xor_sync(0xffffffffu, out[0], m));
    out[1] = __fadd_rn(out[1], __shfl_xor_sync(0xffffffffu, out[1], m));
  }
  if (i < all && g == 0) {
    const float g0 = p.z ? __fmul_rn(z.x, sigmoid_f(z.x)) : 1.f, g1 = p.z ? __fmul_rn(z.y, sigmoid_f(z.y)) : 1.f;
    const float2 y = make_float2(__fmul_rn(__fadd_rn(out[0], __fmul_rn(D.x, x.x)), g0),
                                 __fmul_rn(__fadd_rn(out[1], __fmul_rn(D.y, x.y)), g1));
    st_pair(static_cast<E*>(p.y) + s * p.C + c, y);
  }
}

wkv_status launched(const char* what, const char** why) {
  if (cudaGetLastError() == cudaSuccess) return WKV_OK;
  *why = what;
  return WKV_ERR_CUDA;
}

template <class E, int LPC, int MODE>
wkv_status run_walk(const ScanParams& p, cudaStream_t st, const char** why) {
  using Geo = ScanGeom<E, LPC>;
  constexpr size_t smem = 2 * sizeof(ScanBuf<Geo::CB, Geo::NP>);
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(scan_fwd_kernel<E, LPC, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
          cudaSuccess) {
    *why = "scan kernel: shared memory request failed";
    return WKV_ERR_CUDA;
  }
  const int64_t grid = p.B * p.nseg * p.G * p.nbg;
  scan_fwd_kernel<E, LPC, MODE><<<(unsigned)grid, Geo::THREADS, smem, st>>>(p);
  return launched("scan kernel launch failed", why);
}

template <class E, int LPC>
wkv_status run_forward(const ScanArgs& a, cudaStream_t st, const char** why) {
  const ScanCut cut = scan_fwd_cut(a.B, a.T, a.C, a.N, a.G);
  const ScanParams p = scan_params(a, cut);
  if (cut.nseg > 1)
    if (wkv_status s = run_walk<E, LPC, kScanCarry>(p, st, why)) return s;
  return run_walk<E, LPC, kScanMain>(p, st, why);
}
template <class E, int LPC>
wkv_status run_slots(const ScanArgs& a, cudaStream_t st, unsigned* err, const char** why) {
  ScanParams p = scan_params(a, ScanCut{1, 0});
  p.err = err;
  return run_walk<E, LPC, kScanSlots>(p, st, why);
}
template <class E, int LPC>
wkv_status run_decode(const ScanArgs& a, cudaStream_t st, const char** why) {
  const ScanParams p = scan_params(a, ScanCut{1, 0});
  const int64_t threads = a.B * (a.C / 2) * LPC;
  scan_decode_kernel<E, LPC><<<(unsigned)ceil_div(threads, kDecodeThreads), kDecodeThreads, 0, st>>>(p);
  return launched("scan decode kernel launch failed", why);
}

#define WKV_SCAN_DISPATCH(CALL)                                           \
  const bool bf = a.dtype == WKV_BF16;                                    \
  switch (scan_lanes(a.N)) {                                              \
    case 2: return bf ? CALL(__nv_bfloat16, 2) : CALL(float, 2);          \
    case 4: return bf ? CALL(__nv_bfloat16, 4) : CALL(float, 4);          \
    case 8: return bf ? CALL(__nv_bfloat16, 8) : CALL(float, 8);          \
    default: return bf ? CALL(__nv_bfloat16, 16) : CALL(float, 16);       \
  }

// Pieces along T: none where the channels alone give two CTAs per SM, since
// the carry pass costs most of a second walk; else about four CTAs per SM,
// pieces of at least 4 tiles.
ScanCut cut_for(int64_t ctas, int64_t T) {
  const int64_t tiles = std::max<int64_t>(1, ceil_div(T, kScanTile));
  int64_t nseg = 1;
  if (ctas < 148 * 2) nseg = std::min(ceil_div(148 * 4, std::max<int64_t>(1, ctas)), std::max<int64_t>(1, tiles / 4));
  const int64_t per = ceil_div(tiles, nseg);
  return ScanCut{(int)ceil_div(tiles, per), (int)per};
}

}  // namespace

ScanCut scan_fwd_cut(int64_t B, int64_t T, int64_t C, int64_t N, int64_t G) {
  return cut_for(B * G * scan_group_blocks(C, N, G), T);
}
ScanCut scan_bwd_cut(int64_t B, int64_t T, int64_t C, int64_t N, int64_t G) {
  return cut_for(B * G * scan_group_blocks(C, N, G), T);
}

wkv_status launch_scan_forward(const ScanArgs& a, cudaStream_t stream, const char** why) {
#define CALL(E, L) (run_forward<E, L>(a, stream, why))
  WKV_SCAN_DISPATCH(CALL)
#undef CALL
}
wkv_status launch_scan_chunk_step(const ScanArgs& a, cudaStream_t stream, unsigned* err, const char** why) {
#define CALL(E, L) (run_slots<E, L>(a, stream, err, why))
  WKV_SCAN_DISPATCH(CALL)
#undef CALL
}
wkv_status launch_scan_decode_step(const ScanArgs& a, cudaStream_t stream, const char** why) {
#define CALL(E, L) (run_decode<E, L>(a, stream, why))
  WKV_SCAN_DISPATCH(CALL)
#undef CALL
}

}  // namespace wkv
