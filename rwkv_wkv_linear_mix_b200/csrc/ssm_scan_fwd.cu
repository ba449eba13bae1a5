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

enum { kActX, kActDt, kActZ, kActs };

template <class E, class Geo>
struct ScanFwdShared {
  ScanRaw<E, Geo, kActs> raw[2];         // the tile at work, and the next in flight
  // per channel pair: d0, d1, d0 x0, d1 x1; and with the channels swapped
  // (64 bytes further on in the banks, so that a warp reads both orders at once)
  float4 dd[kScanTile][2][Geo::HB + 4];
  float B[kScanTile][Geo::NP];
  float C[kScanTile][Geo::NP];
};

// Seven CTAs of 4 warps per SM with two states per lane (72 registers): left
// alone the compiler takes up to 168 (prompt, B=8 C=4096: 536 us against 452;
// 9 CTAs, 56 registers: 463).
template <class E, int LPC, int S, bool PAD, int MODE>
__global__ void __launch_bounds__(ScanGeom<E, LPC, S>::THREADS, S == 2 ? 7 : 4) scan_fwd_kernel(const ScanParams p) {
  using Geo = ScanGeom<E, LPC, S>;
  extern __shared__ float4 smem4[];
  auto& sm = *reinterpret_cast<ScanFwdShared<E, Geo>*>(smem4);
  const ScanPlace w = scan_place<Geo::CB, false>(p);
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
  const int nt = (int)((tend - tbeg + kScanTile - 1) / kScanTile);
  const int64_t GN = p.G * p.N;
  const int channels = (int)(w.cend - w.c0);

  // the thread's channel pair and states
  const int pair = tid / LPC, g = tid % LPC, swap = g & 1;
  const LaneOrder order{swap, 0};
  const int64_t c = w.c0 + 2 * pair;
  const bool ch_on = 2 * pair < channels, on = ch_on && S * g < p.N;  // channel counts are even
  const States<S> A2 = scan_rates<S>(ld_states<S>(p.A + c * p.N + S * g, p.N, on, order));
  const float D = MODE != kScanCarry && p.D && ch_on ? p.D[c + swap] : 0.f;
  const int64_t state_at = (w.b * p.C + c) * p.N + S * g;
  States<S> h = ld_states<S>(p.init_state + state_at, p.N, MODE != kScanCarry && on && p.init_state, order);
  if constexpr (MODE == kScanMain) {
    // Through the pieces before this one, the loads of four in flight together
    // (eight spill: 235 against 186 us at B=1 T=65536 C=16, 1,024 pieces), and
    // before the copies take their registers.
    constexpr int U = 4;
    const float* sums = p.carry + p.B * p.nseg * p.C * p.N;
    const int before = on ? w.seg : 0;
    for (int j = 0; j < before; j += U) {
      States<S> s[U];
      float2 d[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t row = (w.b * p.nseg + min(j + u, before - 1)) * p.C + c;
        s[u] = ld_states<S>(p.carry + row * p.N + S * g, p.N, true, order);
        d[u] = make_float2(sums[row + swap], sums[row + 1 - swap]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (j + u < before) scan_fold<S>(h, d[u], A2, s[u]);
    }
  }

  ScanCopies<E, Geo, kActs> copies;
  {
    const void* const act[kActs] = {p.x, p.dt, MODE != kScanCarry ? p.z : nullptr};
    const void* const bc[2] = {p.Bm, MODE != kScanCarry ? p.Cm : nullptr};
    copies.init(sm.raw[0], act, bc, first + tbeg, p.C, w.c0, channels, GN, w.g * p.N, (int)p.N);
  }
  auto load = [&](int i) {
    copies.issue((i & 1) * (uint32_t)sizeof(sm.raw[0]), (int)min(tend - tbeg - (int64_t)i * kScanTile, (int64_t)kScanTile));
    copies.step(kScanTile * p.C, kScanTile * GN);
  };
  // the thread's channel pair in the conversion
  const int lp = tid % Geo::HB;
  const float2 bias = p.dt_bias && 2 * lp < channels ? ld_pair(p.dt_bias + w.c0 + 2 * lp) : splat2(0.f);
  auto convert = [&](int i) {
    const ScanRaw<E, Geo, kActs>& r = sm.raw[i & 1];
    const int left = (int)min(tend - tbeg - (int64_t)i * kScanTile, (int64_t)kScanTile);
    r.template put_bc<1>(0, &sm.B[0][0]);
    if constexpr (MODE != kScanCarry) r.template put_bc<1>(1, &sm.C[0][0]);
#pragma unroll
    for (int j = 0; j < Geo::PT; ++j) {
      const int t = tid / Geo::HB + j * Geo::ROWS;
      // a token past the end: d = 0 leaves the state as it is
      const float2 d = t < left ? scan_step_size2(ld_pair(&r.act[kActDt][t][2 * lp]), bias, p.softplus) : splat2(0.f);
      const float2 dx = mul2(d, ld_pair(&r.act[kActX][t][2 * lp]));
      sm.dd[t][0][lp] = make_float4(d.x, d.y, dx.x, dx.y);
      sm.dd[t][1][lp] = make_float4(d.y, d.x, dx.y, dx.x);
    }
  };

  float2 sum_d = splat2(0.f);
  const int out0 = pair_sum_first<LPC>(g);

  load(0);
  copy_async_wait();
  __syncthreads();
  for (int i = 0; i < nt; ++i) {
    const int64_t t0 = tbeg + (int64_t)i * kScanTile;
    if (i + 1 < nt) load(i + 1);
    convert(i);
    __syncthreads();
    if (MODE == kScanMain && p.ckpt && on) {
      const int64_t m = t0 / kScanTile, nck = (p.T + kScanTile - 1) / kScanTile;
      st_states_wide<S>(p.ckpt + ((w.b * nck + m) * p.C + c) * p.N + S * g, p.N, h, swap);
    }
    float2 tile_d = splat2(0.f);
    const ScanRaw<E, Geo, kActs>& raw = sm.raw[i & 1];
    float done[kScanTile / 4][kPairSums<LPC>];  // stored after the walk: a store would hold back the loads behind it
#pragma unroll
    for (int tg = 0; tg < kScanTile; tg += 4) {
      float2 dots[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 dd = sm.dd[tg + j][swap][pair];
        const float2 d = make_float2(dd.x, dd.y);
        scan_absorb(h, scan_decay(d, A2), scan_taken<PAD>(dd.z, dd.w, S * g < p.N), ld_row<S>(&sm.B[tg + j][S * g]));
        if constexpr (MODE != kScanCarry)
          dots[j] = scan_dot<S>(h, ld_row<S>(&sm.C[tg + j][S * g]));
        else
          tile_d = add2(tile_d, d);
      }
      if constexpr (MODE != kScanCarry) {
        float out[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) out[j] = pair_give(dots[j]);
        pair_sums<LPC>(out, done[tg / 4], tid);
      }
    }
    if (MODE != kScanCarry && p.y) {
      // done[tg / 4][v]: channel `swap` of token tg + out0 + v
      const int left = ch_on && g < 8 ? (int)min(tend - t0, (int64_t)kScanTile) : 0;
      E* y = static_cast<E*>(p.y) + (first + t0) * p.C + c + swap;
#pragma unroll
      for (int tg = 0; tg < kScanTile; tg += 4) {
#pragma unroll
        for (int v = 0; v < kPairSums<LPC>; ++v) {
          const int t = tg + out0 + v;
          const float x = Elem<E>::to_f32(raw.act[kActX][t][2 * pair + swap]), s = done[tg / 4][v];
          float o = p.D ? __fmaf_rn(D, x, s) : s;  // (0 times an infinite x would be NaN)
          if (p.z) {
            const float z = Elem<E>::to_f32(raw.act[kActZ][t][2 * pair + swap]);
            o = __fmul_rn(o, __fmul_rn(z, sigmoid_f(z)));
          }
          if (t < left) y[t * (int)p.C] = Elem<E>::from_f32(o);
        }
      }
    }
    sum_d = add2(sum_d, tile_d);
    copy_async_wait();
    __syncthreads();
  }
  if constexpr (MODE == kScanCarry) {
    const int64_t row = (w.b * p.nseg + w.seg) * p.C + c;
    if (on) st_states_wide<S>(p.carry + row * p.N + S * g, p.N, h, swap);
    if (on && g == 0) st_pair(p.carry + p.B * p.nseg * p.C * p.N + row, sum_d);
  } else if (p.final_state && on && (MODE == kScanSlots || w.seg == p.nseg - 1)) {
    st_states_wide<S>(p.final_state + w.b * p.final_step + c * p.N + S * g, p.N, h, swap);
  }
}

// One token per slot: a stream of the states, 16 bytes per lane and channel.
// The lanes of a channel pair each work the token's step size out for
// themselves; a thread takes the same states of kDecodeSlots slots, so that
// the loads of both are in flight together and A is read once.
constexpr int kDecodeThreads = 128;
constexpr int kDecodeSlots = 2;  // 1: 31, 2: 27, 4: 28 us for 256 slots, C=4096 N=16 bf16
template <class E, int LPC, int S, bool PAD>
__global__ void __launch_bounds__(kDecodeThreads) scan_decode_kernel(const ScanParams p) {
  constexpr int U = kDecodeSlots;
  const int64_t i = (int64_t)blockIdx.x * kDecodeThreads + threadIdx.x;
  const int64_t np = p.C / 2, all = (p.B + U - 1) / U * np * LPC;
  const int g = (int)(i % LPC);
  const int64_t k0 = min(i, all - 1) / LPC, s0 = k0 / np * U, c = k0 % np * 2;
  const bool state_on = i < all && S * g < p.N;
  const int64_t grp = c / p.Cg;
  States<S> h[U];
  float2 x[U], dt[U], z[U];
  Pack<E, S> pb[U], pc[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t s = min(s0 + u, p.B - 1);
    const bool on = state_on && s0 + u < p.B;
    h[u] = ld_states_wide<S>(p.final_state + (s * p.C + c) * p.N + S * g, p.N, on);
    x[u] = ld_pair(static_cast<const E*>(p.x) + s * p.C + c);
    dt[u] = ld_pair(static_cast<const E*>(p.dt) + s * p.C + c);
    z[u] = p.z ? ld_pair(static_cast<const E*>(p.z) + s * p.C + c) : splat2(0.f);
    pb[u].zero();
    pc[u].zero();
    if (on) {
      pb[u].load(static_cast<const E*>(p.Bm) + (s * p.G + grp) * p.N + S * g);
      pc[u].load(static_cast<const E*>(p.Cm) + (s * p.G + grp) * p.N + S * g);
    }
  }
  const States<S> A2 = scan_rates<S>(ld_states_wide<S>(p.A + c * p.N + S * g, p.N, state_on));
  const float2 bias = p.dt_bias ? ld_pair(p.dt_bias + c) : splat2(0.f);
  const float2 D = p.D ? ld_pair(p.D + c) : splat2(0.f);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const bool there = i < all && s0 + u < p.B;
    Row<S> Bv, Cv;
    pb[u].get(Bv.n);
    pc[u].get(Cv.n);
    const float2 d = scan_step_size2(dt[u], bias, p.softplus);
    const float2 dx = mul2(d, x[u]);
    scan_absorb(h[u], scan_decay(d, A2), scan_taken<PAD>(dx.x, dx.y, state_on), Bv);
    if (state_on && there) st_states_wide<S>(p.final_state + ((s0 + u) * p.C + c) * p.N + S * g, p.N, h[u], 0);
    const float2 dot = scan_dot<S>(h[u], Cv);
    float out[2] = {dot.x, dot.y};
    // one lane bit at a time, as the walk's halving steps do
#pragma unroll
    for (int m = 1; m < LPC; m *= 2) {
      out[0] = __fadd_rn(out[0], __shfl_xor_sync(0xffffffffu, out[0], m));
      out[1] = __fadd_rn(out[1], __shfl_xor_sync(0xffffffffu, out[1], m));
    }
    if (there && g == 0) {
      const float2 sums = make_float2(out[0], out[1]), skip = p.D ? fma2(D, x[u], sums) : sums;
      const float2 gate = p.z ? mul2(z[u], sigmoid2(z[u])) : splat2(1.f);
      st_pair(static_cast<E*>(p.y) + (s0 + u) * p.C + c, mul2(skip, gate));
    }
  }
}

wkv_status launched(const char* what, const char** why) {
  if (cudaGetLastError() == cudaSuccess) return WKV_OK;
  *why = what;
  return WKV_ERR_CUDA;
}

template <class E, int LPC, int S, int MODE>
wkv_status run_walk(const ScanParams& p, cudaStream_t st, const char** why) {
  using Geo = ScanGeom<E, LPC, S>;
  constexpr size_t smem = sizeof(ScanFwdShared<E, Geo>);
  static_assert(smem <= 227 * 1024, "the tiles fit an SM");
  // the carry adds nothing up over lanes and keeps no state of a lane without any
  constexpr bool CAN_PAD = MODE != kScanCarry;
  const auto kernel = p.N < Geo::NP ? scan_fwd_kernel<E, LPC, S, CAN_PAD, MODE> : scan_fwd_kernel<E, LPC, S, false, MODE>;
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) {
    *why = "scan kernel: shared memory request failed";
    return WKV_ERR_CUDA;
  }
  const int64_t grid = p.rows * p.G * p.nbg;
  kernel<<<(unsigned)grid, Geo::THREADS, smem, st>>>(p);
  return launched("scan kernel launch failed", why);
}

template <class E, int LPC, int S>
wkv_status run_forward(const ScanArgs& a, cudaStream_t st, const char** why) {
  const ScanCut cut = scan_fwd_cut(a.B, a.T, a.C, a.N, a.G);
  ScanParams p = scan_params(a, cut);
  if (cut.nseg == 1) return run_walk<E, LPC, S, kScanMain>(p, st, why);
  if (wkv_status s = run_walk<E, LPC, S, kScanCarry>(p, st, why)) return s;
  if (!a.final_state || a.final_state != a.init_state) return run_walk<E, LPC, S, kScanMain>(p, st, why);
  // In place: every piece reads the initial state, so the last one leaves the
  // final state in its own (otherwise unused) slot among the pieces, and it
  // is copied out once all have run.
  p.final_state = p.carry + (cut.nseg - 1) * a.C * a.N;
  p.final_step = cut.nseg * a.C * a.N;
  if (wkv_status s = run_walk<E, LPC, S, kScanMain>(p, st, why)) return s;
  const size_t row = (size_t)a.C * a.N * sizeof(float);
  if (cudaMemcpy2DAsync(a.final_state, row, p.final_state, cut.nseg * row, row, (size_t)a.B, cudaMemcpyDeviceToDevice, st) !=
      cudaSuccess) {
    *why = "copy of the final state failed";
    return WKV_ERR_CUDA;
  }
  return WKV_OK;
}
template <class E, int LPC, int S>
wkv_status run_slots(const ScanArgs& a, cudaStream_t st, unsigned* err, const char** why) {
  ScanParams p = scan_params(a, ScanCut{a.B, 1, 0});
  p.err = err;
  return run_walk<E, LPC, S, kScanSlots>(p, st, why);
}
template <class E, int LPC, int S>
wkv_status run_decode(const ScanArgs& a, cudaStream_t st, const char** why) {
  const ScanParams p = scan_params(a, ScanCut{a.B, 1, 0});
  constexpr int DL = LPC * S / 4;  // a stream of states: 16 bytes per lane and channel
  const int64_t threads = ceil_div(a.B, kDecodeSlots) * (a.C / 2) * DL;
  const auto kernel = a.N < LPC * S ? scan_decode_kernel<E, DL, 4, true> : scan_decode_kernel<E, DL, 4, false>;
  kernel<<<(unsigned)ceil_div(threads, kDecodeThreads), kDecodeThreads, 0, st>>>(p);
  return launched("scan decode kernel launch failed", why);
}

// Lanes and states per lane by state size. Two states per lane up to 16: with
// four (half the lanes) a launch has half the warps, and what it saves in
// lane exchanges it loses in waiting: 411 against 380 us at B=8 T=2048 C=2560
// N=16, the same where there are channels enough.
#define WKV_SCAN_DISPATCH(CALL)                                                   \
  const bool bf = a.dtype == WKV_BF16;                                            \
  switch (scan_padded_states(a.N)) {                                              \
    case 8: return bf ? CALL(__nv_bfloat16, 4, 2) : CALL(float, 4, 2);            \
    case 16: return bf ? CALL(__nv_bfloat16, 8, 2) : CALL(float, 8, 2);           \
    case 32: return bf ? CALL(__nv_bfloat16, 8, 4) : CALL(float, 8, 4);           \
    default: return bf ? CALL(__nv_bfloat16, 16, 4) : CALL(float, 16, 4);         \
  }

}  // namespace

// Cut with fewer than three CTAs for two SMs, about where the two cross. Cut and
// uncut, us, by CTAs (bf16, N=8 f32):
//         N=8 T=2048   N=16 T=512   N=16 T=2048   N=16 T=8192   N=32 T=2048   N=64 T=2048
//   128    150 / 205     35 / 41     110 / 154     399 / 605     175 / 205     169 / 191
//   192    210 / 239     49 / 49     156 / 182     584 / 708     251 / 263     243 / 253
//   224    244 / 239     56 / 49     179 / 182     680 / 708     292 / 262     283 / 254
//   256    271 / 239     60 / 49     193 / 183     731 / 710     316 / 263     304 / 253
ScanCut scan_fwd_cut(int64_t B, int64_t T, int64_t C, int64_t N, int64_t G) {
  return scan_cut_few(B, G * scan_group_blocks(C, N, G), T, 148 * 3 / 2);
}

wkv_status launch_scan_forward(const ScanArgs& a, cudaStream_t stream, const char** why) {
#define CALL(E, L, S) (run_forward<E, L, S>(a, stream, why))
  WKV_SCAN_DISPATCH(CALL)
#undef CALL
}
wkv_status launch_scan_chunk_step(const ScanArgs& a, cudaStream_t stream, unsigned* err, const char** why) {
#define CALL(E, L, S) (run_slots<E, L, S>(a, stream, err, why))
  WKV_SCAN_DISPATCH(CALL)
#undef CALL
}
wkv_status launch_scan_decode_step(const ScanArgs& a, cudaStream_t stream, const char** why) {
#define CALL(E, L, S) (run_decode<E, L, S>(a, stream, why))
  WKV_SCAN_DISPATCH(CALL)
#undef CALL
}

}  // namespace wkv
