// ssm_scan_bwd.cu -- backward of the selective scan. With gs = gy silu(z),
// a_t = e^{d_t A} and Q_t = dL/dh_t, walked from the last token down,
//
//     Q_t = gs_t C_t + a_{t+1} Q_{t+1}
//     gx = d sum_n Q B + gs D        gd = x sum_n Q B + sum_n A Q (a h_{t-1})
//     gA += d Q (a h_{t-1})          gB_t = sum_c Q d x,  gC_t = sum_c gs h_t
//     gz = gy s silu'(z)             gdt = gd softplus'(dt + bias)
//
// The states are recomputed from the forward's checkpoints, one per tile of
// 16 tokens: a tile is walked in sub-blocks, whose decays a and decayed
// states a h_{t-1} stay in registers between the recompute (which also gives
// gC and s) and the reverse walk. a h is kept rather than formed
// as h - d x B, which would cancel where the decay is strong. Sums over the
// states of a channel and over the channels of a group are taken in halving
// steps across lanes; a CTA's gB and gC leave as one partial row per token,
// the parameter gradients as one partial row per piece (in float64, added to
// every 256 tokens), and small kernels add the partial rows in a fixed order.
//
// Cut launches: the carry kernel walks every piece but the first down from
// zero, keeping what enters the piece below (a Q at its first token) and
// its sum of d; the main kernel folds the pieces after its own.
#include "ssm_scan.cuh"

namespace wkv {

namespace {

enum { kActX, kActDt, kActGy, kActZ, kActs };

// Tokens whose decays and decayed states are in registers at a time, and the
// interval of the states that a tile's first walk leaves in shared memory.
constexpr int kBwdSub = 4;
// Tiles whose parameter gradients are added up in float32 (256 tokens) before
// they are added to the piece's row, in float64: one chain over a sequence of
// 65,536 like-signed tokens lost 6e-4 of gA (7e-8 now).
constexpr int kBwdClose = 16;

template <class E, class Geo>
struct ScanBwdShared {
  static constexpr int WARPS = Geo::THREADS / 32;
  ScanRaw<E, Geo, kActs> raw;                    // the tile that is next
  // per channel pair: d0, d1, d0 x0, d1 x1, and gs0, gs1; and with the channels
  // swapped (64 bytes further on in the banks, so that a warp reads both
  // orders at once)
  float4 dd[kScanTile][2][Geo::HB + 4];
  float2 gs[kScanTile][2][Geo::HB + 10];
  // per channel, to finish with: d, x, softplus'(raw), gy silu'(z); channel 1
  // 64 bytes further on, the next token 16, since a lane group reads both
  // channels of 4 tokens at once
  static constexpr int FIN1 = Geo::HB + 4, FIN = 2 * FIN1 + 1;
  float4 fin[kScanTile][FIN];
  float B[kScanTile][Geo::S][Geo::NP];           // in each order of a lane's states
  float C[kScanTile][Geo::S][Geo::NP];
  float sum[2][WARPS][kScanTile][Geo::NP];       // gB, gC of each warp's channels
  // the states before token 0, SUB, 2 SUB, ... of the tile but the last, per thread and channel
  float h[kScanTile / kBwdSub - 1][2][Geo::THREADS][Geo::S];
};

// Sums over the lanes that hold the same states of other channel pairs (lane
// bits LPC and up), for the S states of two tokens. The lane's state order
// (perm) makes the first steps select-free; the step after them exchanges
// tokens, further ones leave copies. GV results per lane: result v is state
// S g + (v % GS) ^ perm of token `tok` (of both, v / GS, where every step was
// one over states).
template <int LPC, int S>
struct ChannelSums {
  static constexpr int RL = 32 / LPC;                          // lanes to add up
  static constexpr int PS = RL < S ? RL : S;                   // of these, by the order of states
  static constexpr int GS = S / PS;                            // states left then
  static constexpr bool TOK = RL > PS;                         // whether a step exchanges the tokens
  static constexpr int GV = TOK ? GS : 2 * GS;
  __device__ static __forceinline__ int perm(int lane) {
    // bit b above the lane group halves the states S/2, S/4, .. apart
    int m = 0;
#pragma unroll
    for (int b = 0; (1 << b) < PS; ++b)
      if (lane & (LPC << b)) m |= S >> (b + 1);
    return m;
  }
  // v[t][j]: token t, register j
  __device__ static __forceinline__ void sum(float (&v)[2][S], float (&out)[GV], int lane) {
#pragma unroll
    for (int b = 0; (1 << b) < PS; ++b) {
      const int half = S >> (b + 1);
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int j = 0; j < half; ++j)
          v[t][j] = __fadd_rn(v[t][j], __shfl_xor_sync(0xffffffffu, v[t][j + half], LPC << b));
    }
    if constexpr (TOK) {
      static_assert(GS == 1, "tokens are exchanged once one state is left");
      float r[2] = {v[0][0], v[1][0]};
      reduce_scatter<2, RL / PS, LPC * PS>(r, lane);
      out[0] = r[0];
    } else {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int j = 0; j < GS; ++j) out[t * GS + j] = v[t][j];
    }
  }
  __device__ static __forceinline__ int token(int v, int lane) { return TOK ? (lane / (LPC * PS)) & 1 : v / GS; }
};

// CTAs of the backward that an SM holds, by states per thread.
constexpr int scan_bwd_resident(int S) { return S == 2 ? 4 : 2; }

template <class E, int LPC, int S, bool PAD, bool Z>
__global__ void __launch_bounds__(ScanGeom<E, LPC, S>::THREADS, scan_bwd_resident(S)) scan_bwd_kernel(const ScanParams p) {
  using Geo = ScanGeom<E, LPC, S>;
  using Shared = ScanBwdShared<E, Geo>;
  constexpr int NP = Geo::NP, WARPS = Shared::WARPS, SUB = kBwdSub;
  using Sums = ChannelSums<LPC, S>;
  extern __shared__ float4 smem4[];
  Shared& sm = *reinterpret_cast<Shared*>(smem4);
  const ScanPlace w = scan_place<Geo::CB, true>(p);
  const int tid = threadIdx.x;
  const int64_t T = p.T, first = w.b * T;
  const int64_t tbeg = w.seg * p.seg_tokens;
  const int64_t tend = w.seg == w.last ? T : tbeg + p.seg_tokens;
  const int nt = (int)((tend - tbeg + kScanTile - 1) / kScanTile);
  const int64_t GN = p.G * p.N, gN = w.g * p.N;
  const int channels = (int)(w.cend - w.c0);
  auto start = [&](int i) { return tbeg + (int64_t)i * kScanTile; };
  auto tokens = [&](int i) { return (int)min(tend - start(i), (int64_t)kScanTile); };

  ScanCopies<E, Geo, kActs> copies;
  {
    const void* const act[kActs] = {p.x, p.dt, p.gy, Z ? p.z : nullptr};
    const void* const bc[2] = {p.Bm, p.Cm};
    copies.init(sm.raw, act, bc, first + start(nt - 1), p.C, w.c0, channels, GN, gN, (int)p.N);
  }
  auto load = [&](int i) {  // from the last tile down
    copies.issue(0, tokens(i));
    copies.step(-kScanTile * p.C, -kScanTile * GN);
  };
  const int lp = tid % Geo::HB;
  const float2 bias = p.dt_bias && 2 * lp < channels ? ld_pair(p.dt_bias + w.c0 + 2 * lp) : splat2(0.f);
  auto convert = [&](int i) {
    const ScanRaw<E, Geo, kActs>& r = sm.raw;
    const int left = tokens(i);
    r.template put_bc<S>(0, &sm.B[0][0][0]);
    r.template put_bc<S>(1, &sm.C[0][0][0]);
#pragma unroll
    for (int j = 0; j < Geo::PT; ++j) {
      const int t = tid / Geo::HB + j * Geo::ROWS;
      const float2 raw = add2(ld_pair(&r.act[kActDt][t][2 * lp]), bias), x = ld_pair(&r.act[kActX][t][2 * lp]);
      // a token past the end: d, x, gs and softplus' are 0, which passes Q on
      // and leaves every sum alone
      const bool real = t < left;
      const float2 d = !real ? splat2(0.f) : p.softplus ? softplus2(raw) : raw;
      const float2 sp = !real ? splat2(0.f) : p.softplus ? sigmoid2(raw) : splat2(1.f);
      const float2 gy = ld_pair(&r.act[kActGy][t][2 * lp]);
      float2 gs = gy, gz = splat2(0.f);
      if constexpr (Z) {
        const float2 z = ld_pair(&r.act[kActZ][t][2 * lp]), s = sigmoid2(z);
        gs = mul2(gy, mul2(z, s));
        gz = mul2(gy, mul2(s, fma2(z, sub2(splat2(1.f), s), splat2(1.f))));
      }
      const float2 dx = mul2(d, x);
      sm.dd[t][0][lp] = make_float4(d.x, d.y, dx.x, dx.y);
      sm.dd[t][1][lp] = make_float4(d.y, d.x, dx.y, dx.x);
      sm.gs[t][0][lp] = gs;
      sm.gs[t][1][lp] = make_float2(gs.y, gs.x);
      sm.fin[t][lp] = make_float4(d.x, x.x, sp.x, gz.x);
      sm.fin[t][Shared::FIN1 + lp] = make_float4(d.y, x.y, sp.y, gz.y);
    }
  };

  const int pair = tid / LPC, g = tid % LPC, warp = tid / 32, lane = tid % 32;
  const LaneOrder order{g & 1, Sums::perm(lane)};
  const bool states = S * g < p.N;
  const int64_t c = w.c0 + 2 * pair;
  const bool ch_on = 2 * pair < channels, on = ch_on && S * g < p.N;
  const int64_t nck = (T + kScanTile - 1) / kScanTile;
  const int64_t state_at = (w.b * p.C + c) * p.N + S * g;
  const States<S> A2 = scan_rates<S>(ld_states<S>(p.A + c * p.N + S * g, p.N, on, order));
  States<S> gA = ld_states<S>(nullptr, 0, false, order);
  States<S> q = ld_states<S>(p.g_final + state_at, p.N, on && p.g_final, order);  // a_{t+1} Q_{t+1}
  const float D = p.D && ch_on ? p.D[c + order.swap] : 0.f;
  {
    const float* sums = p.carry + (p.B - p.whole) * p.nseg * p.C * p.N;
    if (on) {
#pragma unroll 8
      for (int j = w.last; j > w.seg; --j) {
        const int64_t row = ((w.b - p.whole) * p.nseg + j) * p.C + c;
        const States<S> s = ld_states<S>(p.carry + row * p.N + S * g, p.N, true, order);
        scan_fold<S>(q, make_float2(sums[row + order.swap], sums[row + 1 - order.swap]), A2, s);
      }
    }
  }
  float gD = 0.f, gdb = 0.f;  // of the lane's first channel

  auto ld_ckpt = [&](int i) {
    return ld_states<S>(p.ckpt + ((w.b * nck + start(i) / kScanTile) * p.C + c) * p.N + S * g, p.N, on, order);
  };
  auto st_h = [&](int i, const States<S>& h) {
    float a[S], b[S];
#pragma unroll
    for (int j = 0; j < S; ++j) a[j] = h.n[j].x, b[j] = h.n[j].y;
    if constexpr (S == 2) {
      *reinterpret_cast<float2*>(sm.h[i][0][tid]) = make_float2(a[0], a[1]);
      *reinterpret_cast<float2*>(sm.h[i][1][tid]) = make_float2(b[0], b[1]);
    } else {
      *reinterpret_cast<float4*>(sm.h[i][0][tid]) = make_float4(a[0], a[1], a[2], a[3]);
      *reinterpret_cast<float4*>(sm.h[i][1][tid]) = make_float4(b[0], b[1], b[2], b[3]);
    }
  };
  auto put_sums = [&](int i) {
    // the tile's gB, gC of this CTA's channels
    const int left = tokens(i);
    const int64_t t0 = start(i);
    constexpr int VPR = NP / 4;
    for (int k = tid; k < 2 * kScanTile * VPR; k += Geo::THREADS) {
      const int n = k % VPR * 4, t = k / VPR % kScanTile, which = k / (VPR * kScanTile);
      if (t < left && n < p.N) {
        float4 s = *reinterpret_cast<const float4*>(&sm.sum[which][0][t][n]);
#pragma unroll
        for (int v = 1; v < WARPS; ++v) {
          const float4 r = *reinterpret_cast<const float4*>(&sm.sum[which][v][t][n]);
          s = make_float4(__fadd_rn(s.x, r.x), __fadd_rn(s.y, r.y), __fadd_rn(s.z, r.z), __fadd_rn(s.w, r.w));
        }
        const int64_t row = ((int64_t)which * p.nbg + w.blk) * p.B * T + first + t0 + t;
        *reinterpret_cast<float4*>(p.part_bc + row * GN + gN + n) = s;
      }
    }
  };

  // Adds the parameter gradients of up to kBwdClose tiles to the piece's row.
  auto close = [&](bool first) {
    if (on) {
      double* const a = p.part_a + (w.row * p.C + c + order.swap) * p.N + S * g;
      double* const b = p.part_a + (w.row * p.C + c + 1 - order.swap) * p.N + S * g;
#pragma unroll
      for (int j = 0; j < S; ++j) {
        const int n = j ^ order.perm;
        a[n] = (first ? 0. : a[n]) + (double)gA.n[j].x;
        b[n] = (first ? 0. : b[n]) + (double)gA.n[j].y;
        gA.n[j] = splat2(0.f);
      }
    }
    // over the lanes of the channel, each of which finished other tokens
#pragma unroll
    for (int m = 2; m < LPC; m *= 2) {
      gD = __fadd_rn(gD, __shfl_xor_sync(0xffffffffu, gD, m));
      gdb = __fadd_rn(gdb, __shfl_xor_sync(0xffffffffu, gdb, m));
    }
    if (ch_on && g < 2) {
      double* const d = p.part_d + w.row * p.C + c + g;
      d[0] = (first ? 0. : d[0]) + (double)gD;
      d[p.rows * p.C] = (first ? 0. : d[p.rows * p.C]) + (double)gdb;
    }
    gD = gdb = 0.f;
  };

  load(nt - 1);
  States<S> h = ld_ckpt(nt - 1);
  copy_async_wait();
  __syncthreads();
  for (int top = nt; top > 0; top -= kBwdClose) {
    for (int i = top - 1; i >= max(top - kBwdClose, 0); --i) {
      const int64_t t0 = start(i);
      const int left = tokens(i);
      if (i + 1 < nt) put_sums(i + 1);
      convert(i);
      __syncthreads();
      if (i > 0) load(i - 1);
      const int64_t at = (first + t0) * p.C + c + order.swap;
      st_h(0, h);
      // up to the last SUB tokens, leaving the states on the way
#pragma unroll
      for (int t = 0; t < kScanTile - SUB; ++t) {
        const float4 dd = sm.dd[t][order.swap][pair];
        scan_absorb(h, scan_decay(make_float2(dd.x, dd.y), A2), scan_taken<PAD>(dd.z, dd.w, states),
                    ld_row<S>(&sm.B[t][order.perm][S * g]));
        if ((t + 1) % SUB == 0 && t + 1 < kScanTile - SUB) st_h((t + 1) / SUB, h);
      }
#pragma unroll 1
      for (int sub = kScanTile / SUB - 1; sub >= 0; --sub) {
        const int tb = sub * SUB;
        if (sub < kScanTile / SUB - 1) {
          const Row<S> a = ld_row<S>(sm.h[sub][0][tid]), b = ld_row<S>(sm.h[sub][1][tid]);
#pragma unroll
          for (int j = 0; j < S; ++j) h.n[j] = make_float2(a.n[j], b.n[j]);
        }
        // up: the decays and decayed states
        States<S> a[SUB], ah[SUB];
#pragma unroll
        for (int t = 0; t < SUB; ++t) {
          const float4 dd = sm.dd[tb + t][order.swap][pair];
          const Row<S> Bv = ld_row<S>(&sm.B[tb + t][order.perm][S * g]);
          a[t] = scan_decay(make_float2(dd.x, dd.y), A2);
#pragma unroll
          for (int j = 0; j < S; ++j) {
            ah[t].n[j] = mul2(a[t].n[j], h.n[j]);
            h.n[j] = fma2(scan_taken<PAD>(dd.z, dd.w, states), splat2(Bv.n[j]), ah[t].n[j]);
          }
        }
        // down again, the states formed anew from the decayed ones (which is
        // cheaper than to read gs and C on the way up too: the kernel is bound
        // by what it reads of shared memory). Nothing is stored before the end
        // of the sub-block: a store would hold back the loads behind it.
        float gc[SUB / 2][Sums::GV], gb[SUB / 2][Sums::GV];
        float qb[SUB], wa[SUB], s4[SUB];  // sum Q B, sum A2 Q a h, sum C h
#pragma unroll
        for (int t = SUB - 2; t >= 0; t -= 2) {
          float rb[2][S], rc[2][S];
#pragma unroll
          for (int u = 1; u >= 0; --u) {
            const int tt = tb + t + u;
            const float4 dd = sm.dd[tt][order.swap][pair];
            const float2 gss = sm.gs[tt][order.swap][pair], gs = scan_taken<PAD>(gss.x, gss.y, states);
            const Row<S> Bv = ld_row<S>(&sm.B[tt][order.perm][S * g]), Cv = ld_row<S>(&sm.C[tt][order.perm][S * g]);
            const float2 d = make_float2(dd.x, dd.y), dx = scan_taken<PAD>(dd.z, dd.w, states);
            States<S> Q, W, ht;
#pragma unroll
            for (int j = 0; j < S; ++j) {
              ht.n[j] = fma2(dx, splat2(Bv.n[j]), ah[t + u].n[j]);
              Q.n[j] = fma2(gs, splat2(Cv.n[j]), q.n[j]);
              q.n[j] = mul2(a[t + u].n[j], Q.n[j]);
              W.n[j] = mul2(Q.n[j], ah[t + u].n[j]);
              gA.n[j] = fma2(d, W.n[j], gA.n[j]);
              const float2 sb = mul2(dx, Q.n[j]), sc = mul2(gs, ht.n[j]);
              rb[u][j] = __fadd_rn(sb.x, sb.y);
              rc[u][j] = __fadd_rn(sc.x, sc.y);
            }
            qb[t + u] = pair_give(scan_dot<S>(Q, Bv));
            wa[t + u] = pair_give(scan_dot<S>(W, A2));
            if constexpr (Z) s4[t + u] = pair_give(scan_dot<S>(ht, Cv));
          }
          Sums::sum(rb, gb[t / 2], lane);
          Sums::sum(rc, gc[t / 2], lane);
        }
        float out[kPairSums<LPC>], out2[kPairSums<LPC>], sv[kPairSums<LPC>];
        pair_sums<LPC>(qb, out, lane);
        pair_sums<LPC>(wa, out2, lane);
        if constexpr (Z) pair_sums<LPC>(s4, sv, lane);
        // the sub-block's results
#pragma unroll
        for (int t = 0; t < SUB; t += 2)
#pragma unroll
          for (int v = 0; v < Sums::GV; ++v) {
            const int tt = tb + t + Sums::token(v, lane), n = S * g + ((v % Sums::GS) ^ order.perm);
            sm.sum[1][warp][tt][n] = gc[t / 2][v];
            sm.sum[0][warp][tt][n] = gb[t / 2][v];
          }
#pragma unroll
        for (int v = 0; v < kPairSums<LPC>; ++v) {
          const int tt = tb + pair_sum_first<LPC>(g) + v;
          const float4 fin = sm.fin[tt][order.swap * Shared::FIN1 + pair];
          const float d = fin.x, x = fin.y, gs = sm.gs[tt][order.swap][pair].x;
          const float rgx = __fmaf_rn(out[v], d, p.D ? __fmul_rn(gs, D) : 0.f);  // (no product without D: gs may be infinite)
          const float graw = __fmul_rn(__fmaf_rn(out[v], x, __fmul_rn(out2[v], 1.f / kLog2e)), fin.z);
          if (tt < left && ch_on && g < 8) {
            const int64_t to = at + tt * (int)p.C;
            static_cast<E*>(p.gx)[to] = Elem<E>::from_f32(rgx);
            static_cast<E*>(p.gdt)[to] = Elem<E>::from_f32(graw);
            if constexpr (Z)
              static_cast<E*>(p.gz)[to] = Elem<E>::from_f32(__fmul_rn(fin.w, p.D ? __fmaf_rn(D, x, sv[v]) : sv[v]));
            gD = __fmaf_rn(gs, x, gD);
            gdb = __fadd_rn(gdb, graw);
          }
        }
      }
      if (i > 0) h = ld_ckpt(i - 1);
      copy_async_wait();
      __syncthreads();
    }
    close(top == nt);
  }
  put_sums(0);

  if (on && p.g_init && w.seg == 0) st_states<S>(p.g_init + state_at, p.N, q, order);
}

// What a piece, walked down from Q = 0, hands to the piece below, and its sum of d.
template <class E, class Geo>
struct ScanBwdCarryShared {
  ScanRaw<E, Geo, kActs> raw[2];
  float4 dg[2][kScanTile][Geo::HB];  // d0, d1, gs0, gs1
  float C[2][kScanTile][Geo::NP];
};
template <class E, int LPC, int S>
__global__ void __launch_bounds__(ScanGeom<E, LPC, S>::THREADS) scan_bwd_carry_kernel(const ScanParams p) {
  using Geo = ScanGeom<E, LPC, S>;
  extern __shared__ float4 smem4[];
  auto& sm = *reinterpret_cast<ScanBwdCarryShared<E, Geo>*>(smem4);
  const ScanPlace w = scan_place<Geo::CB, true>(p);
  if (w.seg == 0) return;  // nothing lies below the first piece
  const int tid = threadIdx.x;
  const int64_t first = w.b * p.T;
  const int64_t tbeg = w.seg * p.seg_tokens;
  const int64_t tend = w.seg == w.last ? p.T : tbeg + p.seg_tokens;
  const int nt = (int)((tend - tbeg + kScanTile - 1) / kScanTile);
  const int64_t GN = p.G * p.N;
  const int channels = (int)(w.cend - w.c0);
  auto start = [&](int i) { return tbeg + (int64_t)i * kScanTile; };
  auto tokens = [&](int i) { return (int)min(tend - start(i), (int64_t)kScanTile); };
  ScanCopies<E, Geo, kActs> copies;
  {
    const void* const act[kActs] = {nullptr, p.dt, p.gy, p.z};
    const void* const bc[2] = {nullptr, p.Cm};
    copies.init(sm.raw[0], act, bc, first + start(nt - 1), p.C, w.c0, channels, GN, w.g * p.N, (int)p.N);
  }
  auto load = [&](int i) {  // from the last tile down
    copies.issue((i & 1) * (uint32_t)sizeof(sm.raw[0]), tokens(i));
    copies.step(-kScanTile * p.C, -kScanTile * GN);
  };
  const int lp = tid % Geo::HB;
  const float2 bias = p.dt_bias && 2 * lp < channels ? ld_pair(p.dt_bias + w.c0 + 2 * lp) : splat2(0.f);
  auto convert = [&](int i) {
    const ScanRaw<E, Geo, kActs>& r = sm.raw[i & 1];
    const int left = tokens(i);
    r.template put_bc<1>(1, &sm.C[i & 1][0][0]);
#pragma unroll
    for (int j = 0; j < Geo::PT; ++j) {
      const int t = tid / Geo::HB + j * Geo::ROWS;
      const float2 d = t < left ? scan_step_size2(ld_pair(&r.act[kActDt][t][2 * lp]), bias, p.softplus) : splat2(0.f);
      float2 gs = ld_pair(&r.act[kActGy][t][2 * lp]);
      if (p.z) {
        const float2 z = ld_pair(&r.act[kActZ][t][2 * lp]);
        gs = mul2(gs, mul2(z, sigmoid2(z)));
      }
      sm.dg[i & 1][t][lp] = make_float4(d.x, d.y, gs.x, gs.y);
    }
  };
  const int pair = tid / LPC, g = tid % LPC;
  const int64_t c = w.c0 + 2 * pair;
  const bool on = 2 * pair < channels && S * g < p.N;
  const States<S> A2 = scan_rates<S>(ld_states_wide<S>(p.A + c * p.N + S * g, p.N, on));
  States<S> q = ld_states_wide<S>(nullptr, 0, false);
  float2 sum_d = splat2(0.f);
  load(nt - 1);
  if (nt > 1) load(nt - 2);
  copy_async_wait();
  __syncthreads();
  convert(nt - 1);
  __syncthreads();
  for (int i = nt - 1; i >= 0; --i) {
    if (i > 1) load(i - 2);
    if (i > 0) convert(i - 1);
    const int o = i & 1;
    float2 tile_d = splat2(0.f);
#pragma unroll
    for (int t = kScanTile - 1; t >= 0; --t) {
      const float4 dg = sm.dg[o][t][pair];
      const Row<S> Cv = ld_row<S>(&sm.C[o][t][S * g]);
      const float2 d = make_float2(dg.x, dg.y);
      const States<S> a = scan_decay(d, A2);
#pragma unroll
      for (int j = 0; j < S; ++j) q.n[j] = mul2(a.n[j], fma2(make_float2(dg.z, dg.w), splat2(Cv.n[j]), q.n[j]));
      tile_d = add2(tile_d, d);
    }
    sum_d = add2(sum_d, tile_d);
    copy_async_wait();
    __syncthreads();
  }
  const int64_t row = ((w.b - p.whole) * p.nseg + w.seg) * p.C + c;
  if (on) st_states_wide<S>(p.carry + row * p.N + S * g, p.N, q, 0);
  if (on && g == 0) st_pair(p.carry + (p.B - p.whole) * p.nseg * p.C * p.N + row, sum_d);
}

// gB and gC: the sum of the CTAs' partial rows, in order, in the storage type.
template <class E>
__global__ void __launch_bounds__(256) scan_sum_bc_kernel(const float* __restrict__ part, int nbg, int64_t n4, E* __restrict__ gB,
                                                          E* __restrict__ gC) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n4) return;
  const float4* p = reinterpret_cast<const float4*>(part) + (int64_t)blockIdx.y * nbg * n4 + i;
  float4 s = p[0];
#pragma unroll 8
  for (int k = 1; k < nbg; ++k) {
    const float4 r = p[k * n4];
    s = make_float4(__fadd_rn(s.x, r.x), __fadd_rn(s.y, r.y), __fadd_rn(s.z, r.z), __fadd_rn(s.w, r.w));
  }
  Pack<E, 4> o;
  o.set({s.x, s.y, s.z, s.w});
  o.store((blockIdx.y ? gC : gB) + i * 4);
}

wkv_status launched(const char* what, const char** why) {
  if (cudaGetLastError() == cudaSuccess) return WKV_OK;
  *why = what;
  return WKV_ERR_CUDA;
}

// A kernel with more than the static limit of shared memory.
template <class K>
wkv_status run_shared(K kernel, const ScanParams& p, int threads, size_t smem, cudaStream_t st, const char* what,
                      const char** why) {
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) {
    *why = what;
    return WKV_ERR_CUDA;
  }
  kernel<<<(unsigned)(p.rows * p.G * p.nbg), threads, smem, st>>>(p);
  return launched(what, why);
}

template <class E, int LPC, int S>
wkv_status run_backward(const ScanBwdArgs& b, cudaStream_t st, const char** why) {
  const ScanArgs& a = b.f;
  const ScanCut cut = scan_bwd_cut(a.B, a.T, a.C, a.N, a.G);
  ScanParams p = scan_params(a, cut);
  p.gy = b.gy, p.g_final = b.g_final, p.gx = b.gx, p.gdt = b.gdt, p.gz = b.gz, p.g_init = b.g_init;
  p.part_bc = b.part_bc, p.part_a = b.part_a, p.part_d = b.part_d;
  using Geo = ScanGeom<E, LPC, S>;
  constexpr size_t smem = sizeof(ScanBwdShared<E, Geo>);
  static_assert(smem <= 227 * 1024, "the tiles fit an SM");
  if (cut.nseg > 1)
    if (wkv_status s = run_shared(scan_bwd_carry_kernel<E, LPC, S>, p, Geo::THREADS, sizeof(ScanBwdCarryShared<E, Geo>), st,
                                  "scan backward carry kernel launch failed", why))
      return s;
  const bool pad = a.N < Geo::NP;
  const auto kernel = a.z ? pad ? scan_bwd_kernel<E, LPC, S, true, true> : scan_bwd_kernel<E, LPC, S, false, true>
                      : pad ? scan_bwd_kernel<E, LPC, S, true, false>
                            : scan_bwd_kernel<E, LPC, S, false, false>;
  if (wkv_status s = run_shared(kernel, p, Geo::THREADS, smem, st, "scan backward kernel launch failed", why)) return s;
  const int64_t n4 = a.B * a.T * a.G * a.N / 4;
  scan_sum_bc_kernel<E><<<dim3((unsigned)ceil_div(n4, 256), 2), 256, 0, st>>>(b.part_bc, p.nbg, n4, static_cast<E*>(b.gB),
                                                                            static_cast<E*>(b.gC));
  if (wkv_status s = launched("scan gB, gC sum kernel launch failed", why)) return s;
  SumRows<double> sums{};
  sums.rows = cut.rows(a.B);
  sums.add(b.part_a, a.C * a.N, b.gA);
  sums.add(b.part_d, a.C, b.gD);
  sums.add(b.part_d + sums.rows * a.C, a.C, b.gdt_bias);
  return launch_sum_rows(sums, st, why);
}

}  // namespace

// More CTAs than fit at once leave a last wave that idles most SMs. The
// sequences past the last even share of the SMs are cut then, into small
// pieces that fill the gaps, if the share of the time that idles is above
// what their carry pass takes, about a quarter of their walk (T=2048 C=2560,
// 640 CTAs: 1044 -> 900 us at B=8; 960 CTAs: 706 -> 681; where all fit at
// once it does not pay: 384 CTAs, 652 -> 737).
// A launch of few CTAs is cut altogether, up to where the two cross. Cut and
// uncut, us, by CTAs (bf16, N=8 f32):
//          N=8 T=2048   N=16 T=2048   N=32 T=2048   N=64 T=2048
//   192     552 / 649     363 / 498     650 / 778     680 / 820
//   224     640 / 656     428 / 502     757 / 783     790 / 826
//   256     730 / 662     479 / 506     829 / 786     878 / 831
//   288     782 / 668     522 / 511     915 / 792     966 / 838
ScanCut scan_bwd_cut(int64_t B, int64_t T, int64_t C, int64_t N, int64_t G) {
  const int64_t ctas = G * scan_group_blocks(C, N, G), all = B * ctas;
  const int states = scan_padded_states(N);
  if (all > 148 * scan_bwd_resident(states <= 16 ? 2 : 4)) {
    const int64_t whole = all / 148 * 148 / ctas;
    const double idle = 1. - (double)all / (double)(148 * ceil_div(all, 148));
    if (idle > 0.25 * (double)(B - whole) / (double)B) return scan_cut(B, whole, 8, T);
  }
  return scan_cut_few(B, ctas, T, states == 16 ? 148 * 9 / 5 : 148 * 5 / 3);
}

wkv_status launch_scan_backward(const ScanBwdArgs& a, cudaStream_t stream, const char** why) {
  const bool bf = a.f.dtype == WKV_BF16;
  switch (scan_padded_states(a.f.N)) {
    case 8: return bf ? run_backward<__nv_bfloat16, 4, 2>(a, stream, why) : run_backward<float, 4, 2>(a, stream, why);
    case 16: return bf ? run_backward<__nv_bfloat16, 8, 2>(a, stream, why) : run_backward<float, 8, 2>(a, stream, why);
    case 32: return bf ? run_backward<__nv_bfloat16, 8, 4>(a, stream, why) : run_backward<float, 8, 4>(a, stream, why);
    default: return bf ? run_backward<__nv_bfloat16, 16, 4>(a, stream, why) : run_backward<float, 16, 4>(a, stream, why);
  }
}

}  // namespace wkv
