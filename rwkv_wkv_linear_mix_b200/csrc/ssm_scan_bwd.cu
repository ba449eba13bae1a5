// ssm_scan_bwd.cu -- backward of the selective scan. With gs = gy silu(z),
// a_t = e^{d_t A} and Q_t = dL/dh_t, walked from the last token down,
//
//     Q_t = gs_t C_t + a_{t+1} Q_{t+1}
//     gx = d sum_n Q B + gs D        gd = x sum_n Q B + sum_n A Q (a h_{t-1})
//     gA += d Q (a h_{t-1})          gB_t = sum_c Q d x,  gC_t = sum_c gs h_t
//     gz = gy s silu'(z)             gdt = gd softplus'(dt + bias)
//
// The states are recomputed from the forward's checkpoints, one per tile of
// 16 tokens: a tile is walked in two halves of 8 tokens, whose decays a and
// decayed states a h_{t-1} stay in registers between the recompute (which
// also gives gC and s) and the reverse walk. a h is kept rather than formed
// as h - d x B, which would cancel where the decay is strong. Sums over the
// states of a channel and over the channels of a group are taken in halving
// steps across lanes; a CTA's gB and gC leave as one partial row per token,
// the parameter gradients as one partial row per piece, and small kernels
// add the partial rows in a fixed order.
//
// Cut launches: the carry kernel walks every piece but the first down from
// zero, keeping what enters the piece below (a Q at its first token) and
// its sum of d; the main kernel folds the pieces after its own.
#include "ssm_scan.cuh"

namespace wkv {

namespace {

template <int CB, int NP, int WARPS>
struct BwdBuf {
  float4 dd[kScanTile][CB / 2];  // per channel pair: d0, d0 x0, d1, d1 x1
  float4 xg[kScanTile][CB / 2];  // x0, gs0, x1, gs1
  float4 sz[kScanTile][CB / 2];  // softplus'(raw0), gy0 silu'(z0), ... of channel 1
  float B[kScanTile][NP];
  float C[kScanTile][NP];
  float sum[2][WARPS][kScanTile][NP];  // gB, gC of each warp's channels
};

template <class E, int LPC, bool Z>
__global__ void __launch_bounds__(ScanGeom<E, LPC>::THREADS) scan_bwd_kernel(const ScanParams p) {
  using Geo = ScanGeom<E, LPC>;
  constexpr int CB = Geo::CB, NP = Geo::NP, VN = Geo::VN;
  constexpr int WARPS = Geo::THREADS / 32;
  constexpr int HALF = kScanTile / 2;
  constexpr int TG = LPC <= 8 ? 4 : 8;  // tokens whose channel outputs are summed together
  constexpr int RL = 32 / LPC;          // lanes of a warp that share their states' index
  using Buf = BwdBuf<CB, NP, WARPS>;
  extern __shared__ float4 smem4[];
  Buf* buf = reinterpret_cast<Buf*>(smem4);
  const ScanPlace w = scan_place<CB>(p);
  const int tid = threadIdx.x;
  const int64_t T = p.T, first = w.b * T;
  const int64_t tbeg = w.seg * p.seg_tokens;
  const int64_t tend = w.seg == p.nseg - 1 ? T : tbeg + p.seg_tokens;
  const E* xg = static_cast<const E*>(p.x) + first * p.C;
  const E* dtg = static_cast<const E*>(p.dt) + first * p.C;
  const E* gyg = static_cast<const E*>(p.gy) + first * p.C;
  const E* zg = Z ? static_cast<const E*>(p.z) + first * p.C : nullptr;
  E* gxg = static_cast<E*>(p.gx) + first * p.C;
  E* gdtg = static_cast<E*>(p.gdt) + first * p.C;
  E* gzg = Z ? static_cast<E*>(p.gz) + first * p.C : nullptr;
  const int64_t GN = p.G * p.N, gN = w.g * p.N;
  const E* Bg = static_cast<const E*>(p.Bm) + first * GN;
  const E* Cg = static_cast<const E*>(p.Cm) + first * GN;

  const int col = tid % Geo::VPR * VN;
  const bool col_on = w.c0 + col < w.cend;
  float bias[VN];
  ld_param<VN>(p.dt_bias && col_on ? p.dt_bias + w.c0 + col : nullptr, bias, 0.f);

  ScanRows<E, LPC> rx, rdt, rz, rgy;
  ScanVecs<E, LPC> rb, rc;
  auto load = [&](int64_t t0) {
    rx.load(xg, t0, tend, p.C, w.c0, w.cend);
    rdt.load(dtg, t0, tend, p.C, w.c0, w.cend);
    rgy.load(gyg, t0, tend, p.C, w.c0, w.cend);
    if constexpr (Z) rz.load(zg, t0, tend, p.C, w.c0, w.cend);
    rb.load(Bg, t0, tend, GN, gN, p.N);
    rc.load(Cg, t0, tend, GN, gN, p.N);
  };
  auto convert = [&](Buf& o, int64_t t0) {
    rb.put(&o.B[0][0]);
    rc.put(&o.C[0][0]);
#pragma unroll
    for (int i = 0; i < Geo::PT; ++i) {
      const int t = (tid + i * Geo::THREADS) / Geo::VPR;
      if (t < kScanTile) {
        const bool real = t0 + t < tend;
        float x[VN], dt[VN], z[VN], gy[VN];
        rx.v[i].get(x);
        rdt.v[i].get(dt);
        rgy.v[i].get(gy);
        if constexpr (Z) rz.v[i].get(z);
#pragma unroll
        for (int n = 0; n < VN; n += 2) {
          float d[2], gs[2], sp[2], gz[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float raw = __fadd_rn(dt[n + k], bias[n + k]);
            // a token past the end: d, x, gs and sp are 0, which passes Q on
            // and leaves every sum alone
            d[k] = !real ? 0.f : p.softplus ? softplus_f(raw) : raw;
            sp[k] = !real ? 0.f : p.softplus ? sigmoid_f(raw) : 1.f;
            gs[k] = gy[n + k];
            gz[k] = 0.f;
            if constexpr (Z) {
              const float s = sigmoid_f(z[n + k]);
              gs[k] = __fmul_rn(gy[n + k], __fmul_rn(z[n + k], s));
              gz[k] = __fmul_rn(gy[n + k], __fmul_rn(s, __fmaf_rn(z[n + k], __fsub_rn(1.f, s), 1.f)));
            }
          }
          o.dd[t][(col + n) / 2] = make_float4(d[0], __fmul_rn(d[0], x[n]), d[1], __fmul_rn(d[1], x[n + 1]));
          o.xg[t][(col + n) / 2] = make_float4(x[n], gs[0], x[n + 1], gs[1]);
          o.sz[t][(col + n) / 2] = make_float4(sp[0], gz[0], sp[1], gz[1]);
        }
      }
    }
  };

  const int pair = tid / LPC, g = tid % LPC, warp = tid / 32, lane = tid % 32;
  const int64_t c = w.c0 + 2 * pair;
  const bool ch_on = c < w.cend, on = ch_on && 4 * g < p.N;
  const int64_t nck = (T + kScanTile - 1) / kScanTile;
  State4 A2[2], gA[2], q[2];  // q: a_{t+1} Q_{t+1}
  float D[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    A2[k] = scale4(ld_state(p.A + (c + k) * p.N + 4 * g, on), kLog2e);
    gA[k].q[0] = gA[k].q[1] = splat2(0.f);
    q[k] = ld_state(p.g_final + (w.b * p.C + c + k) * p.N + 4 * g, on && p.g_final);
    D[k] = p.D && ch_on ? p.D[c + k] : 0.f;
  }
  {
    const float* sums = p.carry + p.B * p.nseg * p.C * p.N;
    for (int j = p.nseg - 1; j > w.seg; --j) {
      const int64_t row = (w.b * p.nseg + j) * p.C + c;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (on) {
          const State4 s = ld_state(p.carry + (row + k) * p.N + 4 * g, true);
          const State4 a = scan_decay(sums[row + k], A2[k]);
          q[k].q[0] = fma2(a.q[0], q[k].q[0], s.q[0]);
          q[k].q[1] = fma2(a.q[1], q[k].q[1], s.q[1]);
        }
      }
    }
  }
  float gD[2] = {0.f, 0.f}, gdb[2] = {0.f, 0.f};

  const int nt = (int)((tend - tbeg + kScanTile - 1) / kScanTile);
  auto start = [&](int i) { return tbeg + (int64_t)i * kScanTile; };
  auto ld_ckpt = [&](int i, State4 (&h)[2]) {
    const int64_t m = start(i) / kScanTile;
#pragma unroll
    for (int k = 0; k < 2; ++k) h[k] = ld_state(p.ckpt + ((w.b * nck + m) * p.C + c + k) * p.N + 4 * g, on);
  };
  auto put_sums = [&](const Buf& o, int64_t t0) {
    // the tile's gB, gC of this CTA's channels
    constexpr int PER = 2 * kScanTile * LPC;
    for (int i = tid; i < PER; i += Geo::THREADS) {
      const int n = i % LPC * 4, t = i / LPC % kScanTile, which = i / (LPC * kScanTile);
      if (t0 + t < tend && n < p.N) {
        float4 s = *reinterpret_cast<const float4*>(&o.sum[which][0][t][n]);
#pragma unroll
        for (int v = 1; v < WARPS; ++v) {
          const float4 r = *reinterpret_cast<const float4*>(&o.sum[which][v][t][n]);
          s = make_float4(__fadd_rn(s.x, r.x), __fadd_rn(s.y, r.y), __fadd_rn(s.z, r.z), __fadd_rn(s.w, r.w));
        }
        const int64_t row = ((int64_t)which * p.nbg + w.blk) * p.B * T + first + t0 + t;
        *reinterpret_cast<float4*>(p.part_bc + row * GN + gN + n) = s;
      }
    }
  };

  State4 h0[2];
  load(start(nt - 1));
  convert(buf[0], start(nt - 1));
  if (nt > 1) load(start(nt - 2));
  ld_ckpt(nt - 1, h0);
  __syncthreads();
  for (int i = nt - 1, cur = 0; i >= 0; --i, cur ^= 1) {
    const int64_t t0 = start(i);
    if (i + 1 < nt) put_sums(buf[cur ^ 1], start(i + 1));
    if (i > 0) convert(buf[cur ^ 1], start(i - 1));
    if (i > 1) load(start(i - 2));
    Buf& o = buf[cur];
    State4 h[2] = {h0[0], h0[1]};
    if (i > 0) ld_ckpt(i - 1, h0);
    State4 hstart[2] = {h[0], h[1]};
    // up to the second half
#pragma unroll
    for (int t = 0; t < HALF; ++t) {
      const float4 dd = o.dd[t][pair];
      const State4 Bv = lds_state(&o.B[t][4 * g]);
      scan_absorb(h[0], scan_decay(dd.x, A2[0]), dd.y, Bv);
      scan_absorb(h[1], scan_decay(dd.z, A2[1]), dd.w, Bv);
    }
#pragma unroll 1
    for (int half = 1; half >= 0; --half) {
      const int tb = half * HALF;
      if (half == 0) {
        h[0] = hstart[0];
        h[1] = hstart[1];
      }
      State4 a[HALF][2], ah[HALF][2];
      float sv[8];
#pragma unroll
      for (int t = 0; t < HALF; t += 2) {
        float gc[8];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float4 dd = o.dd[tb + t + u][pair], xv = o.xg[tb + t + u][pair];
          const State4 Bv = lds_state(&o.B[tb + t + u][4 * g]);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float d = k ? dd.z : dd.x, dx = k ? dd.w : dd.y;
            a[t + u][k] = scan_decay(d, A2[k]);
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              ah[t + u][k].q[v] = mul2(a[t + u][k].q[v], h[k].q[v]);
              h[k].q[v] = fma2(splat2(dx), Bv.q[v], ah[t + u][k].q[v]);
            }
          }
          // gC: the sum over channels of gs h
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const float2 s = fma2(splat2(xv.w), h[1].q[v], mul2(splat2(xv.y), h[0].q[v]));
            gc[4 * u + 2 * v] = s.x;
            gc[4 * u + 2 * v + 1] = s.y;
          }
          if constexpr (Z) {
            const State4 Cv = lds_state(&o.C[tb + t + u][4 * g]);
            sv[2 * ((t + u) % 4)] = scan_dot(h[0], Cv);
            sv[2 * ((t + u) % 4) + 1] = scan_dot(h[1], Cv);
          }
        }
        reduce_scatter<8, RL, LPC>(gc, lane);
        const int f = reduce_scatter_first<8, RL>(lane / LPC);
#pragma unroll
        for (int v = 0; v < (8 / RL > 0 ? 8 / RL : 1); ++v) o.sum[1][warp][tb + t + (f + v) / 4][4 * g + (f + v) % 4] = gc[v];
        if constexpr (Z) {
          if (t % 4 == 2) {
            // s, and with it gz, of 4 tokens
            reduce_scatter<8, LPC>(sv, lane);
            const int f2 = reduce_scatter_first<8, LPC>(g);
#pragma unroll
            for (int v = 0; v < (8 / LPC > 0 ? 8 / LPC : 1); ++v) {
              const int tt = tb + t - 2 + (f2 + v) / 2, k = (f2 + v) % 2;
              const float4 xv = o.xg[tt][pair], zv = o.sz[tt][pair];
              const float s = __fmaf_rn(k ? D[1] : D[0], k ? xv.z : xv.x, sv[v]);
              if (t0 + tt < tend && ch_on && g < 8)
                gzg[(t0 + tt) * p.C + c + k] = Elem<E>::from_f32(__fmul_rn(k ? zv.w : zv.y, s));
            }
          }
        }
      }
      // down again
#pragma unroll
      for (int t = HALF - TG; t >= 0; t -= TG) {
        float out[4 * TG];  // token, channel, (sum Q B, sum A2 Q a h)
#pragma unroll
        for (int u = TG - 1; u >= 0; --u) {
          const int tt = tb + t + u;
          const float4 dd = o.dd[tt][pair], xv = o.xg[tt][pair];
          const State4 Bv = lds_state(&o.B[tt][4 * g]), Cv = lds_state(&o.C[tt][4 * g]);
          State4 Q[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float d = k ? dd.z : dd.x, gs = k ? xv.w : xv.y;
            State4 W;
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              Q[k].q[v] = fma2(splat2(gs), Cv.q[v], q[k].q[v]);
              q[k].q[v] = mul2(a[t + u][k].q[v], Q[k].q[v]);
              W.q[v] = mul2(Q[k].q[v], ah[t + u][k].q[v]);
              gA[k].q[v] = fma2(splat2(d), W.q[v], gA[k].q[v]);
            }
            out[4 * u + 2 * k] = scan_dot(Q[k], Bv);
            out[4 * u + 2 * k + 1] = scan_dot(W, A2[k]);
          }
          // gB of this token: keep Q's channel sum in place of a (used up)
#pragma unroll
          for (int v = 0; v < 2; ++v)
            a[t + u][0].q[v] = fma2(splat2(dd.w), Q[1].q[v], mul2(splat2(dd.y), Q[0].q[v]));
        }
#pragma unroll
        for (int u = 0; u < TG; u += 2) {
          float gb[8];
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              gb[4 * e + 2 * v] = a[t + u + e][0].q[v].x;
              gb[4 * e + 2 * v + 1] = a[t + u + e][0].q[v].y;
            }
          reduce_scatter<8, RL, LPC>(gb, lane);
          const int f = reduce_scatter_first<8, RL>(lane / LPC);
#pragma unroll
          for (int v = 0; v < (8 / RL > 0 ? 8 / RL : 1); ++v)
            o.sum[0][warp][tb + t + u + (f + v) / 4][4 * g + (f + v) % 4] = gb[v];
        }
        reduce_scatter<4 * TG, LPC>(out, lane);
        const int f = reduce_scatter_first<4 * TG, LPC>(g);
#pragma unroll
        for (int v = 0; v < 4 * TG / LPC; v += 2) {
          const int tt = tb + t + (f + v) / 4, k = (f + v) % 4 / 2;
          const float4 dd = o.dd[tt][pair], xv = o.xg[tt][pair], zv = o.sz[tt][pair];
          const float d = k ? dd.z : dd.x, x = k ? xv.z : xv.x, gs = k ? xv.w : xv.y;
          const float gx = __fmaf_rn(out[v], d, __fmul_rn(gs, k ? D[1] : D[0]));
          const float gd = __fmaf_rn(out[v], x, __fmul_rn(out[v + 1], 1.f / kLog2e));
          const float graw = __fmul_rn(gd, k ? zv.z : zv.x);
          if (t0 + tt < tend && ch_on) {
            gxg[(t0 + tt) * p.C + c + k] = Elem<E>::from_f32(gx);
            gdtg[(t0 + tt) * p.C + c + k] = Elem<E>::from_f32(graw);
          }
          const float gdx = __fmul_rn(gs, x);
          if (k) {
            gD[1] = __fadd_rn(gD[1], gdx);
            gdb[1] = __fadd_rn(gdb[1], graw);
          } else {
            gD[0] = __fadd_rn(gD[0], gdx);
            gdb[0] = __fadd_rn(gdb[0], graw);
          }
        }
      }
    }
    __syncthreads();
  }
  put_sums(buf[(nt - 1) & 1], start(0));

  const int64_t prow = w.b * p.nseg + w.seg;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (on) st_state(p.part_a + (prow * p.C + c + k) * p.N + 4 * g, gA[k]);
    if (on && p.g_init && w.seg == 0) st_state(p.g_init + (w.b * p.C + c + k) * p.N + 4 * g, q[k]);
    // over the lanes of the channel, each of which finished other tokens
#pragma unroll
    for (int m = 1; m < LPC; m *= 2) {
      gD[k] = __fadd_rn(gD[k], __shfl_xor_sync(0xffffffffu, gD[k], m));
      gdb[k] = __fadd_rn(gdb[k], __shfl_xor_sync(0xffffffffu, gdb[k], m));
    }
    if (ch_on && g == 0) {
      p.part_d[prow * p.C + c + k] = gD[k];
      p.part_d[(p.B * p.nseg + prow) * p.C + c + k] = gdb[k];
    }
  }
}

// What a piece, walked down from Q = 0, hands to the piece below, and its sum of d.
template <int CB, int NP>
struct BwdCarryBuf {
  float4 dg[kScanTile][CB / 2];  // d0, gs0, d1, gs1
  float C[kScanTile][NP];
};
template <class E, int LPC>
__global__ void __launch_bounds__(ScanGeom<E, LPC>::THREADS) scan_bwd_carry_kernel(const ScanParams p) {
  using Geo = ScanGeom<E, LPC>;
  constexpr int CB = Geo::CB, VN = Geo::VN;
  __shared__ BwdCarryBuf<CB, Geo::NP> buf[2];
  const ScanPlace w = scan_place<CB>(p);
  if (w.seg == 0) return;  // nothing lies below the first piece
  const int tid = threadIdx.x;
  const int64_t first = w.b * p.T;
  const int64_t tbeg = w.seg * p.seg_tokens;
  const int64_t tend = w.seg == p.nseg - 1 ? p.T : tbeg + p.seg_tokens;
  const E* dtg = static_cast<const E*>(p.dt) + first * p.C;
  const E* gyg = static_cast<const E*>(p.gy) + first * p.C;
  const E* zg = p.z ? static_cast<const E*>(p.z) + first * p.C : nullptr;
  const int64_t GN = p.G * p.N, gN = w.g * p.N;
  const E* Cg = static_cast<const E*>(p.Cm) + first * GN;
  const int col = tid % Geo::VPR * VN;
  const bool col_on = w.c0 + col < w.cend;
  float bias[VN];
  ld_param<VN>(p.dt_bias && col_on ? p.dt_bias + w.c0 + col : nullptr, bias, 0.f);
  ScanRows<E, LPC> rdt, rz, rgy;
  ScanVecs<E, LPC> rc;
  auto load = [&](int64_t t0) {
    rdt.load(dtg, t0, tend, p.C, w.c0, w.cend);
    rgy.load(gyg, t0, tend, p.C, w.c0, w.cend);
    if (zg) rz.load(zg, t0, tend, p.C, w.c0, w.cend);
    rc.load(Cg, t0, tend, GN, gN, p.N);
  };
  auto convert = [&](BwdCarryBuf<CB, Geo::NP>& o, int64_t t0) {
    rc.put(&o.C[0][0]);
#pragma unroll
    for (int i = 0; i < Geo::PT; ++i) {
      const int t = (tid + i * Geo::THREADS) / Geo::VPR;
      if (t < kScanTile) {
        float dt[VN], z[VN], gs[VN];
        rdt.v[i].get(dt);
        rgy.v[i].get(gs);
        if (zg) rz.v[i].get(z);
#pragma unroll
        for (int n = 0; n < VN; ++n) {
          dt[n] = t0 + t < tend ? scan_step_size(dt[n], bias[n], p.softplus) : 0.f;
          if (zg) gs[n] = __fmul_rn(gs[n], __fmul_rn(z[n], sigmoid_f(z[n])));
        }
#pragma unroll
        for (int n = 0; n < VN; n += 2) o.dg[t][(col + n) / 2] = make_float4(dt[n], gs[n], dt[n + 1], gs[n + 1]);
      }
    }
  };
  const int pair = tid / LPC, g = tid % LPC;
  const int64_t c = w.c0 + 2 * pair;
  const bool on = c < w.cend && 4 * g < p.N;
  State4 A2[2], q[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    A2[k] = scale4(ld_state(p.A + (c + k) * p.N + 4 * g, on), kLog2e);
    q[k].q[0] = q[k].q[1] = splat2(0.f);
  }
  float sum_d[2] = {0.f, 0.f};
  const int nt = (int)((tend - tbeg + kScanTile - 1) / kScanTile);
  auto start = [&](int i) { return tbeg + (int64_t)i * kScanTile; };
  load(start(nt - 1));
  convert(buf[0], start(nt - 1));
  if (nt > 1) load(start(nt - 2));
  __syncthreads();
  for (int i = nt - 1, cur = 0; i >= 0; --i, cur ^= 1) {
    if (i > 0) convert(buf[cur ^ 1], start(i - 1));
    if (i > 1) load(start(i - 2));
    const auto& o = buf[cur];
    float tile_d[2] = {0.f, 0.f};
#pragma unroll
    for (int t = kScanTile - 1; t >= 0; --t) {
      const float4 dg = o.dg[t][pair];
      const State4 Cv = lds_state(&o.C[t][4 * g]);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float d = k ? dg.z : dg.x, gs = k ? dg.w : dg.y;
        const State4 a = scan_decay(d, A2[k]);
#pragma unroll
        for (int v = 0; v < 2; ++v) q[k].q[v] = mul2(a.q[v], fma2(splat2(gs), Cv.q[v], q[k].q[v]));
        tile_d[k] = __fadd_rn(tile_d[k], d);
      }
    }
    sum_d[0] = __fadd_rn(sum_d[0], tile_d[0]);
    sum_d[1] = __fadd_rn(sum_d[1], tile_d[1]);
    __syncthreads();
  }
  const int64_t row = (w.b * p.nseg + w.seg) * p.C + c;
  float* sums = p.carry + p.B * p.nseg * p.C * p.N;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (on) st_state(p.carry + (row + k) * p.N + 4 * g, q[k]);
    if (on && g == 0) sums[row + k] = sum_d[k];
  }
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

template <class E, int LPC, bool Z>
wkv_status run_main(const ScanParams& p, cudaStream_t st, const char** why) {
  using Geo = ScanGeom<E, LPC>;
  constexpr size_t smem = 2 * sizeof(BwdBuf<Geo::CB, Geo::NP, Geo::THREADS / 32>);
  static_assert(smem <= 227 * 1024, "the tiles fit an SM");
  if (cudaFuncSetAttribute(scan_bwd_kernel<E, LPC, Z>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
      cudaSuccess) {
    *why = "scan backward kernel: shared memory request failed";
    return WKV_ERR_CUDA;
  }
  const int64_t grid = p.B * p.nseg * p.G * p.nbg;
  scan_bwd_kernel<E, LPC, Z><<<(unsigned)grid, Geo::THREADS, smem, st>>>(p);
  return launched("scan backward kernel launch failed", why);
}

template <class E, int LPC>
wkv_status run_backward(const ScanBwdArgs& b, cudaStream_t st, const char** why) {
  const ScanArgs& a = b.f;
  const ScanCut cut = scan_bwd_cut(a.B, a.T, a.C, a.N, a.G);
  ScanParams p = scan_params(a, cut);
  p.gy = b.gy, p.g_final = b.g_final, p.gx = b.gx, p.gdt = b.gdt, p.gz = b.gz, p.g_init = b.g_init;
  p.part_bc = b.part_bc, p.part_a = b.part_a, p.part_d = b.part_d;
  if (cut.nseg > 1) {
    const int64_t grid = p.B * p.nseg * p.G * p.nbg;
    scan_bwd_carry_kernel<E, LPC><<<(unsigned)grid, ScanGeom<E, LPC>::THREADS, 0, st>>>(p);
    if (wkv_status s = launched("scan backward carry kernel launch failed", why)) return s;
  }
  if (wkv_status s = a.z ? run_main<E, LPC, true>(p, st, why) : run_main<E, LPC, false>(p, st, why)) return s;
  const int64_t n4 = a.B * a.T * a.G * a.N / 4;
  scan_sum_bc_kernel<E><<<dim3((unsigned)ceil_div(n4, 256), 2), 256, 0, st>>>(b.part_bc, p.nbg, n4, static_cast<E*>(b.gB),
                                                                            static_cast<E*>(b.gC));
  if (wkv_status s = launched("scan gB, gC sum kernel launch failed", why)) return s;
  const int64_t rows = a.B * cut.nseg;
  if (wkv_status s = launch_sum_rows(b.part_a, 1, rows, a.C * a.N, b.gA, st, why)) return s;
  if (b.gD)
    if (wkv_status s = launch_sum_rows(b.part_d, 1, rows, a.C, b.gD, st, why)) return s;
  return b.gdt_bias ? launch_sum_rows(b.part_d + rows * a.C, 1, rows, a.C, b.gdt_bias, st, why) : WKV_OK;
}

}  // namespace

wkv_status launch_scan_backward(const ScanBwdArgs& a, cudaStream_t stream, const char** why) {
  const bool bf = a.f.dtype == WKV_BF16;
  switch (scan_lanes(a.f.N)) {
    case 2: return bf ? run_backward<__nv_bfloat16, 2>(a, stream, why) : run_backward<float, 2>(a, stream, why);
    case 4: return bf ? run_backward<__nv_bfloat16, 4>(a, stream, why) : run_backward<float, 4>(a, stream, why);
    case 8: return bf ? run_backward<__nv_bfloat16, 8>(a, stream, why) : run_backward<float, 8>(a, stream, why);
    default: return bf ? run_backward<__nv_bfloat16, 16>(a, stream, why) : run_backward<float, 16>(a, stream, why);
  }
}

}  // namespace wkv
