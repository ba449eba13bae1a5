// ssm_scan.cuh -- what the kernels of the selective scan share: the launch
// geometry, where a CTA works, and the loads of a tile of tokens.
//
// A thread carries 4 states of each of 2 adjacent channels; LPC = 2, 4, 8 or
// 16 lanes side by side share the pair, so that 4 LPC >= N. The states above
// N are zero and stay zero (their B is zero). A CTA covers CB channels of one
// group, so that B and C are one row of numbers per token for all of them,
// and walks its tokens in tiles of 16.
#pragma once

#include "ssm_device.cuh"

namespace wkv {

constexpr int kScanTile = WKV_SCAN_CKPT_LEN;  // tokens per tile

template <class E, int LPC>
struct ScanGeom {
  static constexpr int NP = 4 * LPC;                        // padded states
  static constexpr int CB = LPC <= 4 ? 64 : 256 / LPC;      // channels per CTA
  static constexpr int THREADS = CB / 2 * LPC;
  static constexpr int VN = 16 / (int)sizeof(E);            // channels per 16-byte load
  static constexpr int VPR = CB / VN;                       // such loads per token
  static constexpr int PT = (kScanTile * VPR + THREADS - 1) / THREADS;  // per thread and tile
  static constexpr int PB = (kScanTile * LPC + THREADS - 1) / THREADS;  // 4-state loads of B or C
  static_assert(THREADS % VPR == 0, "a thread's loads keep their channels");
};

struct ScanParams {
  int64_t B, T, C, N, G, Cg;  // Cg = C / G
  int nbg, nseg;              // CTAs per group; pieces along T
  int64_t seg_tokens;
  int softplus;
  const void *x, *dt, *Bm, *Cm, *z;
  const float *A, *D, *dt_bias, *init_state;
  void* y;
  float *final_state, *ckpt, *carry;
  const int32_t* cu;
  int64_t n_tokens;
  unsigned* err;
  // backward
  const void* gy;
  const float* g_final;
  void *gx, *gdt, *gz;
  float *g_init, *part_bc, *part_a, *part_d;
};

// Where a CTA works: sequence b, piece seg, group g, channels c0 .. cend-1
// (at most CB of them), block blk of the group.
struct ScanPlace {
  int64_t b, c0, cend;
  int g, blk, seg;
};
template <int CB>
__device__ __forceinline__ ScanPlace scan_place(const ScanParams& p) {
  ScanPlace w;
  const unsigned ncb = (unsigned)(p.G * p.nbg);
  const unsigned cb = blockIdx.x % ncb, rest = blockIdx.x / ncb;
  w.seg = (int)(rest % (unsigned)p.nseg);
  w.b = rest / (unsigned)p.nseg;
  w.g = (int)(cb / (unsigned)p.nbg);
  w.blk = (int)(cb % (unsigned)p.nbg);
  w.c0 = w.g * p.Cg + (int64_t)w.blk * CB;
  w.cend = min((w.g + 1) * p.Cg, w.c0 + CB);
  return w;
}

// The loads of one tile of an activation [tokens][C]: vector i of a thread is
// channels c0 + (tid % VPR) * VN .. of token (tid + i THREADS) / VPR.
template <class E, int LPC>
struct ScanRows {
  using Geo = ScanGeom<E, LPC>;
  Pack<E, Geo::VN> v[Geo::PT];
  // base: token 0 of the sequence; tokens t0 .. tend-1 exist
  __device__ __forceinline__ void load(const E* base, int64_t t0, int64_t tend, int64_t C, int64_t c0, int64_t cend) {
    const int col = (int)threadIdx.x % Geo::VPR * Geo::VN;
#pragma unroll
    for (int i = 0; i < Geo::PT; ++i) {
      const int t = ((int)threadIdx.x + i * Geo::THREADS) / Geo::VPR;
      v[i].zero();
      if (t < kScanTile && t0 + t < tend && c0 + col < cend) v[i].load(base + (t0 + t) * C + c0 + col);
    }
  }
};

// The loads of one tile of B or C, [tokens][G N], and their way into a
// [16][NP] float32 table in shared memory.
template <class E, int LPC>
struct ScanVecs {
  using Geo = ScanGeom<E, LPC>;
  Pack<E, 4> v[Geo::PB];
  __device__ __forceinline__ void load(const E* base, int64_t t0, int64_t tend, int64_t GN, int64_t gN, int64_t N) {
#pragma unroll
    for (int i = 0; i < Geo::PB; ++i) {
      const int k = (int)threadIdx.x + i * Geo::THREADS;
      const int t = k / LPC, n = k % LPC * 4;
      v[i].zero();
      if (t < kScanTile && t0 + t < tend && n < N) v[i].load(base + (t0 + t) * GN + gN + n);
    }
  }
  __device__ __forceinline__ void put(float* table) const {
#pragma unroll
    for (int i = 0; i < Geo::PB; ++i) {
      const int k = (int)threadIdx.x + i * Geo::THREADS;
      if (k / LPC < kScanTile) {
        float f[4];
        v[i].get(f);
        *reinterpret_cast<float4*>(table + k * 4) = make_float4(f[0], f[1], f[2], f[3]);
      }
    }
  }
};

// Four states as two packed pairs.
struct State4 {
  float2 q[2];
};
__device__ __forceinline__ State4 ld_state(const float* p, bool there) {
  State4 s = {{splat2(0.f), splat2(0.f)}};
  if (there) {
    const float4 f = *reinterpret_cast<const float4*>(p);
    s.q[0] = make_float2(f.x, f.y);
    s.q[1] = make_float2(f.z, f.w);
  }
  return s;
}
__device__ __forceinline__ void st_state(float* p, const State4& s) {
  *reinterpret_cast<float4*>(p) = make_float4(s.q[0].x, s.q[0].y, s.q[1].x, s.q[1].y);
}
__device__ __forceinline__ State4 lds_state(const float* p) {
  const float4 f = *reinterpret_cast<const float4*>(p);
  return {{make_float2(f.x, f.y), make_float2(f.z, f.w)}};
}

// d_t of a token from what is stored.
__device__ __forceinline__ float scan_step_size(float dt, float bias, bool softplus) {
  const float raw = __fadd_rn(dt, bias);
  return softplus ? softplus_f(raw) : raw;
}
// The decays of 4 states over step size d (A2 = A log2 e).
__device__ __forceinline__ State4 scan_decay(float d, const State4& A2) {
  return {{ex2_2(mul2(splat2(d), A2.q[0])), ex2_2(mul2(splat2(d), A2.q[1]))}};
}
// h <- a h + dx B, and the lane's part of sum_n C h.
__device__ __forceinline__ void scan_absorb(State4& h, const State4& a, float dx, const State4& Bv) {
  h.q[0] = fma2(a.q[0], h.q[0], mul2(splat2(dx), Bv.q[0]));
  h.q[1] = fma2(a.q[1], h.q[1], mul2(splat2(dx), Bv.q[1]));
}
__device__ __forceinline__ float scan_dot(const State4& a, const State4& b) {
  const float2 s = fma2(a.q[1], b.q[1], mul2(a.q[0], b.q[0]));
  return __fadd_rn(s.x, s.y);
}
__device__ __forceinline__ State4 scale4(const State4& s, float f) {
  return {{mul2(s.q[0], splat2(f)), mul2(s.q[1], splat2(f))}};
}

// Host: the parameters a launch has in common.
inline ScanParams scan_params(const ScanArgs& a, const ScanCut& cut) {
  ScanParams p{};
  p.B = a.B, p.T = a.T, p.C = a.C, p.N = a.N, p.G = a.G, p.Cg = a.C / a.G;
  p.nbg = (int)scan_group_blocks(a.C, a.N, a.G);
  p.nseg = cut.nseg;
  p.seg_tokens = (int64_t)cut.seg_tiles * kScanTile;
  p.softplus = a.softplus;
  p.x = a.x, p.dt = a.dt, p.Bm = a.Bm, p.Cm = a.Cm, p.z = a.z;
  p.A = a.A, p.D = a.D, p.dt_bias = a.dt_bias, p.init_state = a.init_state;
  p.y = a.y, p.final_state = a.final_state, p.ckpt = a.ckpt, p.carry = a.carry;
  p.cu = a.cu, p.n_tokens = a.n_tokens;
  return p;
}

}  // namespace wkv
