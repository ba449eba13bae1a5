// ssm_device.cuh -- device-side building blocks of the state-space operators:
// vectors of N elements as stored, the logistic and softplus functions, and
// sums over lanes that leave each lane its share of the results.
#pragma once

#include "ssm_internal.h"
#include "wkv_device.cuh"

namespace wkv {

// N consecutive elements of E as loaded (packed); N * sizeof(E) is 4, 8, 16 or 32 bytes.
template <class E, int N>
struct Pack {
  static constexpr int kBytes = N * (int)sizeof(E);
  static constexpr int kWords = kBytes / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const E* p) {
    if constexpr (kBytes >= 16) {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const uint4 q = reinterpret_cast<const uint4*>(p)[i];
        w[4 * i] = q.x;
        w[4 * i + 1] = q.y;
        w[4 * i + 2] = q.z;
        w[4 * i + 3] = q.w;
      }
    } else if constexpr (kBytes == 8) {
      const uint2 q = *reinterpret_cast<const uint2*>(p);
      w[0] = q.x;
      w[1] = q.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
  }
  __device__ __forceinline__ void store(E* p) const {
    if constexpr (kBytes >= 16) {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i)
        reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else if constexpr (kBytes == 8) {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
      *reinterpret_cast<uint32_t*>(p) = w[0];
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ void get(float (&f)[N]) const {
    if constexpr (sizeof(E) == 2) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        f[2 * i] = bf16lo(w[i]);
        f[2 * i + 1] = bf16hi(w[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = __uint_as_float(w[i]);
    }
  }
  __device__ __forceinline__ void set(const float (&f)[N]) {
    if constexpr (sizeof(E) == 2) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = __float_as_uint(f[i]);
    }
  }
};

// The same as packed pairs.
template <class E, int N>
__device__ __forceinline__ void get2(const Pack<E, N>& p, float2 (&f)[N / 2]) {
  float v[N];
  p.get(v);
#pragma unroll
  for (int i = 0; i < N / 2; ++i) f[i] = make_float2(v[2 * i], v[2 * i + 1]);
}
template <class E, int N>
__device__ __forceinline__ Pack<E, N> set2(const float2 (&f)[N / 2]) {
  float v[N];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) v[2 * i] = f[i].x, v[2 * i + 1] = f[i].y;
  Pack<E, N> p;
  p.set(v);
  return p;
}

// N float32 parameters, or a constant where there are none.
template <int N>
__device__ __forceinline__ void ld_param(const float* p, float (&f)[N], float otherwise) {
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = otherwise;
  if (p) {
    Pack<float, N> q;
    q.load(p);
    q.get(f);
  }
}

template <int N>
__device__ __forceinline__ void ld_param2(const float* p, float2 (&f)[N / 2], float otherwise) {
  float v[N];
  ld_param<N>(p, v, otherwise);
#pragma unroll
  for (int i = 0; i < N / 2; ++i) f[i] = make_float2(v[2 * i], v[2 * i + 1]);
}

// sigmoid(x) = 1 / (1 + e^-x). e^-x overflows to inf below -88, whose
// reciprocal is the right 0.
__device__ __forceinline__ float sigmoid_f(float x) { return rcp(__fadd_rn(1.f, ex2(__fmul_rn(x, -kLog2e)))); }

// softplus(x) = log(1 + e^x) = max(x, 0) + log1p(e), e = e^-|x| <= 1, of a
// pair. log1p(e) = 2 atanh(s), s = e / (2 + e) <= 1/3, by the series of atanh
// (the first term left out is below 1.5e-8 of the sum): it keeps its relative
// precision where e is small, which log(1 + e) loses.
__device__ __forceinline__ float2 softplus2(float2 x) {
  const float2 e = make_float2(ex2(__fmul_rn(fabsf(x.x), -kLog2e)), ex2(__fmul_rn(fabsf(x.y), -kLog2e)));
  const float2 s = mul2(e, rcp2(add2(e, splat2(2.f))));
  const float2 q = mul2(s, s);
  float2 p = fma2(splat2(1.f / 13.f), q, splat2(1.f / 11.f));
  p = fma2(p, q, splat2(1.f / 9.f));
  p = fma2(p, q, splat2(1.f / 7.f));
  p = fma2(p, q, splat2(1.f / 5.f));
  p = fma2(p, q, splat2(1.f / 3.f));
  p = fma2(p, q, splat2(1.f));
  return fma2(add2(s, s), p, make_float2(fmaxf(x.x, 0.f), fmaxf(x.y, 0.f)));
}

// One copy of 8 or 16 bytes to shared memory that the thread does not wait
// for; zeros where there is nothing to copy (src is then not read). dst: a
// shared-memory address.
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool there) {
  static_assert(BYTES == 8 || BYTES == 16, "copy sizes");
  const int n = there ? BYTES : 0;
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Wait until at most LEFT of the thread's groups of copies are in flight.
template <int LEFT = 0>
__device__ __forceinline__ void copy_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

// Sums of NV values over the NL lanes that differ in the lane bits
// BIT .. BIT * NL / 2, in halving steps: each step sends half of the values
// away and adds the other lane's half, so that NL lanes end with NV / NL sums
// each (or, with NV < NL, with copies of one). Lane bit b of the NL chooses
// the upper half in step b, i.e. the first result of a lane is value
// reduce_scatter_first<NV, NL>(lane / BIT % NL). The partner lanes, and so
// the rounding, are the same for every NV.
template <int NV, int NL, int BIT = 1>
__device__ __forceinline__ void reduce_scatter(float (&v)[NV], int lane) {
  if constexpr (NL > 1) {
    if constexpr (NV > 1) {
      const bool up = lane & BIT;
      float r[NV / 2];
#pragma unroll
      for (int i = 0; i < NV / 2; ++i) {
        const float send = up ? v[i] : v[i + NV / 2];
        const float keep = up ? v[i + NV / 2] : v[i];
        r[i] = __fadd_rn(keep, __shfl_xor_sync(0xffffffffu, send, BIT));
      }
      reduce_scatter<NV / 2, NL / 2, BIT * 2>(r, lane);
#pragma unroll
      for (int i = 0; i < NV / 2; ++i) v[i] = r[i];
    } else {
      v[0] = __fadd_rn(v[0], __shfl_xor_sync(0xffffffffu, v[0], BIT));
      reduce_scatter<1, NL / 2, BIT * 2>(v, lane);
    }
  }
}
template <int NV, int NL>
__device__ __forceinline__ int reduce_scatter_first(int l) {
  int first = 0, half = NV / 2;
#pragma unroll
  for (int b = 1; b < NL; b *= 2) {
    if (half >= 1 && (l & b)) first += half;
    half /= 2;
  }
  return first;
}

}  // namespace wkv
