// ssm_common.cu -- the fixed-order row sum that ends the parameter gradients
// of the state-space operators.
#include "ssm_device.cuh"

namespace wkv {

namespace {

// Warp q of RW adds rows q, q + RW, ..., eight at a time as a tree in their type
// and the eights in float64, then warp 0 adds the RW warp sums: in a fixed
// order, whatever the timing. There are as many rows as sequences and more: in
// float32 alone 2^17 like-signed ones lost 4e-5 of their sum, 2^20 lost 4e-4
// (1.5e-8 now).
template <class P, int RW>
__global__ void __launch_bounds__(32 * RW) sum_rows_kernel(const SumRows<P> s) {
  const typename SumRows<P>::Plane p = s.plane[blockIdx.y];
  if ((int64_t)blockIdx.x * 32 >= p.cols) return;
  __shared__ double sw[RW][32];
  const int lane = threadIdx.x % 32, q = threadIdx.x / 32;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  double a = 0.;
  if (c < p.cols) {
    for (int64_t r = q; r < s.rows; r += 8 * RW) {
      P v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = r + k * RW < s.rows ? p.part[(r + k * RW) * p.cols + c] : P(0);
#pragma unroll
      for (int n = 4; n > 0; n /= 2)
#pragma unroll
        for (int k = 0; k < n; ++k) v[k] += v[k + n];
      a += (double)v[0];
    }
  }
  sw[q][lane] = a;
  __syncthreads();
  if (q == 0 && c < p.cols) {
    double t = sw[0][lane];
#pragma unroll
    for (int k = 1; k < RW; ++k) t += sw[k][lane];
    p.out[c] = (float)t;
  }
}

}  // namespace

template <class P>
wkv_status launch_sum_rows(const SumRows<P>& s, cudaStream_t stream, const char** why) {
  int64_t most = 0, blocks = 0;
  for (int i = 0; i < s.planes; ++i) {
    most = std::max(most, s.plane[i].cols);
    blocks += ceil_div(s.plane[i].cols, 32);
  }
  if (s.planes == 0) return WKV_OK;
  const dim3 grid((unsigned)ceil_div(most, 32), (unsigned)s.planes);
  // A block has 4 warps for few rows; for many, 8 where there are blocks
  // enough for the SMs, else 32, which shortens each warp's chain of loads
  // (296 rows of 5 x 4096 sums: 16 us with 32 warps, 11 with 8).
  if (s.rows <= 32)
    sum_rows_kernel<P, 4><<<grid, 32 * 4, 0, stream>>>(s);
  else if (blocks >= 148)
    sum_rows_kernel<P, 8><<<grid, 32 * 8, 0, stream>>>(s);
  else
    sum_rows_kernel<P, 32><<<grid, 32 * 32, 0, stream>>>(s);
  if (cudaGetLastError() != cudaSuccess) {
    *why = "row sum kernel launch failed";
    return WKV_ERR_CUDA;
  }
  return WKV_OK;
}
template wkv_status launch_sum_rows(const SumRows<float>&, cudaStream_t, const char**);
template wkv_status launch_sum_rows(const SumRows<double>&, cudaStream_t, const char**);

}  // namespace wkv
