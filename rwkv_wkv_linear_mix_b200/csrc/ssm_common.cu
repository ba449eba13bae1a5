// ssm_common.cu -- the fixed-order row sum that ends the parameter gradients
// of the state-space operators.
#include "ssm_device.cuh"

namespace wkv {

namespace {

// Warp q of RW adds rows q, q + RW, ... in ascending order, then warp 0 adds
// the RW warp sums in order: the result does not depend on timing.
template <int RW>
__global__ void __launch_bounds__(32 * RW) sum_rows_kernel(const float* __restrict__ part, int64_t rows, int64_t cols,
                                                           const SumOutputs outs) {
  float* out = outs.plane[blockIdx.y];
  if (!out) return;
  __shared__ float sw[RW][32];
  const int lane = threadIdx.x % 32, q = threadIdx.x / 32;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  const float* p = part + (int64_t)blockIdx.y * rows * cols;
  float a = 0.f;
  if (c < cols) {
#pragma unroll 8
    for (int64_t r = q; r < rows; r += RW) a = __fadd_rn(a, p[r * cols + c]);
  }
  sw[q][lane] = a;
  __syncthreads();
  if (q == 0 && c < cols) {
    float s = sw[0][lane];
#pragma unroll
    for (int k = 1; k < RW; ++k) s = __fadd_rn(s, sw[k][lane]);
    out[c] = s;
  }
}

}  // namespace

wkv_status launch_sum_rows(const float* part, int planes, int64_t rows, int64_t cols, const SumOutputs& out,
                           cudaStream_t stream, const char** why) {
  bool any = false;
  for (int i = 0; i < planes; ++i) any = any || out.plane[i];
  if (!any) return WKV_OK;
  const dim3 grid((unsigned)ceil_div(cols, 32), (unsigned)planes);
  // A block has 4 warps for few rows; for many, 8 where there are blocks
  // enough for the SMs, else 32, which shortens each warp's chain of loads
  // (296 rows of 5 x 4096 sums: 16 us with 32 warps, 11 with 8).
  if (rows <= 32)
    sum_rows_kernel<4><<<grid, 32 * 4, 0, stream>>>(part, rows, cols, out);
  else if ((int64_t)grid.x * planes >= 148)
    sum_rows_kernel<8><<<grid, 32 * 8, 0, stream>>>(part, rows, cols, out);
  else
    sum_rows_kernel<32><<<grid, 32 * 32, 0, stream>>>(part, rows, cols, out);
  if (cudaGetLastError() != cudaSuccess) {
    *why = "row sum kernel launch failed";
    return WKV_ERR_CUDA;
  }
  return WKV_OK;
}

}  // namespace wkv
