// Sums of fp32 records over the record index, in a fixed order (the second
// stage of the parameter gradients).
#include "column_sum.cuh"
#include "dependent.cuh"
#include "kernels.h"

namespace linattn {
namespace {

// 32 columns per CTA; slice y adds records y, y + 32, ..., then the slices are
// added in their order.
constexpr int kCols = 32, kSlices = 32;
__global__ void __launch_bounds__(kCols * kSlices)
    column_sum_kernel(const float *__restrict__ rec, int n, int64_t C, float *__restrict__ out0,
                      int64_t C0, float *__restrict__ out1) {
  __shared__ float sh[kSlices][kCols];
  const int tx = threadIdx.x % kCols, ty = threadIdx.x / kCols;
  const int64_t c = (int64_t)blockIdx.x * kCols + tx;
  float s = 0.f;
  wait_for_previous();
  if (c < C) {
#pragma unroll 8
    for (int r = ty; r < n; r += kSlices) s += rec[r * C + c];
  }
  sh[ty][tx] = s;
  __syncthreads();
  if (ty == 0 && c < C) {
    for (int j = 1; j < kSlices; ++j) s += sh[j][tx];
    put_column(out0, C0, out1, c, s);
  }
}

}  // namespace

cudaError_t launch_column_sum(const float *rec, int n, int64_t C, float *out0, int64_t C0,
                              float *out1, cudaStream_t s) {
  return launch_dependent(column_sum_kernel, (unsigned)((C + kCols - 1) / kCols), 1, kCols * kSlices, 0, s,
                          rec, n, C, out0, C0, out1);
}

}  // namespace linattn
