// Sums of fp32 records over the record index, in a fixed order (the second
// stage of the parameter gradients).
#include "kernels.h"

namespace linattn {
namespace {

__device__ __forceinline__ void put(float *out0, int64_t C0, float *out1, int64_t c, float s) {
  if (c < C0) {
    if (out0) out0[c] = s;
  } else if (out1) {
    out1[c - C0] = s;
  }
}

// Few columns: 32 per CTA; slice y adds records y, y + 32, ..., then the
// slices are added in their order.
constexpr int kCols = 32, kSlices = 32;
__global__ void __launch_bounds__(kCols * kSlices)
    column_sum_kernel(const float *__restrict__ rec, int n, int64_t C, float *__restrict__ out0,
                      int64_t C0, float *__restrict__ out1) {
  __shared__ float sh[kSlices][kCols];
  const int tx = threadIdx.x % kCols, ty = threadIdx.x / kCols;
  const int64_t c = (int64_t)blockIdx.x * kCols + tx;
  float s = 0.f;
  if (c < C) {
#pragma unroll 8
    for (int r = ty; r < n; r += kSlices) s += rec[r * C + c];
  }
  sh[ty][tx] = s;
  __syncthreads();
  if (ty == 0 && c < C) {
    for (int j = 1; j < kSlices; ++j) s += sh[j][tx];
    put(out0, C0, out1, c, s);
  }
}

// Many columns (a multiple of 4): 128 per CTA as 16-byte vectors, 8 slices.
constexpr int kWideVecs = 32, kWideSlices = 8;
__global__ void __launch_bounds__(kWideVecs * kWideSlices)
    column_sum_wide_kernel(const float *__restrict__ rec, int n, int64_t C,
                           float *__restrict__ out0, int64_t C0, float *__restrict__ out1) {
  __shared__ float4 sh[kWideSlices][kWideVecs];
  const int tx = threadIdx.x % kWideVecs, ty = threadIdx.x / kWideVecs;
  const int64_t c = ((int64_t)blockIdx.x * kWideVecs + tx) * 4;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < C) {
#pragma unroll 8
    for (int r = ty; r < n; r += kWideSlices) {
      const float4 v = *reinterpret_cast<const float4 *>(rec + r * C + c);
      s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
  }
  sh[ty][tx] = s;
  __syncthreads();
  if (ty == 0 && c < C) {
    for (int j = 1; j < kWideSlices; ++j) {
      const float4 v = sh[j][tx];
      s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
    put(out0, C0, out1, c, s.x);
    put(out0, C0, out1, c + 1, s.y);
    put(out0, C0, out1, c + 2, s.z);
    put(out0, C0, out1, c + 3, s.w);
  }
}

}  // namespace

cudaError_t launch_column_sum(const float *rec, int n, int64_t C, float *out0, int64_t C0,
                              float *out1, cudaStream_t s) {
  if (C >= 16384 && C % 4 == 0) {
    const unsigned g = (unsigned)((C + 4 * kWideVecs - 1) / (4 * kWideVecs));
    column_sum_wide_kernel<<<g, kWideVecs * kWideSlices, 0, s>>>(rec, n, C, out0, C0, out1);
  } else {
    column_sum_kernel<<<(unsigned)((C + kCols - 1) / kCols), kCols * kSlices, 0, s>>>(rec, n, C, out0,
                                                                                      C0, out1);
  }
  return cudaGetLastError();
}

}  // namespace linattn
