// Sums of fp32 records over the record index, in a fixed order: the device
// part, for kernels of 256 threads.
#pragma once
#include "common.cuh"

namespace linattn {

__device__ __forceinline__ void put_column(float *out0, int64_t C0, float *out1, int64_t c, float s) {
  if (c < C0) {
    if (out0) out0[c] = s;
  } else if (out1) {
    out1[c - C0] = s;
  }
}

// Columns [128 block, 128 block + 128) of n records of C columns (a multiple
// of 4) as 16-byte vectors, 8 slices of the records; `sh` is the CTA's.
constexpr int kWideVecs = 32, kWideSlices = 8, kWideCols = 4 * kWideVecs;
__device__ __forceinline__ void column_sum_wide(const float *__restrict__ rec, int n, int64_t C,
                                                float *__restrict__ out0, int64_t C0,
                                                float *__restrict__ out1, int64_t block,
                                                float4 (*sh)[kWideVecs]) {
  const int tx = threadIdx.x % kWideVecs, ty = threadIdx.x / kWideVecs;
  const int64_t c = block * kWideCols + tx * 4;
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
    put_column(out0, C0, out1, c, s.x);
    put_column(out0, C0, out1, c + 1, s.y);
    put_column(out0, C0, out1, c + 2, s.z);
    put_column(out0, C0, out1, c + 3, s.w);
  }
}

}  // namespace linattn
