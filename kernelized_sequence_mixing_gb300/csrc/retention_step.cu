// One token of retention, in place on fp32 states:  S <- g S + k v^T,
// o = scale q^T S.
//
// The state is read and written once, 8 D Dv bytes against 5 D Dv operations:
// bound by HBM.  A CTA has a slice of columns of one (sequence, head): LN lanes
// of four columns, 256 / LN groups of rows; a thread has up to kRows rows of its
// columns in flight at once, all loaded before anything else is, and the
// read-out is one sum over the row groups through shared memory.  Wide slices
// (LN = 32, whole 512-byte rows) where they fill the card; slices of 32 columns
// where few sequences decode, so that the states of one sequence spread over
// four times the SMs.
//
// Measured at H = 32, D = Dv = 128, bf16: 256 sequences 159 us (1.08 GB, the copy
// rate); one sequence of 16 heads 2.4 us in a graph (22-25 launched one by one, the
// host's time).
#include "common.cuh"
#include "kernels.h"
#include "mixer_common.cuh"

namespace linattn {
namespace {

constexpr int kThreads = 256;

template <typename T, int LN, int ROWS>
__global__ void __launch_bounds__(kThreads) retention_step_kernel(const __grid_constant__ RetStepArgs a) {
  constexpr int kGroups = kThreads / LN;
  __shared__ float q[256], k[256];
  __shared__ float4 sums[kGroups][LN];
  const int slices = (a.Dv + 4 * LN - 1) / (4 * LN);
  const int slice = blockIdx.x % slices;
  const int64_t bh = blockIdx.x / slices;
  const int b = static_cast<int>(bh / a.H), h = static_cast<int>(bh % a.H), hk = h / (a.H / a.Hk);
  const int64_t slot = a.slots ? a.slots[b] : b;
  if (slot < 0 || slot >= a.pool) return;
  const int tid = threadIdx.x, lane = tid % LN, group = tid / LN;
  const int e = 4 * (slice * LN + lane);
  const bool in = e < a.Dv;
  float *S = a.S + ((slot * a.H + h) * a.D) * a.Dv + e;
  const float g = a.g.g[h];
  float4 s[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int d = group + r * kGroups;
    if (in && d < a.D) s[r] = __ldcs(reinterpret_cast<const float4 *>(S + static_cast<int64_t>(d) * a.Dv));
  }
  if (tid < a.D) {
    q[tid] = io<T>::load(static_cast<const T *>(a.q) + b * a.ldq + h * a.D + tid);
    k[tid] = io<T>::load(static_cast<const T *>(a.k) + b * a.ldk + hk * a.D + tid);
  }
  float v[4] = {};
  if (in)
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = io<T>::load(static_cast<const T *>(a.v) + b * a.ldv + hk * a.Dv + e + i);
  __syncthreads();
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int base = 0; base < a.D; base += ROWS * kGroups) {
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const int d = base + group + r * kGroups;
      if (!in || d >= a.D) continue;
      float4 *at = reinterpret_cast<float4 *>(S + static_cast<int64_t>(d) * a.Dv);
      if (base > 0) s[r] = __ldcs(at);
      const float kd = k[d], qd = q[d];
      s[r].x = fmaf(g, s[r].x, kd * v[0]);
      s[r].y = fmaf(g, s[r].y, kd * v[1]);
      s[r].z = fmaf(g, s[r].z, kd * v[2]);
      s[r].w = fmaf(g, s[r].w, kd * v[3]);
      o.x = fmaf(qd, s[r].x, o.x);
      o.y = fmaf(qd, s[r].y, o.y);
      o.z = fmaf(qd, s[r].z, o.z);
      o.w = fmaf(qd, s[r].w, o.w);
      __stcs(at, s[r]);
    }
  }
  sums[group][lane] = o;
  __syncthreads();
  if (group == 0 && in) {
#pragma unroll 8
    for (int i = 1; i < kGroups; ++i) {
      const float4 x = sums[i][lane];
      o.x += x.x, o.y += x.y, o.z += x.z, o.w += x.w;
    }
    T *to = static_cast<T *>(a.o) + (static_cast<int64_t>(b) * a.H + h) * a.Dv + e;
    io<T>::store(to, o.x * a.scale);
    io<T>::store(to + 1, o.y * a.scale);
    io<T>::store(to + 2, o.z * a.scale);
    io<T>::store(to + 3, o.w * a.scale);
  }
}

template <typename T, int LN, int ROWS>
cudaError_t run(const RetStepArgs &a, cudaStream_t s) {
  const int64_t grid = static_cast<int64_t>(a.B) * a.H * ((a.Dv + 4 * LN - 1) / (4 * LN));
  if (grid >= (1LL << 31)) return cudaErrorNotSupported;
  retention_step_kernel<T, LN, ROWS><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t pick(const RetStepArgs &a, cudaStream_t s) {
  const bool wide = static_cast<int64_t>(a.B) * a.H * ((a.Dv + 127) / 128) >= 2 * kSMs;
  if (wide) return a.D <= 64 ? run<T, 32, 8>(a, s) : run<T, 32, 16>(a, s);
  return a.D <= 64 ? run<T, 8, 2>(a, s) : run<T, 8, 4>(a, s);
}

}  // namespace

cudaError_t launch_retention_step(const RetStepArgs &a, Dtype dt, cudaStream_t s) {
  return dt == kF32 ? pick<float>(a, s) : pick<__nv_bfloat16>(a, s);
}

}  // namespace linattn
