// Device helpers of the state space, convolution and norm kernels: pairs of
// fp32 values for the packed instructions, eight-element vectors of either
// element type, softplus and SiLU.
#pragma once
#include <float.h>

#include "common.cuh"

namespace linattn {

// Dynamic shared memory above 48 KB has to be asked for.
template <typename K>
inline cudaError_t allow_smem(K *kernel, int bytes) {
  if (bytes <= 48 * 1024) return cudaSuccess;
  return cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                              cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

// Two fp32 values in one 64-bit register pair.  One packed instruction does
// two fp32 operations in one issue slot; each half rounds as the scalar
// instruction does.
struct f2 {
  unsigned long long v;
};
__device__ __forceinline__ f2 pack2(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(f2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ f2 dup2(float x) { return pack2(x, x); }
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ float sum2(f2 a) {
  const float2 x = unpack2(a);
  return x.x + x.y;
}
// 2^x on the special function unit (relative error about 2^-22)
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ f2 ex2_2(f2 a) {
  const float2 x = unpack2(a);
  return pack2(ex2(x.x), ex2(x.y));
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// A decay rate that is no lower than the lowest finite value: a step of zero
// (of a row behind the end, for one) keeps the state, and zero times infinity
// would not.  NaN stays NaN.
__device__ __forceinline__ float finite_rate(float a) { return a < -FLT_MAX ? -FLT_MAX : a; }

// softplus(x) = max(x, 0) + log1p(exp(-|x|)).  log1p(t)/t on [0, 1] is the
// degree-7 Chebyshev interpolant (relative error 3.2e-7 in fp32 arithmetic,
// evaluated on a grid of 200 001 points): the logarithm's own instruction is
// only accurate absolutely, and steps of 1e-3 need it relatively.  NaN stays
// NaN (through the exponential).
__device__ __forceinline__ f2 softplus_f2(f2 x) {
  const float2 q = unpack2(x);
  const f2 t = pack2(ex2(-fabsf(q.x) * kLog2e), ex2(-fabsf(q.y) * kLog2e));
  f2 p = dup2(-0.00837115291506052f);
  p = fma2(p, t, dup2(0.04349390044808388f));
  p = fma2(p, t, dup2(-0.1068500280380249f));
  p = fma2(p, t, dup2(0.1768747717142105f));
  p = fma2(p, t, dup2(-0.24474774301052094f));
  p = fma2(p, t, dup2(0.3327192962169647f));
  p = fma2(p, t, dup2(-0.49997174739837646f));
  p = fma2(p, t, dup2(0.9999997615814209f));
  return fma2(p, t, pack2(fmaxf(q.x, 0.f), fmaxf(q.y, 0.f)));
}
__device__ __forceinline__ float softplus_f32(float x) { return unpack2(softplus_f2(dup2(x))).x; }

// 1 / (1 + exp(-x)) on the special function unit (two roundings each of the
// exponential and the reciprocal); exp(-x) = inf gives 0, NaN stays NaN
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float sigmoid_f32(float x) { return rcp_approx(1.f + ex2(-x * kLog2e)); }
__device__ __forceinline__ f2 sigmoid_f2(f2 x) {
  const float2 q = unpack2(mul2(x, dup2(-kLog2e)));
  const float2 s = unpack2(add2(pack2(ex2(q.x), ex2(q.y)), dup2(1.f)));
  return pack2(rcp_approx(s.x), rcp_approx(s.y));
}

// Asynchronous copy of 16 bytes to shared memory (zeros where !valid: the
// source is then not read).
__device__ __forceinline__ void copy16_async(void *smem, const void *gmem, bool valid) {
  const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
  const int bytes = valid ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(gmem), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copy8_async(void *smem, const void *gmem, bool valid) {
  const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
  const int bytes = valid ? 8 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(gmem), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

__device__ __forceinline__ void bf16x2_to_f32(uint32_t u, float &lo, float &hi) {
  lo = __uint_as_float(u << 16);
  hi = __uint_as_float(u & 0xffff0000u);
}
__device__ __forceinline__ f2 bf16x2_to_f2(uint32_t u) {
  float lo, hi;
  bf16x2_to_f32(u, lo, hi);
  return pack2(lo, hi);
}
__device__ __forceinline__ uint32_t f32_to_bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}
// Eight consecutive elements, rounded once; `p` is 16-byte aligned.
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&x)[8]) {
  *reinterpret_cast<uint4 *>(p) =
      make_uint4(f32_to_bf16x2(x[0], x[1]), f32_to_bf16x2(x[2], x[3]), f32_to_bf16x2(x[4], x[5]),
                 f32_to_bf16x2(x[6], x[7]));
}

// Eight consecutive elements as four pairs; `p` is 16-byte aligned.
__device__ __forceinline__ void load8p(const float *p, f2 (&x)[4]) {
  const ulonglong2 a = *reinterpret_cast<const ulonglong2 *>(p);
  const ulonglong2 b = *reinterpret_cast<const ulonglong2 *>(p + 4);
  x[0] = {a.x};
  x[1] = {a.y};
  x[2] = {b.x};
  x[3] = {b.y};
}
__device__ __forceinline__ void load8p(const __nv_bfloat16 *p, f2 (&x)[4]) {
  const uint4 a = *reinterpret_cast<const uint4 *>(p);
  x[0] = bf16x2_to_f2(a.x);
  x[1] = bf16x2_to_f2(a.y);
  x[2] = bf16x2_to_f2(a.z);
  x[3] = bf16x2_to_f2(a.w);
}
__device__ __forceinline__ void store8p(float *p, const f2 (&x)[4]) {
  *reinterpret_cast<ulonglong2 *>(p) = make_ulonglong2(x[0].v, x[1].v);
  *reinterpret_cast<ulonglong2 *>(p + 4) = make_ulonglong2(x[2].v, x[3].v);
}
__device__ __forceinline__ void store8p(__nv_bfloat16 *p, const f2 (&x)[4]) {
  const float2 a = unpack2(x[0]), b = unpack2(x[1]), c = unpack2(x[2]), d = unpack2(x[3]);
  *reinterpret_cast<uint4 *>(p) = make_uint4(f32_to_bf16x2(a.x, a.y), f32_to_bf16x2(b.x, b.y),
                                             f32_to_bf16x2(c.x, c.y), f32_to_bf16x2(d.x, d.y));
}

// Four consecutive elements as fp32 (8- or 16-byte aligned).
__device__ __forceinline__ float4 load4(const float *p) {
  return *reinterpret_cast<const float4 *>(p);
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) {
  const uint2 a = *reinterpret_cast<const uint2 *>(p);
  float4 r;
  bf16x2_to_f32(a.x, r.x, r.y);
  bf16x2_to_f32(a.y, r.z, r.w);
  return r;
}
__device__ __forceinline__ void store4(float *p, const float4 &x) {
  *reinterpret_cast<float4 *>(p) = x;
}
__device__ __forceinline__ void store4(__nv_bfloat16 *p, const float4 &x) {
  *reinterpret_cast<uint2 *>(p) = make_uint2(f32_to_bf16x2(x.x, x.y), f32_to_bf16x2(x.z, x.w));
}

// Four consecutive elements as two pairs.
__device__ __forceinline__ void load4p(const float *p, f2 (&x)[2]) {
  const ulonglong2 a = *reinterpret_cast<const ulonglong2 *>(p);
  x[0] = {a.x};
  x[1] = {a.y};
}
__device__ __forceinline__ void load4p(const __nv_bfloat16 *p, f2 (&x)[2]) {
  const uint2 a = *reinterpret_cast<const uint2 *>(p);
  x[0] = bf16x2_to_f2(a.x);
  x[1] = bf16x2_to_f2(a.y);
}
__device__ __forceinline__ void store4p(float *p, const f2 (&x)[2]) {
  *reinterpret_cast<ulonglong2 *>(p) = make_ulonglong2(x[0].v, x[1].v);
}
__device__ __forceinline__ void store4p(__nv_bfloat16 *p, const f2 (&x)[2]) {
  const float2 a = unpack2(x[0]), b = unpack2(x[1]);
  *reinterpret_cast<uint2 *>(p) = make_uint2(f32_to_bf16x2(a.x, a.y), f32_to_bf16x2(b.x, b.y));
}

// Eight elements as they lie in memory, for loads that are issued well ahead
// of their use (bf16: four registers, fp32: eight).
template <typename T> struct raw8;
template <> struct raw8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
    a = *reinterpret_cast<const uint4 *>(p);
  }
  __device__ __forceinline__ void zero() { a = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void getp(f2 (&x)[4]) const {
    x[0] = bf16x2_to_f2(a.x);
    x[1] = bf16x2_to_f2(a.y);
    x[2] = bf16x2_to_f2(a.z);
    x[3] = bf16x2_to_f2(a.w);
  }
};
template <> struct raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float *p) {
    a = *reinterpret_cast<const float4 *>(p);
    b = *reinterpret_cast<const float4 *>(p + 4);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void getp(f2 (&x)[4]) const {
    x[0] = pack2(a.x, a.y);
    x[1] = pack2(a.z, a.w);
    x[2] = pack2(b.x, b.y);
    x[3] = pack2(b.z, b.w);
  }
};

}  // namespace linattn
