// Retention on CUDA cores in fp32: fp32 inputs, and the widths that the
// tensor-core kernel does not take.
//
// One CTA works a slice of SW columns of w over a part of the tokens, by
// chunks of 64: x and y lie transposed in shared memory (feature-major), so
// that every product reads float4 along the tokens; the state of the slice
// stays in shared memory.  Bound by the fp32 pipe and by shared memory (two
// 16-byte loads for 16 multiply-adds a thread).
#include "common.cuh"
#include "mixer_common.cuh"
#include "retention.cuh"

namespace linattn {
namespace {

constexpr int kC = 64;
constexpr int kLd = kC + 4;  // floats between feature rows
constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ float4 load4(const T *p);
template <>
__device__ __forceinline__ float4 load4<float>(const float *p) {
  return *reinterpret_cast<const float4 *>(p);
}
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16 *p) {
  const uint2 r = *reinterpret_cast<const uint2 *>(p);
  return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u), __uint_as_float(r.y << 16),
                     __uint_as_float(r.y & 0xffff0000u));
}

// Four columns of a row, zero behind the end.
template <typename T>
__device__ __forceinline__ float4 load_if(bool in, const T *p) {
  return in ? load4(p) : make_float4(0.f, 0.f, 0.f, 0.f);
}
// A thread's share of 64 feature columns from d on (4 of each 16), for one token,
// feature-major.
__device__ __forceinline__ void store_turned(float *dst, const float4 *v, int t, int g, int d, int W) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int c = d + 4 * g + 16 * k;
    if (c >= W) break;
    dst[c * kLd + t] = v[k].x;
    dst[(c + 1) * kLd + t] = v[k].y;
    dst[(c + 2) * kLd + t] = v[k].z;
    dst[(c + 3) * kLd + t] = v[k].w;
  }
}

template <int N>
struct Cols {
  float v[N];
};
template <int N>
__device__ __forceinline__ Cols<N> cols(const float *p) {
  Cols<N> r;
  if constexpr (N == 4) {
    const float4 x = *reinterpret_cast<const float4 *>(p);
    r.v[0] = x.x, r.v[1] = x.y, r.v[2] = x.z, r.v[3] = x.w;
  } else {
    const float2 x = *reinterpret_cast<const float2 *>(p);
    r.v[0] = x.x, r.v[1] = x.y;
  }
  return r;
}

struct SimtParams {
  RetArgs a;
  int parts, cpp, slices;  // cpp: chunks of a part; slices: of the widest role
};

// The pass that only sums states has no x and no weights.
int smem_bytes(int Dx, int SW, bool state) {
  return 4 * (Dx * kLd + Dx * SW + kC * SW + 2 * kC + (state ? 0 : Dx * kLd + kC * kLd));
}

// STATE: only the part's own state, into its record.
template <typename T, int SW, bool STATE>
__global__ void __launch_bounds__(kThreads) retention_simt_kernel(const __grid_constant__ SimtParams p) {
  constexpr int CW = SW / 16;
  extern __shared__ float sm[];
  const RetRole &r = p.a.role[blockIdx.z];
  const int np = STATE ? p.parts - 1 : p.parts;
  const int slice = blockIdx.x % p.slices, part = blockIdx.x / p.slices % np;
  const int64_t bh = blockIdx.x / p.slices / np;
  const int e0 = slice * SW;
  if (e0 >= r.Dw) return;
  const int b = static_cast<int>(bh / p.a.H), h = static_cast<int>(bh % p.a.H);
  const int Dx = r.Dx, Dw = r.Dw;
  float *yt = sm, *S = yt + Dx * kLd, *w = S + Dx * SW, *pw = w + kC * SW, *xt = pw + 2 * kC, *pt = xt + Dx * kLd;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int tokens = ret_tokens(p.a.lens, b, p.a.L);
  const int n = (tokens + kC - 1) / kC;
  const float lg = p.a.lg.g[h];
  const T *x = static_cast<const T *>(r.x) + b * r.xs.b + (h / r.xg) * r.xs.h;
  const T *y = static_cast<const T *>(r.y) + b * r.ys.b + (h / r.yg) * r.ys.h;
  const T *wp = static_cast<const T *>(r.w) + b * r.ws.b + (h / r.wg) * r.ws.h + e0;
  const float *rec = r.rec + bh * (p.parts - 1) * Dx * Dw;

  if (tid <= kC) pw[tid] = exp2f(lg * static_cast<float>(tid));
  for (int i = tid; i < Dx * SW; i += kThreads) {
    const int d = i / SW, e = e0 + i % SW;
    S[i] = STATE || e >= Dw ? 0.f : ret_start(r, rec, bh, part, p.cpp, n, tokens, kC, lg, d, e);
  }
  const int c0 = part * p.cpp, c1 = part == p.parts - 1 ? n : min(n, c0 + p.cpp);
  const bool keep = STATE || (part == p.parts - 1 && r.end);  // the state behind the last chunk is wanted
  for (int c = c0; c < c1; ++c) {
    const int t0 = (r.reverse ? n - 1 - c : c) * kC;
    const int nv = min(kC, tokens - t0);
    {
      // the loads of a round under way together: one by one their latency took
      // half of the time
      const int t = tid & (kC - 1), g = tid >> 6;
      constexpr int kRows = kC * SW / 4 / kThreads;
      float4 wv[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int at = tid + i * kThreads, row = at / (SW / 4), e = 4 * (at % (SW / 4));
        wv[i] = load_if(row < nv && e0 + e < Dw, wp + (t0 + row) * r.ws.t + e);
      }
      for (int d = 0; d < Dx; d += 64) {
        float4 xv[4], yv[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int c = d + 4 * g + 16 * k;
          if (!STATE) xv[k] = load_if(t < nv && c < Dx, x + (t0 + t) * r.xs.t + c);
          yv[k] = load_if(t < nv && c < Dx, y + (t0 + t) * r.ys.t + c);
        }
        if (!STATE) store_turned(xt, xv, t, g, d, Dx);
        store_turned(yt, yv, t, g, d, Dx);
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i) reinterpret_cast<float4 *>(w)[tid + i * kThreads] = wv[i];
    }
    __syncthreads();
    if (!STATE) {
      float a[4][4] = {};
#pragma unroll 8
      for (int d = 0; d < Dx; ++d) {
        const Cols<4> u = cols<4>(xt + d * kLd + 4 * ty), v = cols<4>(yt + d * kLd + 4 * tx);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) a[i][j] = fmaf(u.v[i], v.v[j], a[i][j]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float col[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int far = r.reverse ? 4 * tx + j - 4 * ty - i : 4 * ty + i - 4 * tx - j;
          col[i] = far >= 0 ? a[i][j] * pw[far] : 0.f;
        }
        *reinterpret_cast<float4 *>(pt + (4 * tx + j) * kLd + 4 * ty) = make_float4(col[0], col[1], col[2], col[3]);
      }
      __syncthreads();
      float o[4][CW] = {};
#pragma unroll 8
      for (int d = 0; d < Dx; ++d) {
        const Cols<4> u = cols<4>(xt + d * kLd + 4 * ty);
        const Cols<CW> v = cols<CW>(S + d * SW + CW * tx);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < CW; ++j) o[i][j] = fmaf(u.v[i], v.v[j], o[i][j]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 4 * ty + i;
        const float f = t >= nv ? 0.f : pw[r.reverse ? nv - 1 - t : t + 1];
#pragma unroll
        for (int j = 0; j < CW; ++j) o[i][j] *= f;
      }
      // the weights that are not masked, for the two groups of rows of a warp
      const int s0 = r.reverse ? 4 * (ty & ~1) : 0, s1 = r.reverse ? kC : 4 * (ty | 1) + 4;
#pragma unroll 8
      for (int s = s0; s < s1; ++s) {
        const Cols<4> u = cols<4>(pt + s * kLd + 4 * ty);
        const Cols<CW> v = cols<CW>(w + s * SW + CW * tx);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < CW; ++j) o[i][j] = fmaf(u.v[i], v.v[j], o[i][j]);
      }
      if (e0 + CW * tx < Dw) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = 4 * ty + i;
          if (t >= nv) break;
          const int64_t at = b * r.os.b + (t0 + t) * r.os.t + h * r.os.h + e0 + CW * tx;
#pragma unroll
          for (int j = 0; j < CW; ++j) {
            const float v = o[i][j] * r.out_scale;
            if (r.o_f32) static_cast<float *>(r.o)[at + j] = v;
            else io<T>::store(static_cast<T *>(r.o) + at + j, v);
          }
        }
      }
      __syncthreads();
    }
    if (keep || c + 1 < c1) {
      const float gn = pw[nv];
      for (int d = 4 * ty; d < Dx; d += 64) {
        float s[4][CW] = {};
#pragma unroll 2
        for (int j = 0; j < kC; j += 4) {
          Cols<4> u[4];
          Cols<CW> v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            u[i] = cols<4>(yt + (d + i) * kLd + j);
            v[i] = cols<CW>(w + (j + i) * SW + CW * tx);
            const int t = j + i;
            const float f = t >= nv ? 0.f : pw[r.reverse ? t + 1 : nv - 1 - t];
#pragma unroll
            for (int k = 0; k < CW; ++k) v[i].v[k] *= f;
          }
#pragma unroll
          for (int jj = 0; jj < 4; ++jj)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int k = 0; k < CW; ++k) s[i][k] = fmaf(u[i].v[jj], v[jj].v[k], s[i][k]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int k = 0; k < CW; ++k) {
            float *at = S + (d + i) * SW + CW * tx + k;
            *at = fmaf(gn, *at, s[i][k]);
          }
      }
    }
    __syncthreads();
  }
  __syncthreads();
  if (STATE || (part == p.parts - 1 && r.end)) {
    float *out = STATE ? const_cast<float *>(rec) + static_cast<int64_t>(part) * Dx * Dw : r.end + bh * r.state;
    const float f = STATE ? 1.f : r.end_scale;
    for (int i = tid; i < Dx * SW; i += kThreads) {
      const int d = i / SW, e = e0 + i % SW;
      if (e < Dw) out[d * Dw + e] = f * S[i];
    }
  }
  if (!STATE && p.a.fill && part == p.parts - 1) {
    for (int64_t i = tid; i < static_cast<int64_t>(p.a.L - tokens) * SW; i += kThreads) {
      const int e = e0 + static_cast<int>(i % SW);
      if (e >= Dw) continue;
      const int64_t at = b * r.os.b + (tokens + i / SW) * r.os.t + h * r.os.h + e;
      if (r.o_f32) static_cast<float *>(r.o)[at] = 0.f;
      else io<T>::store(static_cast<T *>(r.o) + at, 0.f);
    }
  }
}

template <typename T, int SW>
cudaError_t run(const RetArgs &a, int parts, int widest, int Dx, cudaStream_t s) {
  SimtParams p = {a, parts, 0, (widest + SW - 1) / SW};
  const int chunks = (a.L + kC - 1) / kC;
  p.cpp = (chunks + parts - 1) / parts;
  const int64_t units = static_cast<int64_t>(a.B) * a.H * p.slices;
  if (units * parts >= (1LL << 31)) return cudaErrorNotSupported;
  if (parts > 1) {
    auto k = retention_simt_kernel<T, SW, true>;
    const int bytes = smem_bytes(Dx, SW, true);
    cudaError_t e = allow_smem(k, bytes);
    if (e != cudaSuccess) return e;
    k<<<dim3(static_cast<unsigned>(units * (parts - 1)), 1, a.roles), kThreads, bytes, s>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  auto k = retention_simt_kernel<T, SW, false>;
  const int bytes = smem_bytes(Dx, SW, false);
  const cudaError_t e = allow_smem(k, bytes);
  if (e != cudaSuccess) return e;
  k<<<dim3(static_cast<unsigned>(units * parts), 1, a.roles), kThreads, bytes, s>>>(p);
  return cudaGetLastError();
}

void widths(const RetArgs &a, int *Dx, int *Dw) {
  *Dx = *Dw = 0;
  for (int i = 0; i < a.roles; ++i) {
    if (a.role[i].Dx > *Dx) *Dx = a.role[i].Dx;
    if (a.role[i].Dw > *Dw) *Dw = a.role[i].Dw;
  }
}

// How a call is cut: slices of SW columns and parts of the tokens.
struct Cut {
  int SW, parts;
};

// The cut that is done first by a model of the CTAs that an SM holds (by shared
// memory, up to three): a chunk takes 1 unit of time with slices of 64 columns and
// 0.8 with 32 (14 and 12 us of 64 features, alone on an SM), half of that where
// states are summed, 0.35 more for each further CTA on the SM, and a CTA 1 unit to
// begin and end.  Above 128 features slices of 64 columns do not fit.
Cut cut_of(const RetArgs &a) {
  int Dx, Dw;
  widths(a, &Dx, &Dw);
  const int chunks = (a.L + kC - 1) / kC;
  Cut best = {32, 1};
  double least = 1e300;
  for (int SW = 32; SW <= (Dx > 128 || Dw <= 32 ? 32 : 64); SW += 32) {
    const int64_t units = static_cast<int64_t>(a.B) * a.H * ((Dw + SW - 1) / SW) * a.roles;
    auto time = [&](int64_t n, double chunk, bool state) {
      int held = 227 * 1024 / (smem_bytes(Dx, SW, state) + 1024);
      if (held > 3) held = 3;
      if (n < static_cast<int64_t>(kSMs) * held) held = static_cast<int>((n + kSMs - 1) / kSMs);
      const int64_t slots = static_cast<int64_t>(kSMs) * (held > 0 ? held : 1);
      return static_cast<double>((n + slots - 1) / slots) * (chunk * (1 + 0.35 * (held - 1)) + 1);
    };
    for (int parts = 1; parts <= 32 && (parts == 1 || parts * 2 <= chunks); ++parts) {
      const double chunk = ((chunks + parts - 1) / parts) * (SW == 64 ? 1.0 : 0.8);
      double t = time(units * parts, chunk, false);
      if (parts > 1) t += time(units * (parts - 1), 0.5 * chunk, true);
      if (t < least) least = t, best = {SW, parts};
    }
  }
  return best;
}

template <typename T>
__global__ void __launch_bounds__(256) group_sum_kernel(const __grid_constant__ GroupSumArgs a, int64_t total) {
  for (int64_t i = blockIdx.x * 256LL + threadIdx.x; i < total; i += static_cast<int64_t>(gridDim.x) * 256) {
    // four columns of one output head: its shares lie behind one another
    const int e = static_cast<int>(i % (a.width / 4)) * 4;
    const int64_t rh = i / (a.width / 4);
    const int h = static_cast<int>(rh % a.heads);
    const int64_t row = rh / a.heads;
    const int t = static_cast<int>(row % a.L), b = static_cast<int>(row / a.L);
    if (t >= ret_tokens(a.lens, b, a.L)) continue;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = 0; j < a.g; ++j) {
      const float4 v = __ldcs(reinterpret_cast<const float4 *>(a.part + (rh * a.g + j) * a.width + e));
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    T *o = static_cast<T *>(a.out) + b * a.os.b + t * a.os.t + h * a.os.h + e;
    io<T>::store(o, s.x), io<T>::store(o + 1, s.y), io<T>::store(o + 2, s.z), io<T>::store(o + 3, s.w);
  }
}

}  // namespace

int ret_parts_simt(const RetArgs &a) { return cut_of(a).parts; }

cudaError_t launch_retention_simt(const RetArgs &a, Dtype dt, int parts, cudaStream_t s) {
  int Dx, Dw;
  widths(a, &Dx, &Dw);
  const bool wide = cut_of(a).SW == 64;
  if (dt == kF32) return wide ? run<float, 64>(a, parts, Dw, Dx, s) : run<float, 32>(a, parts, Dw, Dx, s);
  return wide ? run<__nv_bfloat16, 64>(a, parts, Dw, Dx, s) : run<__nv_bfloat16, 32>(a, parts, Dw, Dx, s);
}

cudaError_t launch_group_sum(const GroupSumArgs &a, Dtype dt, cudaStream_t s) {
  const int64_t total = static_cast<int64_t>(a.B) * a.L * a.heads * (a.width / 4);
  const int64_t want = (total + 255) / 256;
  const unsigned grid = static_cast<unsigned>(want < 8 * kSMs ? want : 8 * kSMs);
  if (dt == kF32) group_sum_kernel<float><<<grid, 256, 0, s>>>(a, total);
  else group_sum_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(a, total);
  return cudaGetLastError();
}

// ---- choice between the kernels, shared host code ----

int ret_parts(const RetArgs &a, Dtype dt) { return ret_tc_supported(a, dt) ? ret_parts_tc(a) : ret_parts_simt(a); }

int ret_records(const RetArgs &a, int parts) {
  for (int i = 0; i < a.roles; ++i)
    if (a.role[i].end) return parts;
  return parts - 1;
}

size_t ret_record_floats(const RetArgs &a, int parts) {
  size_t n = 0;
  for (int i = 0; i < a.roles; ++i) n += static_cast<size_t>(a.role[i].Dx) * a.role[i].Dw;
  return n * a.B * a.H * ret_records(a, parts);
}

void ret_layout(RetArgs *a, int parts, float *ws) {
  for (int i = 0; i < a->roles; ++i) {
    a->role[i].rec = ws;
    ws += static_cast<size_t>(a->B) * a->H * ret_records(*a, parts) * a->role[i].Dx * a->role[i].Dw;
  }
}

cudaError_t launch_retention(const RetArgs &a, Dtype dt, int parts, cudaStream_t s) {
  return ret_tc_supported(a, dt) ? launch_retention_tc(a, parts, s) : launch_retention_simt(a, dt, parts, s);
}

}  // namespace linattn
