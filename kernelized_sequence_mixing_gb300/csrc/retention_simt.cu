// Retention on CUDA cores in fp32: fp32 inputs, and the widths that the
// tensor-core kernel does not take.  Roles of up to 128 features.
//
// One CTA works a slice of SW columns of w over a part of the tokens, by chunks of
// 64 in the order of the pass (a pass backward in time loads its rows turned
// round, so that every chunk looks forward).  Per chunk and thread:
//
//   weights x y^T and x S in one pass over the features (4 x 4 and 4 x CW of them
//   from the same x), blocks of 16 x 16 behind the diagonal left out; two
//   multiply-adds an instruction (128 features: 7% less time than one);
//   weights times w from shared memory; the decayed y^T w into the state, which
//   stays in registers and goes to shared memory once a chunk for x S.
//
// The next chunk's rows travel meanwhile (fp32 by cp.async, bf16 in registers).
// Bound by shared memory (60% of its wavefronts) and the waits of 8 or 16 warps an
// SM; the fp32 pipe is busy 30 to 45% of the time.  Measured, fp32: B2 L2047 H8 64/128
// with both states 107 us; B2 L7629 H8 D128 512; B8 L2000 H32 D128 1533, D64 468.
#include "common.cuh"
#include "dependent.cuh"
#include "mixer_common.cuh"
#include "retention.cuh"

namespace linattn {
namespace {

constexpr int kC = 64;
constexpr int kLdP = kC + 4;  // floats between rows of weights
constexpr int kThreads = 256;

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
template <int N>
__device__ __forceinline__ void put(float *p, const float *v) {
  if constexpr (N == 4) *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
  else *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]);
}
template <int N>
__device__ __forceinline__ void put(__nv_bfloat16 *p, const float *v) {
#pragma unroll
  for (int i = 0; i < N; i += 2)
    *reinterpret_cast<__nv_bfloat162 *>(p + i) = __floats2bfloat162_rn(v[i], v[i + 1]);
}

// Rows of a chunk on their way to shared memory: 16 bytes a piece, 1 << sh pieces a
// row (of those, the ones below width), rows from nv on zero.  N: pieces of a thread.
template <typename T, int N>
struct Rows;
template <int N>
struct Rows<float, N> {
  __device__ __forceinline__ void begin(const float *from, int64_t stride, int t0, int nv, bool turned, int sh,
                                        int width, float *to, int ld) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int i = threadIdx.x + k * kThreads, row = i >> sh, col = (i & ((1 << sh) - 1)) * 4;
      if (row >= kC) break;
      const bool in = row < nv && col < width;
      const int t = t0 + (in ? (turned ? nv - 1 - row : row) : 0);
      if (col < ld) copy16_async(to + row * ld + col, from + t * stride + (in ? col : 0), in);
    }
  }
  __device__ __forceinline__ void settle(int, float *, int) {}
};
template <int N>
struct Rows<__nv_bfloat16, N> {
  uint4 v[N];
  __device__ __forceinline__ void begin(const __nv_bfloat16 *from, int64_t stride, int t0, int nv, bool turned, int sh,
                                        int width, float *, int) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int i = threadIdx.x + k * kThreads, row = i >> sh, col = (i & ((1 << sh) - 1)) * 8;
      v[k] = make_uint4(0u, 0u, 0u, 0u);
      if (row < nv && col < width)
        v[k] = *reinterpret_cast<const uint4 *>(from + (t0 + (turned ? nv - 1 - row : row)) * stride + col);
    }
  }
  __device__ __forceinline__ void settle(int sh, float *to, int ld) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int i = threadIdx.x + k * kThreads, row = i >> sh, col = (i & ((1 << sh) - 1)) * 8;
      if (row >= kC || col + 8 > ld) continue;
      float *at = to + row * ld + col;
      auto lo = [](uint32_t u) { return __uint_as_float(u << 16); };
      auto hi = [](uint32_t u) { return __uint_as_float(u & 0xffff0000u); };
      *reinterpret_cast<float4 *>(at) = make_float4(lo(v[k].x), hi(v[k].x), lo(v[k].y), hi(v[k].y));
      *reinterpret_cast<float4 *>(at + 4) = make_float4(lo(v[k].z), hi(v[k].z), lo(v[k].w), hi(v[k].w));
    }
  }
};

struct SimtParams {
  RetArgs a;
  int parts, cpp, slices;  // cpp: chunks of a part; slices: of the widest role
  int bufs;                // 2: the next chunk is loaded during this one
};

// The pass that only sums states has no x, no weights and its state in registers.
int smem_bytes(int Dx, int SW, bool state, int bufs) {
  const int rows = kC * (Dx + 4);
  return 4 * (bufs * ((state ? 1 : 2) * rows + kC * SW) + 2 * kC + (state ? 0 : Dx * SW + kC * kLdP));
}

// NI: 64 features each; STATE: only the part's own state, into its record.
template <typename T, int NI, int SW, bool STATE>
__global__ void __launch_bounds__(kThreads, NI == 1 ? 2 : 1)
    retention_simt_kernel(const __grid_constant__ SimtParams p) {
  constexpr int CW = SW / 16, kPer = 16 / sizeof(T);
  constexpr int kShW = SW / kPer == 16 ? 4 : SW / kPer == 8 ? 3 : 2;  // pieces of a row of w, log2
  constexpr int kNX = kC * 64 * NI / kPer / kThreads, kNW = kC * SW / kPer / kThreads;
  extern __shared__ __align__(16) float sm[];
  const RetRole &r = p.a.role[blockIdx.z];
  const int np = STATE ? p.parts - 1 : p.parts;
  const int slice = blockIdx.x % p.slices, part = blockIdx.x / p.slices % np;
  const int64_t bh = blockIdx.x / p.slices / np;
  const int e0 = slice * SW;
  if (e0 >= r.Dw) return;
  const int b = static_cast<int>(bh / p.a.H), h = static_cast<int>(bh % p.a.H);
  const int Dx = r.Dx, Dw = r.Dw, ld = Dx + 4;
  float *pw = sm, *S = pw + 2 * kC, *pt = S + (STATE ? 0 : Dx * SW), *rows = pt + (STATE ? 0 : kC * kLdP);
  const int per_buf = (STATE ? 1 : 2) * kC * ld + kC * SW;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // a warp covers 4 x 8 threads of 16 x 16: few distinct rows in each of its loads
  const int tx = (warp & 1) * 8 + (lane & 7), ty = (warp >> 1) * 4 + (lane >> 3);
  const int tokens = ret_tokens(p.a.lens, b, p.a.L);
  const int n = (tokens + kC - 1) / kC;
  const float lg = p.a.lg.g[h];
  const T *x = static_cast<const T *>(r.x) + b * r.xs.b + (h / r.xg) * r.xs.h;
  const T *y = static_cast<const T *>(r.y) + b * r.ys.b + (h / r.yg) * r.ys.h;
  const T *wp = static_cast<const T *>(r.w) + b * r.ws.b + (h / r.wg) * r.ws.h + e0;
  const float *rec = r.rec + bh * r.records * Dx * Dw;
  const int after = r.reverse ? 0 : 1;  // o_0 meets the state in front of it decayed once, in time
  int sh = 0;
  while ((kPer << sh) < Dx) ++sh;

  if (tid <= kC) pw[tid] = exp2f(lg * static_cast<float>(tid));
  const int c0 = part * p.cpp, c1 = part == p.parts - 1 ? n : min(n, c0 + p.cpp);
  const bool keep = STATE || (part == p.parts - 1 && r.end);  // the state behind the last chunk is wanted

  Rows<T, kNX> xr, yr;
  Rows<T, kNW> wr;
  auto begin = [&](int c, float *to) {
    const int t0 = (r.reverse ? n - 1 - c : c) * kC, nv = min(kC, tokens - t0);
    yr.begin(y, r.ys.t, t0, nv, r.reverse, sh, Dx, to, ld);
    wr.begin(wp, r.ws.t, t0, nv, r.reverse, kShW, min(SW, Dw - e0), to + kC * ld, SW);
    if (!STATE) xr.begin(x, r.xs.t, t0, nv, r.reverse, sh, Dx, to + kC * ld + kC * SW, ld);
    if constexpr (sizeof(T) == 4) copies_commit();
  };
  auto settle = [&](float *to) {
    yr.settle(sh, to, ld);
    wr.settle(kShW, to + kC * ld, SW);
    if (!STATE) xr.settle(sh, to + kC * ld + kC * SW, ld);
    if constexpr (sizeof(T) == 4) copies_wait<0>();
  };
  if (c0 < c1) begin(c0, rows);

  // the thread's share of the state: features 64 i + 4 ty + u, columns CW tx + k
  float s[NI][4][CW];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int k = 0; k < CW; ++k) {
        const int d = 64 * i + 4 * ty + u, e = e0 + CW * tx + k;
        s[i][u][k] = STATE || d >= Dx || e >= Dw ? 0.f : ret_start(r, rec, bh, part, p.cpp, n, tokens, kC, lg, d, e);
      }
  auto show = [&] {
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int d = 64 * i + 4 * ty + u;
        if (d < Dx) put<CW>(S + d * SW + CW * tx, s[i][u]);
      }
  };
  if (!STATE) show();
  if (c0 < c1) settle(rows);

  int cur = 0;
  for (int c = c0; c < c1; ++c) {
    const int t0 = (r.reverse ? n - 1 - c : c) * kC;
    const int nv = min(kC, tokens - t0);
    const bool more = c + 1 < c1;
    const float *yb = rows + cur * per_buf, *wb = yb + kC * ld, *xb = wb + kC * SW;
    cur ^= p.bufs - 1;
    float *next = rows + cur * per_buf;
    __syncthreads();  // chunk and state are there, the other buffer is read
    if (more && p.bufs == 2) begin(c + 1, next);
    if (!STATE) {
      f2 a2[4][4] = {}, o2[4][CW / 2] = {};
      float o[4][CW];
#pragma unroll 2
      for (int d = 0; d < Dx; d += 4) {
        Cols<4> u[4], v[4];
        Cols<CW> st[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          u[i] = cols<4>(xb + (ty + 16 * i) * ld + d);
          v[i] = cols<4>(yb + (tx + 16 * i) * ld + d);
          st[i] = cols<CW>(S + (d + i) * SW + CW * tx);
        }
#pragma unroll
        for (int q = 0; q < 4; q += 2)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j <= i; ++j)
              a2[i][j] = fma2(pack2(u[i].v[q], u[i].v[q + 1]), pack2(v[j].v[q], v[j].v[q + 1]), a2[i][j]);
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < CW; k += 2)
              o2[i][k / 2] = fma2(dup2(u[i].v[q]), pack2(st[q].v[k], st[q].v[k + 1]), o2[i][k / 2]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int j = 0; j <= i; ++j) {
          const int far = ty - tx + 16 * (i - j);
          pt[(ty + 16 * i) * kLdP + tx + 16 * j] = far >= 0 ? sum2(a2[i][j]) * pw[far] : 0.f;
        }
        const float f = pw[ty + 16 * i + after];
#pragma unroll
        for (int k = 0; k < CW; k += 2) {
          const float2 t = unpack2(o2[i][k / 2]);
          o[i][k] = t.x * f, o[i][k + 1] = t.y * f;
        }
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll 2
        for (int t = 16 * j; t < 16 * j + 16; t += 4) {
          Cols<CW> v[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] = cols<CW>(wb + (t + q) * SW + CW * tx);
#pragma unroll
          for (int i = j; i < 4; ++i) {
            const Cols<4> u = cols<4>(pt + (ty + 16 * i) * kLdP + t);
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
              for (int k = 0; k < CW; ++k) o[i][k] = fmaf(u.v[q], v[q].v[k], o[i][k]);
          }
        }
      if (e0 + CW * tx < Dw) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = ty + 16 * i;
          if (t >= nv) break;
#pragma unroll
          for (int k = 0; k < CW; ++k) o[i][k] *= r.out_scale;
          const int64_t at = b * r.os.b + (t0 + (r.reverse ? nv - 1 - t : t)) * r.os.t + h * r.os.h + e0 + CW * tx;
          if (r.o_f32) put<CW>(static_cast<float *>(r.o) + at, o[i]);
          else put<CW>(static_cast<T *>(r.o) + at, o[i]);
        }
      }
    }
    if (keep || more) {
      const float gn = pw[nv];
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int k = 0; k < CW; ++k) s[i][u][k] *= gn;
#pragma unroll 4
      for (int t = 0; t < nv; ++t) {
        const float f = pw[nv - after - t];
        Cols<CW> v = cols<CW>(wb + t * SW + CW * tx);
#pragma unroll
        for (int k = 0; k < CW; ++k) v.v[k] *= f;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          // behind the last feature: the first ones again, not kept
          const int d = 64 * i + 4 * ty;
          const Cols<4> yv = cols<4>(yb + t * ld + (d < Dx ? d : 0));
#pragma unroll
          for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int k = 0; k < CW; k += 2) {
              const float2 t = unpack2(fma2(dup2(yv.v[u]), pack2(v.v[k], v.v[k + 1]), pack2(s[i][u][k], s[i][u][k + 1])));
              s[i][u][k] = t.x, s[i][u][k + 1] = t.y;
            }
        }
      }
    }
    if (more) {
      if (p.bufs == 1) {
        __syncthreads();
        begin(c + 1, next);
      }
      if (!STATE) show();
      settle(next);
    }
  }
  if (keep) {
    float *out = STATE ? const_cast<float *>(rec) + static_cast<int64_t>(part) * Dx * Dw : r.end + bh * r.state;
    const float f = STATE ? 1.f : r.end_scale;
    const int e = e0 + CW * tx;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int d = 64 * i + 4 * ty + u;
#pragma unroll
        for (int k = 0; k < CW; ++k) s[i][u][k] *= f;
        if (d < Dx && e < Dw) put<CW>(out + d * Dw + e, s[i][u]);
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

constexpr int kSmSmem = 227 * 1024;

// CTAs that an SM holds, and whether the next chunk is loaded during this one:
// not where its room would cost the second CTA.
int held_of(int Dx, int SW, bool state, int *bufs) {
  const int most = Dx <= 64 ? 2 : 1;
  for (int held = most; held >= 1; --held)
    for (*bufs = 2; *bufs >= 1; --*bufs)
      if (held * (smem_bytes(Dx, SW, state, *bufs) + 1024) <= kSmSmem + 1024) return held;
  return 0;
}

template <typename T, int NI, int SW, bool STATE>
cudaError_t pass(SimtParams p, int64_t blocks, int Dx, cudaStream_t s) {
  if (!held_of(Dx, SW, STATE, &p.bufs) || blocks >= (1LL << 31)) return cudaErrorNotSupported;
  auto k = retention_simt_kernel<T, NI, SW, STATE>;
  const int bytes = smem_bytes(Dx, SW, STATE, p.bufs);
  const cudaError_t e = allow_smem(k, bytes);
  if (e != cudaSuccess) return e;
  k<<<dim3(static_cast<unsigned>(blocks), 1, p.a.roles), kThreads, bytes, s>>>(p);
  return cudaGetLastError();
}

template <typename T, int NI, int SW>
cudaError_t run(const RetArgs &a, int parts, int widest, int Dx, cudaStream_t s) {
  SimtParams p = {a, parts, 0, (widest + SW - 1) / SW, 0};
  const int chunks = (a.L + kC - 1) / kC;
  p.cpp = (chunks + parts - 1) / parts;
  const int64_t units = static_cast<int64_t>(a.B) * a.H * p.slices;
  if (parts > 1) {
    const cudaError_t e = pass<T, NI, SW, true>(p, units * (parts - 1), Dx, s);
    if (e != cudaSuccess) return e;
  }
  return pass<T, NI, SW, false>(p, units * parts, Dx, s);
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

// The cut that is done first by a model of the CTAs that an SM holds: a chunk takes
// 1 unit of time with slices of 64 columns and 0.65 with 32, 0.4 of that where
// states are summed, 0.7 more for a second CTA on the SM, and a CTA 1 unit to begin
// and end.
Cut cut_of(const RetArgs &a) {
  int Dx, Dw;
  widths(a, &Dx, &Dw);
  const int chunks = (a.L + kC - 1) / kC;
  Cut best = {32, 1};
  double least = 1e300;
  for (int SW = 32; SW <= (Dw <= 32 ? 32 : 64); SW += 32) {
    int64_t units = 0;
    for (int i = 0; i < a.roles; ++i) units += static_cast<int64_t>(a.B) * a.H * ((a.role[i].Dw + SW - 1) / SW);
    auto time = [&](int64_t n, double chunk, bool state) {
      int bufs, held = held_of(Dx, SW, state, &bufs);
      if (n < static_cast<int64_t>(kSMs) * held) held = static_cast<int>((n + kSMs - 1) / kSMs);
      const int64_t slots = static_cast<int64_t>(kSMs) * (held > 0 ? held : 1);
      return static_cast<double>((n + slots - 1) / slots) * (chunk * (1 + 0.7 * (held - 1)) + 1);
    };
    for (int parts = 1; parts <= 32 && (parts == 1 || parts * 2 <= chunks); ++parts) {
      const double chunk = ((chunks + parts - 1) / parts) * (SW == 64 ? 1.0 : 0.65);
      double t = time(units * parts, chunk, false);
      if (parts > 1) t += time(units * (parts - 1), 0.4 * chunk, true);
      if (t < least) least = t, best = {SW, parts};
    }
  }
  return best;
}

// One launch for all roles, laid out for the widest (two launches, each for its own
// widths, one behind the other, take longer: few CTAs each).
template <typename T>
cudaError_t cut_and_run(const RetArgs &a, int parts, cudaStream_t s) {
  int Dx, Dw;
  widths(a, &Dx, &Dw);
  if (Dx > 128) return cudaErrorNotSupported;
  if (cut_of(a).SW == 64) return Dx > 64 ? run<T, 2, 64>(a, parts, Dw, Dx, s) : run<T, 1, 64>(a, parts, Dw, Dx, s);
  return Dx > 64 ? run<T, 2, 32>(a, parts, Dw, Dx, s) : run<T, 1, 32>(a, parts, Dw, Dx, s);
}

struct Sums {
  GroupSumArgs s[3];
};

// A block takes rows of about 1024 pieces of four columns; blockIdx.y: which output.
// Bound by HBM: 84 MB (B1 L4095 H16 over 8, D128) in 19.6 us, cold.
template <typename T>
__global__ void __launch_bounds__(256) group_sum_kernel(const __grid_constant__ Sums p) {
  const GroupSumArgs &a = p.s[blockIdx.y];
  wait_for_previous();
  const int quarter = a.width / 4, per = a.heads * quarter;
  const int rows = max(1, 1024 / per);
  const int64_t all = static_cast<int64_t>(a.B) * a.L;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * rows; r0 < all; r0 += static_cast<int64_t>(gridDim.x) * rows) {
    for (int i = threadIdx.x; i < rows * per; i += 256) {
      const int64_t row = r0 + i / per;
      if (row >= all) break;
      const int h = i % per / quarter, e = i % quarter * 4;
      const int b = static_cast<int>(row) / a.L, t = static_cast<int>(row) % a.L;  // rows below 2^31
      if (t >= ret_tokens(a.lens, b, a.L)) continue;
      // the shares of an output head lie behind one another
      const float *from = a.part + ((row * a.heads + h) * a.g) * a.width + e;
      float s[4] = {};
      for (int j = 0; j < a.g; ++j) {
        const float4 v = __ldcs(reinterpret_cast<const float4 *>(from + static_cast<int64_t>(j) * a.width));
        s[0] += v.x, s[1] += v.y, s[2] += v.z, s[3] += v.w;
      }
      put<4>(static_cast<T *>(a.out) + b * a.os.b + t * a.os.t + h * a.os.h + e, s);
    }
  }
}

}  // namespace

int ret_parts_simt(const RetArgs &a) { return cut_of(a).parts; }

cudaError_t launch_retention_simt(const RetArgs &a, Dtype dt, int parts, cudaStream_t s) {
  return dt == kF32 ? cut_and_run<float>(a, parts, s) : cut_and_run<__nv_bfloat16>(a, parts, s);
}

cudaError_t launch_group_sums(const GroupSumArgs *a, int n, Dtype dt, cudaStream_t s) {
  if (n == 0) return cudaSuccess;
  Sums p = {};
  int64_t want = 1;
  for (int i = 0; i < n; ++i) {
    p.s[i] = a[i];
    const int64_t blocks = (static_cast<int64_t>(a[i].B) * a[i].L * a[i].heads * (a[i].width / 4) + 1023) / 1024;
    if (blocks > want) want = blocks;
  }
  const unsigned grid = static_cast<unsigned>(want < 8 * kSMs ? want : 8 * kSMs);
  return launch_dependent(dt == kF32 ? group_sum_kernel<float> : group_sum_kernel<__nv_bfloat16>, grid, n, 256, 0, s, p);
}

// ---- choice between the kernels, shared host code ----

int ret_parts(const RetArgs &a, Dtype dt) { return ret_tc_supported(a, dt) ? ret_parts_tc(a) : ret_parts_simt(a); }

// The tensor-core kernel takes a returned state from a record of the last part too,
// the other one from its registers.
static int records_of(const RetRole &r, bool tc, int parts) { return tc && r.end ? parts : parts - 1; }

size_t ret_record_floats(const RetArgs &a, Dtype dt, int parts) {
  const bool tc = ret_tc_supported(a, dt);
  size_t n = 0;
  for (int i = 0; i < a.roles; ++i)
    n += static_cast<size_t>(a.role[i].Dx) * a.role[i].Dw * records_of(a.role[i], tc, parts);
  return n * a.B * a.H;
}

void ret_layout(RetArgs *a, Dtype dt, int parts, float *ws) {
  const bool tc = ret_tc_supported(*a, dt);
  for (int i = 0; i < a->roles; ++i) {
    RetRole &r = a->role[i];
    r.rec = ws;
    r.records = records_of(r, tc, parts);
    ws += static_cast<size_t>(a->B) * a->H * r.records * r.Dx * r.Dw;
  }
}

cudaError_t launch_retention(const RetArgs &a, Dtype dt, int parts, cudaStream_t s) {
  return ret_tc_supported(a, dt) ? launch_retention_tc(a, parts, s) : launch_retention_simt(a, dt, parts, s);
}

}  // namespace linattn
