// Selective state space scan: prompts and single tokens (fp32 arithmetic).
//
// Per batch entry b, channel e and state n:
//   dt_t = softplus(dt_raw_t + dt_bias)        (or the plain sum)
//   h_t  = exp(dt_t A[e][n]) h_(t-1) + dt_t x_t B_t[n]
//   y_t  = sum_n C_t[n] h_t[n] + D[e] x_t,     y_t *= silu(z_t)
// ("Linear Attention Mechanisms" (dileepadev.github.io), the state space form
// h_t = A_t h_(t-1) + B_t x_t beside the gated recurrence of "Gating and
// Selective State Updates": a decay chosen per token.)  B_t and C_t are shared
// by the channels of a group.
//
// What bounds it: one exponential and four fp32 operations per (channel,
// state, token) against 8 bytes per (channel, token) in bf16, so at 16 states
// the special function unit and the fp32 pipe, not memory.  Hence:
//   - a thread owns 4 channels x 4 states in registers: per token it reads one
//     16-byte vector of dt, of u = dt x, and two of B and of C from shared
//     memory for 16 state updates, done as packed pairs of channels;
//   - the sum over states crosses N/4 lanes by a transposing exchange (3
//     shuffles per token for 16 states);
//   - softplus, the D term and the gate are applied once per (channel, token)
//     when a tile of tokens is staged and when it is stored.
// A tile's inputs are copied asynchronously while the previous tile computes;
// the copying thread also converts them, so the raw buffers need no barrier.
//
// Few channels leave SMs idle, so the tokens split into S parts: the state
// pass leaves every part but the last its end state from zero and its sum of
// dt (the part's decay is exp(A sum dt): no product is kept), and the output
// pass folds the records before its part in front of its own scan.
#include "kernels.h"
#include "mixer_common.cuh"

namespace linattn {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 2048;  // (token, channel) pairs per tile: 16 per thread
constexpr int kMaxParts = 32;

template <typename T, int N>
struct Shape {
  static constexpr int LN = N / 4;            // lanes that share a channel's states
  static constexpr int LC = 32 / LN;          // channel quads per warp
  static constexpr int CPW = LC * 4;          // channels per warp
  static constexpr int CT = CPW * kWarps;     // channels per CTA
  static constexpr int TT = kTile / CT;       // tokens per tile
  static constexpr int VC = CT / 8;           // 8-channel vectors per token
  static constexpr int NV = kTile / 8 / kThreads;  // vectors per thread (2)
  static constexpr int BV = TT * N / 8;       // vectors of B (and of C) per tile
  static constexpr int NBV = (2 * BV + kThreads - 1) / kThreads;
};

template <typename T, int N>
struct Smem {
  using S = Shape<T, N>;
  float dt[kTile];
  float u[kTile];  // dt x; overwritten by y
  float2 B[S::TT * N], C[S::TT * N];  // each value twice, for the packed pairs
  alignas(16) T raw[3][kTile];        // x, dt, z as loaded
  alignas(16) T rawBC[2 * S::TT * N];
};

// The sum over a channel quad's state lanes.  After it, lane sl of a quad
// holds channel 2 (sl & 1) + ((sl >> 1) & 1) in v[0] (LN >= 4), or channels
// 2 sl, 2 sl + 1 in v[0], v[1] (LN = 2).
template <int LN>
__device__ __forceinline__ void reduce_states(float (&v)[4], int lane) {
  constexpr unsigned all = 0xffffffffu;
  {
    const bool hi = lane & 1;
    const float k0 = hi ? v[2] : v[0], k1 = hi ? v[3] : v[1];
    const float s0 = hi ? v[0] : v[2], s1 = hi ? v[1] : v[3];
    v[0] = k0 + __shfl_xor_sync(all, s0, 1);
    v[1] = k1 + __shfl_xor_sync(all, s1, 1);
  }
  if constexpr (LN >= 4) {
    const bool hi = lane & 2;
    const float k = hi ? v[1] : v[0], s = hi ? v[0] : v[1];
    v[0] = k + __shfl_xor_sync(all, s, 2);
  }
  if constexpr (LN >= 8) v[0] += __shfl_xor_sync(all, v[0], 4);
  if constexpr (LN >= 16) v[0] += __shfl_xor_sync(all, v[0], 8);
}

// OUT: the output pass; otherwise the state pass of the parts but the last.
template <typename T, int N, bool OUT>
__global__ void __launch_bounds__(kThreads)
    scan_kernel(const __grid_constant__ ScanArgs a, float *__restrict__ rec_h,
                float *__restrict__ rec_dt, int S, int part_len) {
  using Sh = Shape<T, N>;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Smem<T, N> &sm = *reinterpret_cast<Smem<T, N> *>(smem_raw);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int sl = lane & (Sh::LN - 1), lc = lane / Sh::LN;
  const int Eg = a.E / a.G;  // channels per group
  const int gtiles = (Eg + Sh::CT - 1) / Sh::CT, tiles = gtiles * a.G;
  const int nparts = OUT ? S : S - 1;
  const int tile = blockIdx.x % tiles;
  const int part = (blockIdx.x / tiles) % nparts;
  const int b = blockIdx.x / tiles / nparts;
  const int grp = tile / gtiles;
  const int cg = (tile % gtiles) * Sh::CT;      // first channel within the group
  const int e0 = grp * Eg + cg;                 // first channel
  const int nch = min(Sh::CT, Eg - cg);         // channels of this tile
  const int len = a.lens ? min(max(a.lens[b], 0), a.L) : a.L;
  const int t0 = part * part_len, t1 = min(len, t0 + part_len);

  const T *x = static_cast<const T *>(a.x) + (int64_t)b * a.L * a.ldx + e0;
  const T *dt = static_cast<const T *>(a.dt) + (int64_t)b * a.L * a.lddt + e0;
  const T *z = a.z ? static_cast<const T *>(a.z) + (int64_t)b * a.L * a.ldz + e0 : nullptr;
  const T *Bm = static_cast<const T *>(a.Bm) + (int64_t)b * a.L * a.ldb + grp * N;
  const T *Cm = static_cast<const T *>(a.Cm) + (int64_t)b * a.L * a.ldc + grp * N;
  T *y = OUT ? static_cast<T *>(a.y) + (int64_t)b * a.L * a.E + e0 : nullptr;

  // this thread's channels and states
  const int c0 = warp * Sh::CPW + lc * 4, n0 = sl * 4;
  f2 A[2][4], h[2][4];  // channel pairs x states; A in units of log2 e
  {
    float av[4][4], hv[4][4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float4 q = make_float4(0.f, 0.f, 0.f, 0.f), r = q;
      if (c0 + c < nch) {
        q = *reinterpret_cast<const float4 *>(a.A + (int64_t)(e0 + c0 + c) * N + n0);
        if (OUT && a.h0)
          r = *reinterpret_cast<const float4 *>(a.h0 + ((int64_t)b * a.E + e0 + c0 + c) * N + n0);
      }
      av[c][0] = q.x * kLog2e; av[c][1] = q.y * kLog2e;
      av[c][2] = q.z * kLog2e; av[c][3] = q.w * kLog2e;
      hv[c][0] = r.x; hv[c][1] = r.y; hv[c][2] = r.z; hv[c][3] = r.w;
    }
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        A[c][n] = pack2(av[2 * c][n], av[2 * c + 1][n]);
        h[c][n] = pack2(hv[2 * c][n], hv[2 * c + 1][n]);
      }
  }
  if constexpr (OUT) {
    // the state before this part: the records of the parts before it
    for (int q = 0; q < part; ++q) {
      const int64_t rc = ((int64_t)b * (S - 1) + q) * a.E + e0 + c0;
      float4 r[4];
      float sd[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const bool in = c0 + c < nch;
        r[c] = in ? *reinterpret_cast<const float4 *>(rec_h + (rc + c) * N + n0)
                  : make_float4(0.f, 0.f, 0.f, 0.f);
        sd[c] = in ? rec_dt[rc + c] : 0.f;
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const f2 s2 = pack2(sd[2 * c], sd[2 * c + 1]);
        const float4 lo = r[2 * c], hi = r[2 * c + 1];
        h[c][0] = fma2(ex2_2(mul2(s2, A[c][0])), h[c][0], pack2(lo.x, hi.x));
        h[c][1] = fma2(ex2_2(mul2(s2, A[c][1])), h[c][1], pack2(lo.y, hi.y));
        h[c][2] = fma2(ex2_2(mul2(s2, A[c][2])), h[c][2], pack2(lo.z, hi.z));
        h[c][3] = fma2(ex2_2(mul2(s2, A[c][3])), h[c][3], pack2(lo.w, hi.w));
      }
    }
  }
  float dtsum[4] = {0.f, 0.f, 0.f, 0.f};

  // per-channel parameters of the staged vectors (one column per thread:
  // kThreads is a multiple of VC)
  const int vcol = (tid % Sh::VC) * 8, vrow = tid / Sh::VC;
  constexpr int kRowStep = kThreads / Sh::VC;
  const bool vin = vcol < nch;
  float bias[8], dskip[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) bias[i] = dskip[i] = 0.f;
  if (vin && a.dt_bias) load8(a.dt_bias + e0 + vcol, bias);
  if (OUT && vin && a.D) load8(a.D + e0 + vcol, dskip);

  auto issue = [&](int tb) {
#pragma unroll
    for (int i = 0; i < Sh::NV; ++i) {
      const int r = vrow + i * kRowStep, t = tb + r;
      const bool ok = vin && t < t1;
      const int64_t tt = ok ? t : 0;
      const int col = ok ? vcol : 0;
      constexpr int per = 16 / sizeof(T);  // elements per 16-byte copy
#pragma unroll
      for (int j = 0; j < 8; j += per) {
        const int s = r * Sh::CT + vcol + j;
        copy16_async(&sm.raw[0][s], x + tt * a.ldx + col + j, ok);
        copy16_async(&sm.raw[1][s], dt + tt * a.lddt + col + j, ok);
        if (OUT && z) copy16_async(&sm.raw[2][s], z + tt * a.ldz + col + j, ok);
      }
    }
#pragma unroll
    for (int i = 0; i < Sh::NBV; ++i) {
      const int v = tid + i * kThreads;
      const int which = v / Sh::BV, r = v % Sh::BV;
      const int row = r / (N / 8), col = (r % (N / 8)) * 8;
      if (which < (OUT ? 2 : 1)) {
        const bool ok = tb + row < t1;
        const int64_t t = ok ? tb + row : 0;
        const T *src = (which ? Cm + t * a.ldc : Bm + t * a.ldb) + col;
        constexpr int per = 16 / sizeof(T);
#pragma unroll
        for (int j = 0; j < 8; j += per) copy16_async(&sm.rawBC[v * 8 + j], src + j, ok);
      }
    }
    copies_commit();
  };

  if (t0 < t1) issue(t0);
  for (int tb = t0; tb < t1; tb += Sh::TT) {
    copies_wait<0>();
    raw8<T> rx[Sh::NV], rz[Sh::NV];
#pragma unroll
    for (int i = 0; i < Sh::NV; ++i) {
      const int r = vrow + i * kRowStep, s = r * Sh::CT + vcol;
      rx[i].load(&sm.raw[0][s]);
      if (OUT && z) rz[i].load(&sm.raw[2][s]);
      float xv[8], dv[8];
      rx[i].get(xv);
      load8(&sm.raw[1][s], dv);
      const bool in = tb + r < t1;  // rows behind the end leave the state as it is
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float q = dv[k] + bias[k];
        dv[k] = in ? (a.softplus ? softplus_f32(q) : q) : 0.f;
        xv[k] *= dv[k];
      }
      store8(&sm.dt[s], dv);
      store8(&sm.u[s], xv);
    }
#pragma unroll
    for (int i = 0; i < Sh::NBV; ++i) {
      const int v = tid + i * kThreads;
      if (v < (OUT ? 2 : 1) * Sh::BV) {
        float q[8];
        load8(&sm.rawBC[v * 8], q);
        float4 *d = reinterpret_cast<float4 *>(v < Sh::BV ? &sm.B[v * 8] : &sm.C[(v - Sh::BV) * 8]);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          d[k] = make_float4(q[2 * k], q[2 * k], q[2 * k + 1], q[2 * k + 1]);
      }
    }
    if (tb + Sh::TT < t1) issue(tb + Sh::TT);
    __syncthreads();
#pragma unroll 4
    for (int t = 0; t < Sh::TT; ++t) {
      const int s = t * Sh::CT + c0;
      const ulonglong2 dq = *reinterpret_cast<const ulonglong2 *>(&sm.dt[s]);
      const ulonglong2 uq = *reinterpret_cast<const ulonglong2 *>(&sm.u[s]);
      const ulonglong2 b01 = *reinterpret_cast<const ulonglong2 *>(&sm.B[t * N + n0]);
      const ulonglong2 b23 = *reinterpret_cast<const ulonglong2 *>(&sm.B[t * N + n0 + 2]);
      const f2 d2[2] = {{dq.x}, {dq.y}}, u2[2] = {{uq.x}, {uq.y}};
      const f2 bn[4] = {{b01.x}, {b01.y}, {b23.x}, {b23.y}};
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int n = 0; n < 4; ++n)
          h[c][n] = fma2(ex2_2(mul2(d2[c], A[c][n])), h[c][n], mul2(u2[c], bn[n]));
      if constexpr (OUT) {
        const ulonglong2 c01 = *reinterpret_cast<const ulonglong2 *>(&sm.C[t * N + n0]);
        const ulonglong2 c23 = *reinterpret_cast<const ulonglong2 *>(&sm.C[t * N + n0 + 2]);
        const f2 cn[4] = {{c01.x}, {c01.y}, {c23.x}, {c23.y}};
        f2 y2[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          y2[c] = mul2(h[c][0], cn[0]);
#pragma unroll
          for (int n = 1; n < 4; ++n) y2[c] = fma2(h[c][n], cn[n], y2[c]);
        }
        const float2 ya = unpack2(y2[0]), yb = unpack2(y2[1]);
        float v[4] = {ya.x, ya.y, yb.x, yb.y};
        reduce_states<Sh::LN>(v, lane);
        // every lane of the warp has read u of this token (the shuffles), so
        // y takes its place
        if constexpr (Sh::LN == 2) {
          *reinterpret_cast<float2 *>(&sm.u[s + 2 * sl]) = make_float2(v[0], v[1]);
        } else if (sl < 4) {
          sm.u[s + 2 * (sl & 1) + (sl >> 1)] = v[0];
        }
      } else {
        const float2 p = unpack2(d2[0]), q = unpack2(d2[1]);
        dtsum[0] += p.x; dtsum[1] += p.y; dtsum[2] += q.x; dtsum[3] += q.y;
      }
    }
    __syncthreads();
    if constexpr (OUT) {
#pragma unroll
      for (int i = 0; i < Sh::NV; ++i) {
        const int r = vrow + i * kRowStep;
        if (vin && tb + r < t1) {
          float yv[8], xv[8];
          load8(&sm.u[r * Sh::CT + vcol], yv);
          rx[i].get(xv);
#pragma unroll
          for (int k = 0; k < 8; ++k) yv[k] = fmaf(dskip[k], xv[k], yv[k]);
          if (z) {
            float zv[8];
            rz[i].get(zv);
#pragma unroll
            for (int k = 0; k < 8; ++k) yv[k] *= zv[k] * sigmoid_f32(zv[k]);
          }
          store8(y + (int64_t)(tb + r) * a.E + vcol, yv);
        }
      }
    }
  }

  // the state after this part: the record, or the final state
  float *hd = nullptr;
  if constexpr (OUT) {
    if (part == S - 1 && a.hN) hd = a.hN + ((int64_t)b * a.E + e0 + c0) * N + n0;
  } else {
    const int64_t rc = ((int64_t)b * (S - 1) + part) * a.E + e0 + c0;
    hd = rec_h + rc * N + n0;
    if (sl == 0)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c0 + c < nch) rec_dt[rc + c] = dtsum[c];
  }
  if (hd) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const float2 p = unpack2(h[c][0]), q = unpack2(h[c][1]), r = unpack2(h[c][2]),
                   s = unpack2(h[c][3]);
      if (c0 + 2 * c < nch)
        *reinterpret_cast<float4 *>(hd + 2 * c * N) = make_float4(p.x, q.x, r.x, s.x);
      if (c0 + 2 * c + 1 < nch)
        *reinterpret_cast<float4 *>(hd + (2 * c + 1) * N) = make_float4(p.y, q.y, r.y, s.y);
    }
  }
}

template <typename T, int N>
cudaError_t scan_typed(const ScanArgs &a, void *ws, int S, cudaStream_t s) {
  using Sh = Shape<T, N>;
  constexpr int smem = sizeof(Smem<T, N>);
  const int tiles = a.G * ((a.E / a.G + Sh::CT - 1) / Sh::CT);
  const int part_len = selective_part_len(a.L, S);
  float *rec_h = static_cast<float *>(ws);
  float *rec_dt = rec_h + (size_t)a.B * (S - 1) * a.E * N;
  if (S > 1) {
    cudaError_t e = allow_smem(scan_kernel<T, N, false>, smem);
    if (e != cudaSuccess) return e;
    scan_kernel<T, N, false><<<(unsigned)((int64_t)a.B * (S - 1) * tiles), kThreads, smem, s>>>(
        a, rec_h, rec_dt, S, part_len);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  cudaError_t e = allow_smem(scan_kernel<T, N, true>, smem);
  if (e != cudaSuccess) return e;
  scan_kernel<T, N, true><<<(unsigned)((int64_t)a.B * S * tiles), kThreads, smem, s>>>(
      a, rec_h, rec_dt, S, part_len);
  return cudaGetLastError();
}

template <typename T>
cudaError_t scan_states(const ScanArgs &a, void *ws, int S, cudaStream_t s) {
  switch (a.N) {
    case 8: return scan_typed<T, 8>(a, ws, S, s);
    case 16: return scan_typed<T, 16>(a, ws, S, s);
    case 32: return scan_typed<T, 32>(a, ws, S, s);
    case 64: return scan_typed<T, 64>(a, ws, S, s);
  }
  return cudaErrorNotSupported;
}

// One token, in place on the fp32 state.  Bound by the state's bytes (8 per
// element): N/4 lanes share a channel, each streams one 16-byte piece of its
// states.  A thread keeps its channel's parameters for U sequences, whose
// state loads are all in flight at once.
template <typename T, int N, int U>
__global__ void __launch_bounds__(256) scan_step_kernel(const __grid_constant__ ScanArgs a) {
  constexpr int LN = N / 4, PER = 256 / LN;
  const int tid = threadIdx.x, sl = tid & (LN - 1);
  const int e = blockIdx.x * PER + tid / LN;  // equal in all lanes of a channel
  const bool in = e < a.E;
  const int ec = in ? e : 0;
  const int goff = (a.G == 1 ? 0 : ec / (a.E / a.G)) * N + sl * 4;
  const float4 A = *reinterpret_cast<const float4 *>(a.A + (int64_t)ec * N + sl * 4);
  const float bias = a.dt_bias ? a.dt_bias[ec] : 0.f, skip = a.D ? a.D[ec] : 0.f;
  for (int b0 = blockIdx.y * U; b0 < a.B; b0 += gridDim.y * U) {
    float4 h[U];
    float x[U], d[U], zv[U];
    float4 Bv[U], Cv[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int64_t b = min(b0 + j, a.B - 1);
      h[j] = __ldcs(reinterpret_cast<const float4 *>(a.hN + (b * a.E + ec) * N) + sl);
      x[j] = io<T>::load(static_cast<const T *>(a.x) + b * a.ldx + ec);
      d[j] = io<T>::load(static_cast<const T *>(a.dt) + b * a.lddt + ec);
      zv[j] = a.z ? io<T>::load(static_cast<const T *>(a.z) + b * a.ldz + ec) : 0.f;
      Bv[j] = load4(static_cast<const T *>(a.Bm) + b * a.ldb + goff);
      Cv[j] = load4(static_cast<const T *>(a.Cm) + b * a.ldc + goff);
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const bool live = in && b0 + j < a.B;
      const int64_t row = (int64_t)(b0 + j) * a.E + e;
      float dt = d[j] + bias;
      if (a.softplus) dt = softplus_f32(dt);
      const float dl = dt * kLog2e, u = dt * x[j];
      h[j].x = fmaf(ex2(dl * A.x), h[j].x, u * Bv[j].x);
      h[j].y = fmaf(ex2(dl * A.y), h[j].y, u * Bv[j].y);
      h[j].z = fmaf(ex2(dl * A.z), h[j].z, u * Bv[j].z);
      h[j].w = fmaf(ex2(dl * A.w), h[j].w, u * Bv[j].w);
      if (live) __stcs(reinterpret_cast<float4 *>(a.hN + row * N) + sl, h[j]);
      float y = h[j].x * Cv[j].x;
      y = fmaf(h[j].y, Cv[j].y, y);
      y = fmaf(h[j].z, Cv[j].z, y);
      y = fmaf(h[j].w, Cv[j].w, y);
#pragma unroll
      for (int o = 1; o < LN; o <<= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
      y = fmaf(skip, x[j], y);
      if (a.z) y *= zv[j] * sigmoid_f32(zv[j]);
      if (live && sl == 0) io<T>::store(static_cast<T *>(a.y) + row, y);
    }
  }
}

template <typename T, int N>
cudaError_t step_typed(const ScanArgs &a, cudaStream_t s) {
  constexpr int PER = 256 / (N / 4), kMaxY = 65535;
  const unsigned nx = (a.E + PER - 1) / PER;
  // four sequences per thread once that still gives every SM four CTAs
  if ((int64_t)nx * a.B >= 152 * 4 * 4) {
    const int ny = (a.B + 3) / 4;
    scan_step_kernel<T, N, 4><<<dim3(nx, ny < kMaxY ? ny : kMaxY), 256, 0, s>>>(a);
  } else {
    scan_step_kernel<T, N, 1><<<dim3(nx, a.B < kMaxY ? a.B : kMaxY), 256, 0, s>>>(a);
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t step_states(const ScanArgs &a, cudaStream_t s) {
  switch (a.N) {
    case 8: return step_typed<T, 8>(a, s);
    case 16: return step_typed<T, 16>(a, s);
    case 32: return step_typed<T, 32>(a, s);
    case 64: return step_typed<T, 64>(a, s);
  }
  return cudaErrorNotSupported;
}

}  // namespace

bool selective_states_supported(int N) { return N == 8 || N == 16 || N == 32 || N == 64; }

int selective_part_len(int L, int S) {
  // whole tiles of every state size (64 tokens at most)
  const int l = (L + S - 1) / S;
  return (l + 63) / 64 * 64;
}

int selective_parts(int B, int L, int E, int N, int G) {
  const int CT = 2048 / N;  // channels per CTA
  const int64_t ctas = (int64_t)B * G * ((E / G + CT - 1) / CT);
  // about four CTAs per SM; parts of at least 128 tokens
  int64_t S = (152 * 4) / (ctas > 0 ? ctas : 1);
  const int most = L / 128 < kMaxParts ? L / 128 : kMaxParts;
  if (S > most) S = most;
  if (S < 2) return 1;
  const int len = selective_part_len(L, static_cast<int>(S));
  return (L + len - 1) / len;  // no part is empty
}

size_t selective_workspace_bytes(int B, int E, int N, int S) {
  return S > 1 ? sizeof(float) * (size_t)B * (S - 1) * E * (N + 1) : 0;
}

cudaError_t launch_selective(const ScanArgs &a, Dtype dt, void *ws, int S, cudaStream_t s) {
  return dt == kF32 ? scan_states<float>(a, ws, S, s) : scan_states<__nv_bfloat16>(a, ws, S, s);
}

cudaError_t launch_selective_step(const ScanArgs &a, Dtype dt, cudaStream_t s) {
  return dt == kF32 ? step_states<float>(a, s) : step_states<__nv_bfloat16>(a, s);
}

}  // namespace linattn
