// Backward pass of the selective state space scan (fp32 arithmetic).
//
// Forward, per (b, e, n):  a_t = exp(dt_t A),  h_t = a_t h_(t-1) + u_t B_t,
// u_t = dt_t x_t,  y_t = sum_n C_t h_t + D x_t,  out_t = y_t silu(z_t).
// With gy_t = dout_t silu(z_t) and the adjoint state, from the last token back,
//   g_t = C_t gy_t + a_(t+1) g_(t+1)       (behind the last token: dh_N)
// the gradients are
//   dC_t = sum_e h_t gy_t,   dB_t = sum_e g_t u_t     (over a group's channels)
//   du_t = sum_n g_t B_t,    w_t = g_t a_t h_(t-1),
//   dx_t = du_t dt_t + D gy_t,   d(dt_t) = sum_n w_t A + du_t x_t  (then through softplus)
//   dA = sum_t w_t dt_t,  dD = sum gy_t x_t,  dz_t = dout_t y_t silu'(z_t),  dh_0 = a_1 g_1.
// Dividing h_t by a_t to walk the states back loses everything once a_t is
// small, so states are recomputed from checkpoints instead.
//
// Passes (the first two only when there is more than one part of kPart
// tokens):
//   local   every part's end state from zero, its adjoint contribution to the
//           state before it, sum_t (a_1..a_t) C_t gy_t, and its sum of dt;
//   carry   the parts in order: the state before and the adjoint behind each;
//   main    a part in tiles of TT tokens: forward over all tiles but the last
//           for the state in front of each, then the tiles from the end; in a
//           tile forward again for a checkpoint every 4 tokens, then 4 tokens
//           at a time from the end: their states again into registers, and
//           the adjoint recurrence over them (decays are computed again:
//           holding them too costs the registers of a fourth CTA);
//   sums    dB and dC over the channel tiles, dA, dD and d(dt_bias) over the
//           parts, in a fixed order.
//
// What bounds it: the instructions issued, 4 exponentials and about 15 packed
// fp32 operations per two states and token, plus the sums.  A thread of the
// main pass owns 2 channels x 4 states (packed pairs of channels): sums over
// states cross N/4 lanes, sums over channels the other lanes by a transposing
// exchange (7 shuffles for 16 states), then the CTA's warps in shared memory.
// The two levels of checkpoints keep a CTA within 52 KB and 128 registers a
// thread at 16 states, so that four share an SM; one level (8 tokens of
// states and decays in registers, 104 KB) ran at two CTAs per SM and 366 us
// for B2 L4096 E2048 N16 in bf16.
#include "kernels.h"
#include "mixer_common.cuh"

namespace linattn {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kSub = 4;  // tokens whose states a thread holds

template <int N> constexpr int kPart = N == 8 ? 32 : 64;  // tokens per part

struct BwdRecords {
  float *h;     // [B][S][E][N]: end states, then the states before a part, then dA
  float *g;     // [B][S][E][N]: adjoint contributions, then the adjoints behind a part
  float *dt;    // [B][S][E]
  float *cols;  // [B][S][2][E]: dD, d(dt_bias)
  float *bc;    // [B][tiles][L][2N]: dB | dC of a channel tile
};

// ------------------------------------------------------------------- local

template <typename T, int N>
struct LocalShape {
  static constexpr int LN = N / 4, LC = 32 / LN, CPW = LC * 4, CT = CPW * kWarps;
  static constexpr int TT = 2048 / CT, VC = CT / 8, NV = 2;
  static constexpr int smem = sizeof(float) * (3 * 2048 + 4 * TT * N);
};

template <typename T, int N>
__global__ void __launch_bounds__(kThreads, 4)
    scan_bwd_local_kernel(const __grid_constant__ ScanArgs a, const T *__restrict__ dout,
                          const __grid_constant__ BwdRecords rec, int S) {
  using Sh = LocalShape<T, N>;
  extern __shared__ __align__(16) float smem_local[];
  float *sdt = smem_local, *su = sdt + 2048, *sg = su + 2048;
  f2 *sB = reinterpret_cast<f2 *>(sg + 2048), *sC = sB + Sh::TT * N;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int sl = lane & (Sh::LN - 1), lc = lane / Sh::LN;
  const int Eg = a.E / a.G, gtiles = (Eg + Sh::CT - 1) / Sh::CT, tiles = gtiles * a.G;
  const int tile = blockIdx.x % tiles, part = (blockIdx.x / tiles) % S, b = blockIdx.x / tiles / S;
  const int grp = tile / gtiles, cg = (tile % gtiles) * Sh::CT, e0 = grp * Eg + cg;
  const int nch = min(Sh::CT, Eg - cg);
  const int t0 = part * kPart<N>, t1 = min(a.L, t0 + kPart<N>);
  const T *x = static_cast<const T *>(a.x) + (int64_t)b * a.L * a.ldx + e0;
  const T *dt = static_cast<const T *>(a.dt) + (int64_t)b * a.L * a.lddt + e0;
  const T *z = a.z ? static_cast<const T *>(a.z) + (int64_t)b * a.L * a.ldz + e0 : nullptr;
  const T *dy = dout + (int64_t)b * a.L * a.E + e0;
  const T *Bm = static_cast<const T *>(a.Bm) + (int64_t)b * a.L * a.ldb + grp * N;
  const T *Cm = static_cast<const T *>(a.Cm) + (int64_t)b * a.L * a.ldc + grp * N;
  const int c0 = warp * Sh::CPW + lc * 4, n0 = sl * 4;
  f2 A[2][4], h[2][4], P[2][4], r[2][4];
  {
    float av[4][4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float4 q = c0 + c < nch
                           ? *reinterpret_cast<const float4 *>(a.A + (int64_t)(e0 + c0 + c) * N + n0)
                           : make_float4(0.f, 0.f, 0.f, 0.f);
      av[c][0] = q.x * kLog2e; av[c][1] = q.y * kLog2e;
      av[c][2] = q.z * kLog2e; av[c][3] = q.w * kLog2e;
    }
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        A[c][n] = pack2(av[2 * c][n], av[2 * c + 1][n]);
        h[c][n] = r[c][n] = dup2(0.f);
        P[c][n] = dup2(1.f);
      }
  }
  float dtsum[4] = {0.f, 0.f, 0.f, 0.f};
  const int vcol = (tid % Sh::VC) * 8, vrow = tid / Sh::VC;
  const bool vin = vcol < nch;
  float bias[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) bias[i] = 0.f;
  if (vin && a.dt_bias) load8(a.dt_bias + e0 + vcol, bias);

  for (int tb = t0; tb < t1; tb += Sh::TT) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < Sh::NV; ++i) {
      const int row = vrow + i * (kThreads / Sh::VC), s = row * Sh::CT + vcol;
      const int64_t t = tb + row;
      float dv[8], uv[8], gv[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) dv[k] = uv[k] = gv[k] = 0.f;
      if (vin && t < t1) {
        load8(x + t * a.ldx + vcol, uv);
        load8(dt + t * a.lddt + vcol, dv);
        load8(dy + t * a.E + vcol, gv);
        if (z) {
          float zv[8];
          load8(z + t * a.ldz + vcol, zv);
#pragma unroll
          for (int k = 0; k < 8; ++k) gv[k] *= zv[k] * sigmoid_f32(zv[k]);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float q = dv[k] + bias[k];
          dv[k] = a.softplus ? softplus_f32(q) : q;
          uv[k] *= dv[k];
        }
      }
      store8(&sdt[s], dv);
      store8(&su[s], uv);
      store8(&sg[s], gv);
    }
    for (int v = tid; v < Sh::TT * N / 8; v += kThreads) {
      const int row = v / (N / 8), col = (v % (N / 8)) * 8;
      const int64_t t = tb + row;
      float q[8], p[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) q[k] = p[k] = 0.f;
      if (t < t1) {
        load8(Bm + t * a.ldb + col, q);
        load8(Cm + t * a.ldc + col, p);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        sB[row * N + k % 4 * Sh::LN + col / 4 + k / 4] = dup2(q[k]);
        sC[row * N + k % 4 * Sh::LN + col / 4 + k / 4] = dup2(p[k]);
      }
    }
    __syncthreads();
#pragma unroll 2
    for (int t = 0; t < Sh::TT; ++t) {
      const int s = t * Sh::CT + c0;
      const ulonglong2 dq = *reinterpret_cast<const ulonglong2 *>(&sdt[s]);
      const ulonglong2 uq = *reinterpret_cast<const ulonglong2 *>(&su[s]);
      const ulonglong2 gq = *reinterpret_cast<const ulonglong2 *>(&sg[s]);
      const f2 d2[2] = {{dq.x}, {dq.y}}, u2[2] = {{uq.x}, {uq.y}}, g2[2] = {{gq.x}, {gq.y}};
      f2 bn[4], cn[4];
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        bn[n] = sB[t * N + n * Sh::LN + sl];
        cn[n] = sC[t * N + n * Sh::LN + sl];
      }
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const f2 e = ex2_2(mul2(d2[c], A[c][n]));
          h[c][n] = fma2(e, h[c][n], mul2(u2[c], bn[n]));
          P[c][n] = mul2(P[c][n], e);
          r[c][n] = fma2(P[c][n], mul2(g2[c], cn[n]), r[c][n]);
        }
      const float2 p = unpack2(d2[0]), q = unpack2(d2[1]);
      dtsum[0] += p.x; dtsum[1] += p.y; dtsum[2] += q.x; dtsum[3] += q.y;
    }
  }
  const int64_t rc = ((int64_t)b * S + part) * a.E + e0 + c0;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    if (c0 + c < nch) {
      auto half = [&](const f2 &v) { const float2 q = unpack2(v); return c & 1 ? q.y : q.x; };
      const int cp = c / 2;
      *reinterpret_cast<float4 *>(rec.h + (rc + c) * N + n0) =
          make_float4(half(h[cp][0]), half(h[cp][1]), half(h[cp][2]), half(h[cp][3]));
      *reinterpret_cast<float4 *>(rec.g + (rc + c) * N + n0) =
          make_float4(half(r[cp][0]), half(r[cp][1]), half(r[cp][2]), half(r[cp][3]));
      if (sl == 0) rec.dt[rc + c] = dtsum[c];
    }
  }
}

// ------------------------------------------------------------------- carry

// One thread per (b, e, n) and direction: the records of the parts in order,
// in place.  h: slot p <- the state before part p.  g: slot p <- the adjoint
// behind part p.
__global__ void __launch_bounds__(256)
    scan_bwd_carry_kernel(const __grid_constant__ ScanArgs a, const float *__restrict__ dhN,
                          const __grid_constant__ BwdRecords rec, int S) {
  const int64_t EN = (int64_t)a.E * a.N;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= a.B * EN) return;
  const int64_t b = i / EN, en = i - b * EN;
  const int e = static_cast<int>(en / a.N);
  const float A = a.A[en] * kLog2e;
  const bool back = blockIdx.y == 1;
  float *r = (back ? rec.g : rec.h) + b * S * EN + en;
  const float *sd = rec.dt + b * S * a.E + e;
  float acc = back ? (dhN ? dhN[i] : 0.f) : (a.h0 ? a.h0[i] : 0.f);
  constexpr int kAhead = 8;
  for (int q0 = 0; q0 < S; q0 += kAhead) {
    float v[kAhead], d[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int p = back ? S - 1 - (q0 + k) : q0 + k;
      const bool in = q0 + k < S;
      v[k] = in ? r[p * EN] : 0.f;
      d[k] = in ? sd[(int64_t)p * a.E] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (q0 + k < S) {
        const int p = back ? S - 1 - (q0 + k) : q0 + k;
        r[p * EN] = acc;
        acc = fmaf(ex2(d[k] * A), acc, v[k]);
      }
    }
  }
}

// -------------------------------------------------------------------- main

template <typename T, int N>
struct MainShape {
  static constexpr int LN = N / 4, LC = 32 / LN, CPW = LC * 2, CT = CPW * kWarps;
  static constexpr int TT = 1024 / CT < 32 ? 1024 / CT : 32;  // tokens per tile
  static constexpr int NT = kPart<N> / TT;                    // tiles per part
  static constexpr int NSUB = TT / kSub;
  static constexpr int VC = CT / 8;
  static constexpr int VECS = TT * VC;  // 8-channel vectors of a tile: at most one per thread
};

template <typename T, int N>
struct MainSmem {
  using Sh = MainShape<T, N>;
  float dt[Sh::TT * Sh::CT];  // then sum_n w A
  float u[Sh::TT * Sh::CT];   // then du
  float g[Sh::TT * Sh::CT];   // gy, then y
  f2 B[Sh::TT * N], C[Sh::TT * N];      // each value twice; state 4 l + n at n LN + l
  f2 coarse[Sh::NT - 1][4][kThreads];   // states in front of tiles 1 ..
  f2 fine[Sh::NSUB - 1][4][kThreads];   // states in front of a tile's groups 1 ..
  float cols[2][Sh::VECS * 8];          // dD and d(dt_bias) of each vector's threads
  float red[2][kWarps][kSub][2 * N];
};

template <typename T, int N>
__global__ void __launch_bounds__(kThreads, N <= 16 ? 4 : 2)
    scan_bwd_main_kernel(const __grid_constant__ ScanArgs a, const __grid_constant__ ScanGrads gr,
                         const __grid_constant__ BwdRecords rec, int S) {
  using Sh = MainShape<T, N>;
  constexpr int CT = Sh::CT, LN = Sh::LN, TT = Sh::TT;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  MainSmem<T, N> &sm = *reinterpret_cast<MainSmem<T, N> *>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int sl = lane & (LN - 1), lc = lane / LN;
  const int Eg = a.E / a.G, gtiles = (Eg + CT - 1) / CT, tiles = gtiles * a.G;
  const int tile = blockIdx.x % tiles, part = (blockIdx.x / tiles) % S, b = blockIdx.x / tiles / S;
  const int grp = tile / gtiles, cg = (tile % gtiles) * CT, e0 = grp * Eg + cg;
  const int nch = min(CT, Eg - cg);
  const int t0 = part * kPart<N>, t1 = min(a.L, t0 + kPart<N>);
  const bool gated = a.z != nullptr;

  // this thread's vector of a staged tile
  const int vcol = (tid % Sh::VC) * 8, vrow = tid / Sh::VC;
  const bool vlive = tid < Sh::VECS, vin = vlive && vcol < nch;
  const int vs = vrow * CT + vcol;
  if (vlive)
#pragma unroll
    for (int i = 0; i < 8; ++i) sm.cols[0][tid * 8 + i] = sm.cols[1][tid * 8 + i] = 0.f;

  // The tile at token tb into shared memory (first = true: what the states
  // need, otherwise everything).
  auto stage = [&](int tb, bool all) {
    const int64_t t = tb + vrow;
    if (vlive) {
      raw8<T> rx, rd, rg, rz;
      rx.zero();
      rd.zero();
      rg.zero();
      rz.zero();
      const bool in = vin && t < t1;
      if (in) {
        const int64_t row = (int64_t)b * a.L + t;
        rx.load(static_cast<const T *>(a.x) + row * a.ldx + e0 + vcol);
        rd.load(static_cast<const T *>(a.dt) + row * a.lddt + e0 + vcol);
        if (all) {
          rg.load(static_cast<const T *>(gr.dy) + row * a.E + e0 + vcol);
          if (gated) rz.load(static_cast<const T *>(a.z) + row * a.ldz + e0 + vcol);
        }
      }
      f2 dv[4], uv[4], bias[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) bias[i] = dup2(0.f);
      if (vin && a.dt_bias) load8p(a.dt_bias + e0 + vcol, bias);
      rx.getp(uv);
      rd.getp(dv);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        dv[k] = add2(dv[k], bias[k]);
        if (a.softplus) dv[k] = softplus_f2(dv[k]);
        if (!in) dv[k] = dup2(0.f);
        uv[k] = mul2(uv[k], dv[k]);
      }
      store8p(&sm.dt[vs], dv);
      store8p(&sm.u[vs], uv);
      if (all) {
        f2 gv[4];
        rg.getp(gv);
        if (gated) {
          f2 zv[4];
          rz.getp(zv);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 q = unpack2(zv[k]);
            gv[k] = mul2(gv[k], mul2(zv[k], pack2(sigmoid_f32(q.x), sigmoid_f32(q.y))));
          }
        }
        store8p(&sm.g[vs], gv);
      }
    }
    constexpr int BV = TT * N / 8;
    for (int v = tid; v < (all ? 2 : 1) * BV; v += kThreads) {
      const bool second = v >= BV;
      const int r = second ? v - BV : v;
      const int row = r / (N / 8), col = (r % (N / 8)) * 8;
      float q[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) q[k] = 0.f;
      if (tb + row < t1) {
        const int64_t tr = (int64_t)b * a.L + tb + row;
        load8((second ? static_cast<const T *>(a.Cm) + tr * a.ldc
                      : static_cast<const T *>(a.Bm) + tr * a.ldb) + grp * N + col, q);
      }
      f2 *d = (second ? sm.C : sm.B) + row * N + col / 4;
#pragma unroll
      for (int k = 0; k < 8; ++k) d[k % 4 * LN + k / 4] = dup2(q[k]);
    }
  };

  // this thread's channel pair and states
  const int c0 = warp * Sh::CPW + lc * 2, n0 = sl * 4;
  const bool cin = c0 < nch;  // pairs: widths are multiples of 8
  const int64_t en = (int64_t)(e0 + c0) * N + n0;            // within [E][N]
  const int64_t ben = (int64_t)b * a.E * N + en;             // within [B][E][N]
  const int64_t pen = ((int64_t)b * S + part) * a.E * N + en;  // within the records
  auto load_pair = [&](const float *p, f2 (&v)[4], float scale) {
    float4 lo = make_float4(0.f, 0.f, 0.f, 0.f), hi = lo;
    if (p && cin) {
      lo = *reinterpret_cast<const float4 *>(p);
      hi = *reinterpret_cast<const float4 *>(p + N);
    }
    v[0] = pack2(lo.x * scale, hi.x * scale);
    v[1] = pack2(lo.y * scale, hi.y * scale);
    v[2] = pack2(lo.z * scale, hi.z * scale);
    v[3] = pack2(lo.w * scale, hi.w * scale);
  };
  auto store_pair = [&](float *p, const f2 (&v)[4]) {
    if (!cin) return;
    const float2 q0 = unpack2(v[0]), q1 = unpack2(v[1]), q2 = unpack2(v[2]), q3 = unpack2(v[3]);
    *reinterpret_cast<float4 *>(p) = make_float4(q0.x, q1.x, q2.x, q3.x);
    *reinterpret_cast<float4 *>(p + N) = make_float4(q0.y, q1.y, q2.y, q3.y);
  };
  const float *start = S > 1 ? rec.h + pen : a.h0 ? a.h0 + ben : nullptr;
  f2 A[4], h[4], gc[4], dA[4];
  load_pair(a.A + en, A, kLog2e);
  load_pair(start, h, 1.f);
  load_pair(S > 1 ? rec.g + pen : gr.dhN ? gr.dhN + ben : nullptr, gc, 1.f);
#pragma unroll
  for (int n = 0; n < 4; ++n) dA[n] = dup2(0.f);

  auto tok2 = [&](const float *arr, int t) {
    return f2{*reinterpret_cast<const unsigned long long *>(&arr[t * CT + c0])};
  };
  auto shared4 = [&](const f2 *arr, int t, f2 (&v)[4]) {
#pragma unroll
    for (int n = 0; n < 4; ++n) v[n] = arr[t * N + n * LN + sl];
  };
  // h one token on
  auto advance = [&](int t) {
    const f2 d2 = tok2(sm.dt, t), u2 = tok2(sm.u, t);
    f2 bn[4];
    shared4(sm.B, t, bn);
#pragma unroll
    for (int n = 0; n < 4; ++n) h[n] = fma2(ex2_2(mul2(d2, A[n])), h[n], mul2(u2, bn[n]));
  };

  const int ntiles = (t1 - t0 + TT - 1) / TT;
  for (int q = 0; q + 1 < ntiles; ++q) {
    stage(t0 + q * TT, false);
    __syncthreads();
#pragma unroll 4
    for (int t = 0; t < TT; ++t) advance(t);
#pragma unroll
    for (int n = 0; n < 4; ++n) sm.coarse[q][n][tid] = h[n];
    __syncthreads();
  }

  for (int q = ntiles - 1; q >= 0; --q) {
    const int tb = t0 + q * TT;
    const int nsub = (min(TT, t1 - tb) + kSub - 1) / kSub;
    stage(tb, true);
    if (q > 0) {
#pragma unroll
      for (int n = 0; n < 4; ++n) h[n] = sm.coarse[q - 1][n][tid];
    } else {
      load_pair(start, h, 1.f);
    }
    f2 first[4] = {h[0], h[1], h[2], h[3]};
    __syncthreads();
    for (int sub = 0; sub + 1 < nsub; ++sub) {
#pragma unroll
      for (int j = 0; j < kSub; ++j) advance(sub * kSub + j);
#pragma unroll
      for (int n = 0; n < 4; ++n) sm.fine[sub][n][tid] = h[n];
    }

    float *bc = rec.bc + (((int64_t)b * tiles + tile) * a.L + tb) * (2 * N);
    for (int sub = nsub - 1; sub >= 0; --sub) {
      f2 hs[kSub + 1][4], ys[kSub];  // hs[j]: the state in front of token j
#pragma unroll
      for (int n = 0; n < 4; ++n) hs[0][n] = sub > 0 ? sm.fine[sub > 0 ? sub - 1 : 0][n][tid] : first[n];
#pragma unroll
      for (int j = 0; j < kSub; ++j) {
        const int t = sub * kSub + j;
        const f2 d2 = tok2(sm.dt, t), u2 = tok2(sm.u, t);
        f2 bn[4], cn[4];
        shared4(sm.B, t, bn);
        shared4(sm.C, t, cn);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          hs[j + 1][n] = fma2(ex2_2(mul2(d2, A[n])), hs[j][n], mul2(u2, bn[n]));
          ys[j] = n ? fma2(hs[j + 1][n], cn[n], ys[j]) : mul2(hs[j + 1][n], cn[n]);
        }
      }
#pragma unroll
      for (int j = kSub - 1; j >= 0; --j) {
        const int t = sub * kSub + j;
        const f2 d2 = tok2(sm.dt, t), u2 = tok2(sm.u, t), g2 = tok2(sm.g, t);
        f2 bn[4], cn[4];
        shared4(sm.B, t, bn);
        shared4(sm.C, t, cn);
        f2 du, dd;
        float r[8];  // dB, dC of this thread's states, over its channel pair
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const f2 g = fma2(cn[n], g2, gc[n]);
          r[n] = sum2(mul2(g, u2));
          r[4 + n] = sum2(mul2(hs[j + 1][n], g2));
          du = n ? fma2(g, bn[n], du) : mul2(g, bn[n]);
          gc[n] = mul2(g, ex2_2(mul2(d2, A[n])));
          const f2 w = mul2(gc[n], hs[j][n]);
          dd = n ? fma2(w, A[n], dd) : mul2(w, A[n]);
          dA[n] = fma2(w, d2, dA[n]);
        }
        // over the states: lane bit 0 takes one channel of the pair
        {
          const bool hi = lane & 1;
          const float2 p0 = unpack2(du), p1 = unpack2(dd), p2 = unpack2(ys[j]);
          float v0 = hi ? p0.y : p0.x, v1 = hi ? p1.y : p1.x, v2 = hi ? p2.y : p2.x;
          v0 += __shfl_xor_sync(0xffffffffu, hi ? p0.x : p0.y, 1);
          v1 += __shfl_xor_sync(0xffffffffu, hi ? p1.x : p1.y, 1);
          v2 += __shfl_xor_sync(0xffffffffu, hi ? p2.x : p2.y, 1);
#pragma unroll
          for (int o = 2; o < LN; o <<= 1) {
            v0 += __shfl_xor_sync(0xffffffffu, v0, o);
            v1 += __shfl_xor_sync(0xffffffffu, v1, o);
            v2 += __shfl_xor_sync(0xffffffffu, v2, o);
          }
          __syncwarp();  // every lane has read this token's inputs
          if (sl < 2) {
            const int s = t * CT + c0 + sl;
            sm.u[s] = v0;
            sm.dt[s] = v1;
            sm.g[s] = v2;
          }
        }
        // over the channels: each lane bit keeps half of the eight values
        float *rd = sm.red[sub & 1][warp][j];
        {
          const bool h1 = lane & LN;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float keep = h1 ? r[4 + k] : r[k], send = h1 ? r[k] : r[4 + k];
            r[k] = keep + __shfl_xor_sync(0xffffffffu, send, LN);
          }
          int idx = (h1 ? N : 0) + n0;
          if constexpr (Sh::LC >= 4) {
            const bool h2 = lane & (2 * LN);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float keep = h2 ? r[2 + k] : r[k], send = h2 ? r[k] : r[2 + k];
              r[k] = keep + __shfl_xor_sync(0xffffffffu, send, 2 * LN);
            }
            idx += h2 ? 2 : 0;
            if constexpr (Sh::LC >= 8) {
              const bool h3 = lane & (4 * LN);
              const float keep = h3 ? r[1] : r[0], send = h3 ? r[0] : r[1];
              r[0] = keep + __shfl_xor_sync(0xffffffffu, send, 4 * LN);
              idx += h3 ? 1 : 0;
              if constexpr (Sh::LC >= 16) r[0] += __shfl_xor_sync(0xffffffffu, r[0], 8 * LN);
              if (Sh::LC < 16 || !(lane & (8 * LN))) rd[idx] = r[0];
            } else {
              *reinterpret_cast<float2 *>(&rd[idx]) = make_float2(r[0], r[1]);
            }
          } else {
            *reinterpret_cast<float4 *>(&rd[idx]) = make_float4(r[0], r[1], r[2], r[3]);
          }
        }
      }
      // the other half of `red` is written before this half is again, with
      // this barrier in between
      __syncthreads();
      for (int i = tid; i < kSub * 2 * N; i += kThreads) {
        const int t = sub * kSub + i / (2 * N);
        if (tb + t < t1) {
          const float *p = &sm.red[sub & 1][0][0][0] + i;
          float s = p[0];
#pragma unroll
          for (int w = 1; w < kWarps; ++w) s += p[w * kSub * 2 * N];
          bc[(int64_t)sub * kSub * 2 * N + i] = s;
        }
      }
    }

    // the tile's per-token gradients, and its share of the column sums
    const int64_t t = tb + vrow;
    if (vin && t < t1) {
      const int64_t row = (int64_t)b * a.L + t, o = row * a.E + e0 + vcol;
      f2 xv[4], dv[4], gv[4], du[4], dd[4], yv[4], dskip[4], bias[4];
      load8p(static_cast<const T *>(a.x) + row * a.ldx + e0 + vcol, xv);
      load8p(static_cast<const T *>(a.dt) + row * a.lddt + e0 + vcol, dv);
      load8p(static_cast<const T *>(gr.dy) + o, gv);
#pragma unroll
      for (int i = 0; i < 4; ++i) dskip[i] = bias[i] = dup2(0.f);
      if (a.D) load8p(a.D + e0 + vcol, dskip);
      if (a.dt_bias) load8p(a.dt_bias + e0 + vcol, bias);
      load8p(&sm.u[vs], du);
      load8p(&sm.dt[vs], dd);
      load8p(&sm.g[vs], yv);
      if (gated) {
        f2 zv[4];
        load8p(static_cast<const T *>(a.z) + row * a.ldz + e0 + vcol, zv);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 z2 = unpack2(zv[k]);
          const f2 sg = pack2(sigmoid_f32(z2.x), sigmoid_f32(z2.y));
          // silu'(z) = s (1 + z (1 - s))
          const f2 slope = mul2(sg, fma2(zv[k], fma2(sg, dup2(-1.f), dup2(1.f)), dup2(1.f)));
          yv[k] = mul2(mul2(gv[k], fma2(dskip[k], xv[k], yv[k])), slope);
          gv[k] = mul2(gv[k], mul2(zv[k], sg));
        }
        store8p(static_cast<T *>(gr.dz) + o, yv);
      }
      f2 sD[4], sb[4];
      load8p(&sm.cols[0][tid * 8], sD);
      load8p(&sm.cols[1][tid * 8], sb);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const f2 v = add2(dv[k], bias[k]);
        dv[k] = a.softplus ? softplus_f2(v) : v;
        dd[k] = fma2(du[k], xv[k], mul2(dd[k], dup2(kLn2)));
        if (a.softplus) {
          const float2 r = unpack2(v);
          dd[k] = mul2(dd[k], pack2(sigmoid_f32(r.x), sigmoid_f32(r.y)));
        }
        du[k] = fma2(du[k], dv[k], mul2(dskip[k], gv[k]));
        sD[k] = fma2(gv[k], xv[k], sD[k]);
        sb[k] = add2(sb[k], dd[k]);
      }
      store8p(&sm.cols[0][tid * 8], sD);
      store8p(&sm.cols[1][tid * 8], sb);
      store8p(static_cast<T *>(gr.dx) + o, du);
      store8p(static_cast<T *>(gr.ddt) + o, dd);
    }
    // the next tile's staging writes only what this thread itself has read
    // here, and B and C, which were last read before the barrier above
  }
  store_pair(rec.h + pen, dA);
  if (part == 0 && gr.dh0) store_pair(gr.dh0 + ben, gc);
  __syncthreads();
  float *cols = rec.cols + ((int64_t)b * S + part) * 2 * a.E + e0;
  for (int i = tid; i < 2 * CT; i += kThreads) {
    if (i % CT < nch) {
      const float *p = sm.cols[i / CT] + i % CT;  // [rows of threads][CT]
      float s = 0.f;
      for (int r = 0; r < Sh::VECS / Sh::VC; ++r) s += p[r * CT];
      cols[(i < CT ? 0 : a.E) + i % CT] = s;
    }
  }
}

// -------------------------------------------------------------------- sums

// dB, dC of a token and group: the channel tiles' records in order.
template <typename T>
__global__ void __launch_bounds__(256)
    scan_bwd_bc_kernel(const float *__restrict__ bc, T *__restrict__ dB, T *__restrict__ dC, int B,
                       int L, int G, int N, int gtiles) {
  const int64_t per = (int64_t)L * 2 * N;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)B * G * per) return;
  const int64_t bg = i / per, tk = i - bg * per;
  const float *p = bc + bg * gtiles * per + tk;
  float s = 0.f;
#pragma unroll 8
  for (int k = 0; k < gtiles; ++k) s += p[k * per];
  const int64_t t = tk / (2 * N);
  const int k = static_cast<int>(tk - t * 2 * N);
  const int64_t b = bg / G, g = bg - b * G;
  const int64_t o = ((b * L + t) * G + g) * N + (k < N ? k : k - N);
  io<T>::store((k < N ? dB : dC) + o, s);
}

int bwd_part_tokens(int N) { return N == 8 ? 32 : 64; }
int bwd_tiles(int E, int N, int G) {
  const int CT = 1024 / N;
  return G * ((E / G + CT - 1) / CT);
}

struct BwdSizes {
  size_t h, g, dt, cols, bc;
  int S;
};
BwdSizes bwd_sizes(int B, int L, int E, int N, int G) {
  BwdSizes z;
  const int pt = bwd_part_tokens(N);
  z.S = L > pt ? (L + pt - 1) / pt : 1;
  const size_t bs = (size_t)B * z.S;
  z.h = bs * E * N;
  z.g = z.S > 1 ? z.h : 0;
  z.dt = z.S > 1 ? (bs * E + 3) / 4 * 4 : 0;
  z.cols = bs * 2 * E;
  z.bc = (size_t)B * bwd_tiles(E, N, G) * L * 2 * N;
  return z;
}

template <typename T, int N>
cudaError_t bwd_typed(const ScanArgs &a, const ScanGrads &g, void *ws, cudaStream_t s) {
  const BwdSizes z = bwd_sizes(a.B, a.L, a.E, N, a.G);
  BwdRecords rec;
  rec.h = static_cast<float *>(ws);
  rec.g = rec.h + z.h;
  rec.dt = rec.g + z.g;
  rec.cols = rec.dt + z.dt;
  rec.bc = rec.cols + z.cols;
  cudaError_t e;
  if (z.S > 1) {
    using Sh = LocalShape<T, N>;
    const int tiles = a.G * ((a.E / a.G + Sh::CT - 1) / Sh::CT);
    if ((e = allow_smem(scan_bwd_local_kernel<T, N>, Sh::smem)) != cudaSuccess) return e;
    scan_bwd_local_kernel<T, N><<<(unsigned)((int64_t)a.B * z.S * tiles), kThreads, Sh::smem, s>>>(
        a, static_cast<const T *>(g.dy), rec, z.S);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const int64_t n = (int64_t)a.B * a.E * N;
    scan_bwd_carry_kernel<<<dim3((unsigned)((n + 255) / 256), 2), 256, 0, s>>>(a, g.dhN, rec, z.S);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  const int tiles = bwd_tiles(a.E, N, a.G);
  constexpr int smem = sizeof(MainSmem<T, N>);
  if ((e = allow_smem(scan_bwd_main_kernel<T, N>, smem)) != cudaSuccess) return e;
  scan_bwd_main_kernel<T, N><<<(unsigned)((int64_t)a.B * z.S * tiles), kThreads, smem, s>>>(
      a, g, rec, z.S);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (a.L > 0) {
    const int64_t nbc = (int64_t)a.B * a.G * a.L * 2 * N;
    scan_bwd_bc_kernel<T><<<(unsigned)((nbc + 255) / 256), 256, 0, s>>>(
        rec.bc, static_cast<T *>(g.dBm), static_cast<T *>(g.dCm), a.B, a.L, a.G, N, tiles / a.G);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  e = launch_column_sum(rec.h, a.B * z.S, (int64_t)a.E * N, g.dA, (int64_t)a.E * N, nullptr, s);
  if (e != cudaSuccess || (!g.dD && !g.ddt_bias)) return e;
  return launch_column_sum(rec.cols, a.B * z.S, 2 * (int64_t)a.E, g.dD, a.E, g.ddt_bias, s);
}

template <typename T>
cudaError_t bwd_states(const ScanArgs &a, const ScanGrads &g, void *ws, cudaStream_t s) {
  switch (a.N) {
    case 8: return bwd_typed<T, 8>(a, g, ws, s);
    case 16: return bwd_typed<T, 16>(a, g, ws, s);
    case 32: return bwd_typed<T, 32>(a, g, ws, s);
    case 64: return bwd_typed<T, 64>(a, g, ws, s);
  }
  return cudaErrorNotSupported;
}

}  // namespace

size_t selective_backward_workspace_bytes(int B, int L, int E, int N, int G) {
  const BwdSizes z = bwd_sizes(B, L, E, N, G);
  return sizeof(float) * (z.h + z.g + z.dt + z.cols + z.bc);
}

cudaError_t launch_selective_backward(const ScanArgs &a, const ScanGrads &g, Dtype dt, void *ws,
                                      cudaStream_t s) {
  return dt == kF32 ? bwd_states<float>(a, g, ws, s) : bwd_states<__nv_bfloat16>(a, g, ws, s);
}

}  // namespace linattn
