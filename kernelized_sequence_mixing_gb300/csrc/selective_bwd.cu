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
// Passes:
//   local   (the forward kernel's third mode) every part's end state from zero
//           with a checkpoint of it every 8 tokens, its adjoint contribution
//           to the state before it, sum_t (a_1..a_t) C_t gy_t, and its sums
//           of dt;
//   carry   the parts in order: the state before and the adjoint behind each;
//   main    a part in tiles, and 8 tokens at a time from the end: the state in
//           front of them is the checkpoint plus exp(A sum dt) times the state
//           before the part; from it the 8 states into registers, and the
//           adjoint recurrence over them;
//   sums    dB and dC over the channel tiles, dA, dD and d(dt_bias) over the
//           parts, in a fixed order.
// The checkpoints cost N / 2 bytes of memory traffic per (channel, token) each
// way; computing them again in the main pass, in one level or two, cost 12% to
// 25% of its instructions, and it is the instructions and the shared-memory
// pipe that bound it: 2 exponentials (3 with the local pass) and about 13
// packed fp32 operations per two states and token, plus the sums.  A thread of
// the main pass owns 2 channels x 4 states (packed pairs of channels).  Sums over
// states cross N/4 lanes by transposing exchanges, two tokens at a time; sums
// over channels cross the other lanes and the CTA's warps in shared memory.
// (B2 L4096 E2048 N16 in bf16, the whole backward pass: 399 us; when this was
// chosen 407, both kinds by exchanges 414, both in shared memory 431.)
#include "column_sum.cuh"
#include "dependent.cuh"
#include "kernels.h"
#include "mixer_common.cuh"
#include "scan_maps.cuh"

namespace linattn {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kSub = kScanCheckpoint;  // tokens whose states a thread holds
constexpr int kPart = 64;              // tokens per part, of 16 states and more

__device__ __forceinline__ f2 load_f2(const float *p) {
  return f2{*reinterpret_cast<const unsigned long long *>(p)};
}
__device__ __forceinline__ void store_f2(float *p, f2 v) {
  *reinterpret_cast<unsigned long long *>(p) = v.v;
}

struct BwdRecords {
  ScanRecords s;  // s.h: end states, then the states before a part; s.g: likewise behind it
  float *dA;      // [B][S][E][N], in place of s.h
  float *cols;    // [B][S][2][E]: dD, d(dt_bias)
  float *bc;      // [B][tiles][L][2N]: dB | dC of a channel tile
  int part;       // tokens per part
};

// ------------------------------------------------------------------- carry

// One thread per two states of (b, e) and direction: the records of the parts
// in order, in place.  h: slot p <- the state before part p.  g: slot p <- the
// adjoint behind part p.
constexpr int kCarryThreads = 128;
__global__ void __launch_bounds__(kCarryThreads)
    scan_bwd_carry_kernel(const __grid_constant__ ScanArgs a, const float *__restrict__ dhN,
                          const __grid_constant__ BwdRecords rec, int S) {
  wait_for_previous();
  const int64_t EN = (int64_t)a.E * a.N;
  const int64_t i = ((int64_t)blockIdx.x * kCarryThreads + threadIdx.x) * 2;
  if (i >= a.B * EN) return;
  const int64_t b = i / EN, en = i - b * EN;
  const int e = static_cast<int>(en / a.N);
  const float2 rate = unpack2(mul2(load_f2(a.A + en), dup2(kLog2e)));
  const f2 A = pack2(finite_rate(rate.x), finite_rate(rate.y));
  const bool back = blockIdx.y == 1;
  const float *from = back ? dhN : a.h0;
  f2 acc = from ? load_f2(from + i) : dup2(0.f);
  // from the last part back: steps of the other sign
  const int64_t rstep = back ? -EN : EN, sstep = back ? -a.E : a.E;
  float *r = (back ? rec.s.g + (b * S + S - 1) * EN : rec.s.h + b * S * EN) + en;
  const float *sd = rec.s.dt + (back ? b * S + S - 1 : b * S) * a.E + e;
  constexpr int kAhead = 8;
  for (int q = 0; q < S; q += kAhead) {
    f2 v[kAhead];
    float d[kAhead];
    const int m = S - q;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      v[k] = dup2(0.f);
      d[k] = 0.f;
      if (k < m) {
        v[k] = load_f2(r + k * rstep);
        d[k] = sd[k * sstep];
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (k < m) {
        store_f2(r + k * rstep, acc);
        acc = fma2(ex2_2(mul2(dup2(d[k]), A)), acc, v[k]);
      }
    }
    r += kAhead * rstep;
    sd += kAhead * sstep;
  }
}

// -------------------------------------------------------------------- main

template <typename T, int N>
struct MainShape {
  static constexpr int LN = N / 4, LC = 32 / LN, CPW = LC * 2, CT = CPW * kWarps;
  static constexpr int TT = 1024 / CT < 32 ? 1024 / CT : 32;  // tokens per tile
  static constexpr int QC = CT / 4;                           // channel quads per token
  static constexpr int ROWS = kThreads / QC;                  // token rows staged at a time
  static constexpr int NQ = TT / ROWS;                        // quads per thread
  static constexpr int NP = N + 8;  // floats per token of B and of C: rows in different banks
  static constexpr int NBQ = (2 * TT * LN + kThreads - 1) / kThreads;  // quads of B and C per thread
  // tokens whose dB and dC a warp sums at once: as many as cost an SM no CTA
  static constexpr int BT = N == 64 ? 0 : sizeof(T) == 4 ? (N == 16 ? 1 : 2) : N == 32 ? 2 : 4;
  static constexpr bool CKS = N <= 16;  // the next checkpoint waits in shared memory
  // in a warp's [channels][dB | dC] the halves change places such that eight
  // lanes' 16 bytes fill the banks
  static __device__ __forceinline__ int flip(int lc) {
    return N == 8 ? (lc & 2) * 4 : N == 16 ? (lc & 1) * 16 : 0;
  }
};

// s += p[0..V) (first: s = p).
template <int V>
__device__ __forceinline__ void add_vec(float (&s)[V], const float *p, bool first) {
  float v[V];
  if constexpr (V == 4) {
    const float4 q = *reinterpret_cast<const float4 *>(p);
    v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
  } else if constexpr (V == 2) {
    const float2 q = *reinterpret_cast<const float2 *>(p);
    v[0] = q.x; v[1] = q.y;
  } else {
    v[0] = *p;
  }
  if constexpr (V == 1) {
    s[0] = first ? v[0] : s[0] + v[0];
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const float2 q = unpack2(add2(pack2(first ? 0.f : s[i], first ? 0.f : s[i + 1]), pack2(v[i], v[i + 1])));
      s[i] = first ? v[i] : q.x;
      s[i + 1] = first ? v[i + 1] : q.y;
    }
  }
}
template <int V>
__device__ __forceinline__ void store_vec(float *p, const float (&s)[V]) {
  if constexpr (V == 4) *reinterpret_cast<float4 *>(p) = make_float4(s[0], s[1], s[2], s[3]);
  else if constexpr (V == 2) *reinterpret_cast<float2 *>(p) = make_float2(s[0], s[1]);
  else *p = s[0];
}

// A tile as loaded; the epilogue reads it again.
template <typename T, int N>
struct MainStage {
  using Sh = MainShape<T, N>;
  alignas(128) T x[Sh::TT * Sh::CT];
  alignas(128) T dt[Sh::TT * Sh::CT];
  alignas(128) T z[Sh::TT * Sh::CT];
  alignas(128) T dy[Sh::TT * Sh::CT];
  alignas(128) T B[Sh::TT * N];
  alignas(128) T C[Sh::TT * N];
};

template <typename T, int N>
struct MainSmem {
  using Sh = MainShape<T, N>;
  MainStage<T, N> stage[2];
  uint64_t full[2];
  int abort;
  alignas(16) float dt[Sh::TT * Sh::CT];  // then sum_n w A
  float u[Sh::TT * Sh::CT];   // then du
  float g[Sh::TT * Sh::CT];   // gy, then y
  // states 4 l, 4 l + 1 at 2 l, states 4 l + 2, 4 l + 3 at 2 LN + 2 l: eight
  // bytes a lane, whose repeats in the warp share a wavefront (sixteen do not)
  float B[Sh::TT * Sh::NP], C[Sh::TT * Sh::NP];
  alignas(16) float skip[Sh::CT], bias[Sh::CT];  // D and dt_bias
  float cols[2][kThreads * 4];  // dD and d(dt_bias) of each thread's quads
  alignas(16) float ck[2][Sh::CKS ? kThreads * 4 : 4];  // by channel of the pair
  alignas(8) float ckdt[Sh::CKS ? kThreads * 2 : 2];
  alignas(16) float part[kWarps][Sh::BT ? Sh::BT * 256 : 4];  // dB | dC of the warps' channels
  float red[2][kWarps][kSub][2 * N];
};

template <typename T, int N>
__global__ void __launch_bounds__(kThreads, 3)
    scan_bwd_main_kernel(const __grid_constant__ ScanArgs a, const __grid_constant__ ScanGrads gr,
                         const __grid_constant__ ScanMaps maps,
                         const __grid_constant__ BwdRecords rec, int S, unsigned int *timeouts) {
  using Sh = MainShape<T, N>;
  constexpr int CT = Sh::CT, LN = Sh::LN, TT = Sh::TT;
  constexpr bool kOnce = TT <= 2 * kSub;  // one sum over the warps per tile
  extern __shared__ __align__(128) unsigned char smem_raw[];
  MainSmem<T, N> &sm = *reinterpret_cast<MainSmem<T, N> *>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int sl = lane & (LN - 1), lc = lane / LN;
  const int Eg = a.E / a.G, gtiles = (Eg + CT - 1) / CT, tiles = gtiles * a.G;
  const int tile = blockIdx.x % tiles, seg = (blockIdx.x / tiles) % S, b = blockIdx.x / tiles / S;
  const int grp = tile / gtiles, cg = (tile % gtiles) * CT, e0 = grp * Eg + cg;
  const int nch = min(CT, Eg - cg);
  // a constant where it can be: as a parameter it cost 6 of 403 us
  const int tokens = N > 8 ? kPart : rec.part;
  const int t0 = seg * tokens, t1 = min(a.L, t0 + tokens);
  const bool gated = a.z != nullptr;

  // this thread's quads of a staged tile: one column
  const int qcol = (tid % Sh::QC) * 4, qrow = tid / Sh::QC;
  const bool qin = qcol < nch;
  *reinterpret_cast<float4 *>(&sm.cols[0][tid * 4]) = make_float4(0.f, 0.f, 0.f, 0.f);
  *reinterpret_cast<float4 *>(&sm.cols[1][tid * 4]) = make_float4(0.f, 0.f, 0.f, 0.f);

  if (tid == 0) {
    tc::mbar_init(&sm.full[0], 1);
    tc::mbar_init(&sm.full[1], 1);
    tc::mbar_init_fence();
    sm.abort = 0;
  }
  __syncthreads();
  // The tile at token tb.  A box may reach behind the part's end, the
  // sequence's or the group's: those rows and channels are cleared when staged.
  auto issue = [&](int tb, int st) {
    if (tid != 0) return;
    MainStage<T, N> &g = sm.stage[st];
    uint64_t *bar = &sm.full[st];
    constexpr uint32_t rows = TT * CT * sizeof(T), bc = TT * N * sizeof(T);
    tc::mbar_arrive_expect_tx(bar, (gated ? 4 : 3) * rows + 2 * bc);
    tc::tma_load_3d(g.x, &maps.x, e0, tb, b, bar);
    tc::tma_load_3d(g.dt, &maps.dt, e0, tb, b, bar);
    tc::tma_load_3d(g.dy, &maps.dy, e0, tb, b, bar);
    if (gated) tc::tma_load_3d(g.z, &maps.z, e0, tb, b, bar);
    tc::tma_load_3d(g.B, &maps.B, grp * N, tb, b, bar);
    tc::tma_load_3d(g.C, &maps.C, grp * N, tb, b, bar);
  };
  const int ntiles = (t1 - t0 + TT - 1) / TT;
  if (ntiles > 0) issue(t0 + (ntiles - 1) * TT, 0);
  {  // every thread of a column writes the same values, and reads its own
    f2 v[2] = {dup2(0.f), dup2(0.f)}, w[2] = {v[0], v[1]};
    if (qin && a.dt_bias) load4p(a.dt_bias + e0 + qcol, v);
    if (qin && a.D) load4p(a.D + e0 + qcol, w);
    store4p(&sm.bias[qcol], v);
    store4p(&sm.skip[qcol], w);
  }
  // Stage st, whose first `rows` rows count, as the main loop reads it.
  auto convert = [&](int st, int rows) {
    const MainStage<T, N> &g = sm.stage[st];
    f2 bias[2];
    load4p(&sm.bias[qcol], bias);
#pragma unroll
    for (int i = 0; i < Sh::NQ; ++i) {
      const int row = qrow + i * Sh::ROWS, s = row * CT + qcol;
      const bool in = qin && row < rows;  // other channels would count in dB and dC
      f2 xv[2], dv[2], gv[2], zv[2];
      load4p(&g.x[s], xv);
      load4p(&g.dt[s], dv);
      load4p(&g.dy[s], gv);
      if (gated) load4p(&g.z[s], zv);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        dv[k] = add2(dv[k], bias[k]);
        if (a.softplus) dv[k] = softplus_f2(dv[k]);
        xv[k] = mul2(xv[k], dv[k]);
        if (gated) gv[k] = mul2(gv[k], mul2(zv[k], sigmoid_f2(zv[k])));
        if (!in) dv[k] = xv[k] = gv[k] = dup2(0.f);
      }
      store4p(&sm.dt[s], dv);
      store4p(&sm.u[s], xv);
      store4p(&sm.g[s], gv);
    }
#pragma unroll
    for (int i = 0; i < Sh::NBQ; ++i) {
      const int v = tid + i * kThreads, which = v / (TT * LN), q = v % (TT * LN);
      if (which < 2) {
        float4 w = load4((which ? g.C : g.B) + q * 4);
        if (q / LN >= rows) w = make_float4(0.f, 0.f, 0.f, 0.f);
        float *d = (which ? sm.C : sm.B) + q / LN * Sh::NP + q % LN * 2;
        *reinterpret_cast<float2 *>(d) = make_float2(w.x, w.y);
        *reinterpret_cast<float2 *>(d + 2 * LN) = make_float2(w.z, w.w);
      }
    }
  };

  // this thread's channel pair and states
  const int c0 = warp * Sh::CPW + lc * 2, n0 = sl * 4;
  float *part = sm.part[warp];
  const bool cin = c0 < nch;  // pairs: widths are multiples of 8
  const int64_t en = (int64_t)(e0 + c0) * N + n0;            // within [E][N]
  const int64_t ben = (int64_t)b * a.E * N + en;             // within [B][E][N]
  const int64_t pen = ((int64_t)b * S + seg) * a.E * N + en;  // within the records
  auto load_pair = [&](const float *p, f2 (&v)[4]) {
    float4 lo = make_float4(0.f, 0.f, 0.f, 0.f), hi = lo;
    if (p && cin) {
      lo = *reinterpret_cast<const float4 *>(p);
      hi = *reinterpret_cast<const float4 *>(p + N);
    }
    v[0] = pack2(lo.x, hi.x);
    v[1] = pack2(lo.y, hi.y);
    v[2] = pack2(lo.z, hi.z);
    v[3] = pack2(lo.w, hi.w);
  };
  auto store_pair = [&](float *p, const f2 (&v)[4]) {
    if (!cin) return;
    const float2 q0 = unpack2(v[0]), q1 = unpack2(v[1]), q2 = unpack2(v[2]), q3 = unpack2(v[3]);
    *reinterpret_cast<float4 *>(p) = make_float4(q0.x, q1.x, q2.x, q3.x);
    *reinterpret_cast<float4 *>(p + N) = make_float4(q0.y, q1.y, q2.y, q3.y);
  };
  f2 A[4], hin[4], gc[4], dA[4];
  load_pair(a.A + en, A);
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const float2 q = unpack2(mul2(A[n], dup2(kLog2e)));
    A[n] = pack2(finite_rate(q.x), finite_rate(q.y));
  }
  wait_for_previous();
  load_pair(S > 1 ? rec.s.h + pen : a.h0 ? a.h0 + ben : nullptr, hin);
  load_pair(S > 1 ? rec.s.g + pen : gr.dhN ? gr.dhN + ben : nullptr, gc);
#pragma unroll
  for (int n = 0; n < 4; ++n) dA[n] = dup2(0.f);
  // The checkpoint in front of token group k of the part (k > 0), asked for
  // one group ahead.  In shared memory where there is room: loads into
  // registers are put off to their use for want of registers, and each waits
  // for memory there (B2 L4096 E2048, bf16: 401 us against 394 with 16 states,
  // 263 against 257 with 8).
  auto ck_place = [&](int k) {
    return (((int64_t)b * S + seg) * (tokens / kSub - 1) + k - 1) * a.E + e0 + c0;
  };
  f2 ck[4], cksd = dup2(0.f);
  auto ask_ck = [&](int k) {
    const int64_t rc = ck_place(k);
    if constexpr (Sh::CKS) {
      copy16_async(&sm.ck[0][tid * 4], rec.s.ck + rc * N + n0, cin);
      copy16_async(&sm.ck[1][tid * 4], rec.s.ck + (rc + 1) * N + n0, cin);
      copy8_async(&sm.ckdt[tid * 2], rec.s.ckdt + rc, cin);
      copies_commit();
    } else {
      load_pair(rec.s.ck + rc * N + n0, ck);
      cksd = cin ? load_f2(rec.s.ckdt + rc) : dup2(0.f);
    }
  };
  auto get_ck = [&] {
    if constexpr (Sh::CKS) {
      copies_wait<0>();
      const float4 lo = *reinterpret_cast<const float4 *>(&sm.ck[0][tid * 4]);
      const float4 hi = *reinterpret_cast<const float4 *>(&sm.ck[1][tid * 4]);
      ck[0] = pack2(lo.x, hi.x);
      ck[1] = pack2(lo.y, hi.y);
      ck[2] = pack2(lo.z, hi.z);
      ck[3] = pack2(lo.w, hi.w);
      cksd = load_f2(&sm.ckdt[tid * 2]);
    }
  };

  auto tok2 = [&](const float *arr, int t) {
    return load_f2(&arr[t * CT + c0]);
  };
  // this thread's four states of B or C, each twice
  auto shared4 = [&](const float *arr, int t, f2 (&v)[4]) {
    const float *p = arr + t * Sh::NP + 2 * sl;
    const float2 lo = *reinterpret_cast<const float2 *>(p);
    const float2 hi = *reinterpret_cast<const float2 *>(p + 2 * LN);
    v[0] = dup2(lo.x);
    v[1] = dup2(lo.y);
    v[2] = dup2(hi.x);
    v[3] = dup2(hi.y);
  };

  int grp8 = (t1 - t0 + kSub - 1) / kSub - 1;  // token group of the part, from the last
  if (grp8 > 0) ask_ck(grp8);
  for (int q = ntiles - 1; q >= 0; --q) {
    const int tb = t0 + q * TT, turn = ntiles - 1 - q, st = turn & 1;
    // a wait that gives up ends the CTA; the next tile's copies are only
    // issued after this one, so none is in flight but the one that failed
    if (!tc::mbar_wait(&sm.full[st], (turn >> 1) & 1, &sm.abort, timeouts)) {
      tc::mbar_wait_drain(&sm.full[st], (turn >> 1) & 1);
      sm.abort = 1;
    }
    convert(st, min(TT, t1 - tb));
    __syncthreads();
    if (sm.abort) {
      if constexpr (Sh::CKS) copies_wait<0>();
      return;
    }
    // the other stage was last read before this barrier
    if (q > 0) issue(tb - TT, st ^ 1);
    float *bc = rec.bc + (((int64_t)b * tiles + tile) * a.L + tb) * (2 * N);
    for (int sub = (min(TT, t1 - tb) + kSub - 1) / kSub - 1; sub >= 0; --sub, --grp8) {
      if (grp8 > 0) get_ck();
      f2 hs[kSub + 1][4];  // hs[j]: the state in front of token j of the group
#pragma unroll
      for (int n = 0; n < 4; ++n)
        hs[0][n] = grp8 > 0 ? fma2(ex2_2(mul2(cksd, A[n])), hin[n], ck[n]) : hin[n];
      if constexpr (!Sh::CKS) {
        if (grp8 > 1) ask_ck(grp8 - 1);
      }
#pragma unroll
      for (int j = 0; j < kSub; ++j) {
        const int t = sub * kSub + j;
        const f2 d2 = tok2(sm.dt, t), u2 = tok2(sm.u, t);
        f2 bn[4];
        shared4(sm.B, t, bn);
#pragma unroll
        for (int n = 0; n < 4; ++n)
          hs[j + 1][n] = fma2(ex2_2(mul2(d2, A[n])), hs[j][n], mul2(u2, bn[n]));
      }
      if constexpr (Sh::CKS) {
        __syncwarp();  // this group's has been read
        if (grp8 > 1) ask_ck(grp8 - 1);
      }
#pragma unroll
      for (int j2 = kSub - 2; j2 >= 0; j2 -= 2) {  // tokens j2 + 1, then j2
        f2 sums[2][3];  // du, sum_n w A, y over this thread's states
#pragma unroll
        for (int i = 1; i >= 0; --i) {
          const int j = j2 + i, t = sub * kSub + j;
          const f2 d2 = tok2(sm.dt, t), u2 = tok2(sm.u, t), g2 = tok2(sm.g, t);
          f2 bn[4], cn[4];
          shared4(sm.B, t, bn);
          shared4(sm.C, t, cn);
          float r[8];  // dB, dC of this thread's states, over its channel pair
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const f2 g = fma2(cn[n], g2, gc[n]);
            r[n] = sum2(mul2(g, u2));
            r[4 + n] = sum2(mul2(hs[j + 1][n], g2));
            sums[i][0] = n ? fma2(g, bn[n], sums[i][0]) : mul2(g, bn[n]);
            sums[i][2] = n ? fma2(hs[j + 1][n], cn[n], sums[i][2]) : mul2(hs[j + 1][n], cn[n]);
            gc[n] = mul2(g, ex2_2(mul2(d2, A[n])));
            const f2 w = mul2(gc[n], hs[j][n]);
            sums[i][1] = n ? fma2(w, A[n], sums[i][1]) : mul2(w, A[n]);
            dA[n] = fma2(w, d2, dA[n]);
          }
          // over the warp's channels: through shared memory, several tokens at
          // a time (shuffles and their selects took 29 instructions a token,
          // this takes 10), or with two lanes to a state in one exchange
          if constexpr (Sh::LC > 2) {
            float *pd = part + (j % Sh::BT) * 256 + lc * 2 * N;
            const int flip = Sh::flip(lc);
            *reinterpret_cast<float4 *>(pd + (n0 ^ flip)) = make_float4(r[0], r[1], r[2], r[3]);
            *reinterpret_cast<float4 *>(pd + ((N + n0) ^ flip)) = make_float4(r[4], r[5], r[6], r[7]);
            if (j % Sh::BT == 0) {
              constexpr int V = Sh::BT * N / 16, VV = V < 4 ? V : 4;  // sums per lane, and at once
              __syncwarp();
#pragma unroll
              for (int q = 0; q < V / VV; ++q) {
                const int k = (q * 32 + lane) * VV, tk = k / (2 * N), o = k % (2 * N);
                const float *ps = part + tk * 256;
                float s[VV];
#pragma unroll
                for (int c = 0; c < Sh::LC; ++c) add_vec<VV>(s, ps + c * 2 * N + (o ^ Sh::flip(c)), c == 0);
                store_vec<VV>(&sm.red[sub & 1][warp][j + tk][o], s);
              }
              __syncwarp();
            }
          } else {
            const bool hi = lane & LN;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float keep = hi ? r[4 + k] : r[k], send = hi ? r[k] : r[4 + k];
              r[k] = keep + __shfl_xor_sync(0xffffffffu, send, LN);
            }
            *reinterpret_cast<float4 *>(&sm.red[sub & 1][warp][j][(hi ? N : 0) + n0]) =
                make_float4(r[0], r[1], r[2], r[3]);
          }
        }
        // over the states: lane bit 0 takes one of the two tokens, bit 1 one
        // channel of the pair
        const bool b0 = lane & 1;
        const int s = (sub * kSub + j2 + (b0 ? 1 : 0)) * CT + c0;
        float2 v[3];
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          const float2 keep = unpack2(b0 ? sums[1][k] : sums[0][k]);
          const float2 send = unpack2(b0 ? sums[0][k] : sums[1][k]);
          v[k].x = keep.x + __shfl_xor_sync(0xffffffffu, send.x, 1);
          v[k].y = keep.y + __shfl_xor_sync(0xffffffffu, send.y, 1);
        }
        // the shuffles: every lane has read these tokens' inputs
        __syncwarp();
        if constexpr (LN == 2) {
          *reinterpret_cast<float2 *>(&sm.u[s]) = v[0];
          *reinterpret_cast<float2 *>(&sm.dt[s]) = v[1];
          *reinterpret_cast<float2 *>(&sm.g[s]) = v[2];
        } else {
          const bool b1 = lane & 2;
          float w[3];
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            w[k] = (b1 ? v[k].y : v[k].x) + __shfl_xor_sync(0xffffffffu, b1 ? v[k].x : v[k].y, 2);
#pragma unroll
            for (int o = 4; o < LN; o <<= 1) w[k] += __shfl_xor_sync(0xffffffffu, w[k], o);
          }
          if (sl < 4) {
            const int c = b1 ? 1 : 0;
            sm.u[s + c] = w[0];
            sm.dt[s + c] = w[1];
            sm.g[s + c] = w[2];
          }
        }
      }
      if (!kOnce || sub == 0) {
        // kOnce: `red` holds the tile, and the barrier after the next staging
        // is in front of its next use.  Otherwise the other half of `red` is
        // written before this half is again, with this barrier in between.
        __syncthreads();
        const int subs = kOnce ? (min(TT, t1 - tb) + kSub - 1) / kSub : 1;
        for (int i = tid; i < subs * kSub * 2 * N; i += kThreads) {
          const int s1 = sub + i / (kSub * 2 * N), j = i % (kSub * 2 * N);
          if (tb + s1 * kSub + j / (2 * N) < t1) {
            const float *p = &sm.red[s1 & 1][0][0][0] + j;
            float s = p[0];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) s += p[w * kSub * 2 * N];
            bc[(int64_t)sub * kSub * 2 * N + i] = s;
          }
        }
      }
    }

    // the tile's per-token gradients, and its share of the column sums
    const MainStage<T, N> &sg = sm.stage[st];
    f2 dskip[2], bias[2], sD[2], sb[2];
    load4p(&sm.skip[qcol], dskip);
    load4p(&sm.bias[qcol], bias);
    load4p(&sm.cols[0][tid * 4], sD);
    load4p(&sm.cols[1][tid * 4], sb);
#pragma unroll
    for (int i = 0; i < Sh::NQ; ++i) {
      const int row = qrow + i * Sh::ROWS, s = row * CT + qcol, t = tb + row;
      if (qin && t < t1) {
        const int64_t o = ((int64_t)b * a.L + t) * a.E + e0 + qcol;
        f2 du[2], dd[2], yv[2], xv[2], dv[2], gv[2], zv[2];
        load4p(&sg.x[s], xv);
        load4p(&sg.dt[s], dv);
        load4p(&sg.dy[s], gv);
        if (gated) load4p(&sg.z[s], zv);
        load4p(&sm.u[s], du);
        load4p(&sm.dt[s], dd);
        load4p(&sm.g[s], yv);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          f2 g = gv[k];
          if (gated) {
            const f2 act = sigmoid_f2(zv[k]);
            // silu'(z) = s (1 + z (1 - s))
            const f2 slope = mul2(act, fma2(zv[k], fma2(act, dup2(-1.f), dup2(1.f)), dup2(1.f)));
            yv[k] = mul2(mul2(g, fma2(dskip[k], xv[k], yv[k])), slope);
            g = mul2(g, mul2(zv[k], act));
          }
          const f2 v = add2(dv[k], bias[k]);
          const f2 step = a.softplus ? softplus_f2(v) : v;
          dd[k] = fma2(du[k], xv[k], mul2(dd[k], dup2(kLn2)));
          if (a.softplus) dd[k] = mul2(dd[k], sigmoid_f2(v));
          du[k] = fma2(du[k], step, mul2(dskip[k], g));
          sD[k] = fma2(g, xv[k], sD[k]);
          sb[k] = add2(sb[k], dd[k]);
        }
        if (gated) store4p(static_cast<T *>(gr.dz) + o, yv);
        store4p(static_cast<T *>(gr.dx) + o, du);
        store4p(static_cast<T *>(gr.ddt) + o, dd);
      }
    }
    store4p(&sm.cols[0][tid * 4], sD);
    store4p(&sm.cols[1][tid * 4], sb);
    // the next tile's staging writes only what this thread itself has read
    // here, and B and C, which were last read before the barrier above
  }
  store_pair(rec.dA + pen, dA);
  if (seg == 0 && gr.dh0) store_pair(gr.dh0 + ben, gc);
  __syncthreads();
  float *cols = rec.cols + ((int64_t)b * S + seg) * 2 * a.E + e0;
  for (int i = tid; i < 2 * CT; i += kThreads) {
    if (i % CT < nch) {
      const float *p = sm.cols[i / CT] + i % CT;  // [rows of threads][CT]
      float s = 0.f;
      for (int r = 0; r < Sh::ROWS; ++r) s += p[r * CT];
      cols[(i < CT ? 0 : a.E) + i % CT] = s;
    }
  }
}

// -------------------------------------------------------------------- sums

struct SumBlocks {
  int64_t bc, dA;  // blocks of each kind, in this order; the rest are dD and d(dt_bias)
};

// All the sums in one launch, so that they share the machine: a block adds
// either four values of dB or dC per thread over a group's channel tiles, or
// 128 columns of dA, or of dD and d(dt_bias), over the parts.
template <typename T>
__global__ void __launch_bounds__(256)
    scan_bwd_sum_kernel(const __grid_constant__ ScanArgs a, const __grid_constant__ ScanGrads g,
                        const __grid_constant__ BwdRecords rec, int S, int gtiles, SumBlocks nb) {
  __shared__ float4 sh[kWideSlices][kWideVecs];
  wait_for_previous();
  const int64_t block = blockIdx.x;
  if (block >= nb.bc + nb.dA) {
    column_sum_wide(rec.cols, a.B * S, 2 * (int64_t)a.E, g.dD, a.E, g.ddt_bias, block - nb.bc - nb.dA, sh);
    return;
  }
  if (block >= nb.bc) {
    const int64_t C = (int64_t)a.E * a.N;
    column_sum_wide(rec.dA, a.B * S, C, g.dA, C, nullptr, block - nb.bc, sh);
    return;
  }
  const int N = a.N;
  const int64_t per = (int64_t)a.L * 2 * N;
  const int64_t i = (block * 256 + threadIdx.x) * 4;
  if (i >= (int64_t)a.B * a.G * per) return;
  const int64_t bg = i / per, tk = i - bg * per;
  const float *p = rec.bc + bg * gtiles * per + tk;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int k = 0; k < gtiles; ++k) {
    const float4 v = *reinterpret_cast<const float4 *>(p + k * per);
    s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
  }
  const int64_t t = tk / (2 * N);
  const int k = static_cast<int>(tk - t * 2 * N);
  const int64_t b = bg / a.G, gi = bg - b * a.G;
  const int64_t o = ((b * a.L + t) * a.G + gi) * N + (k < N ? k : k - N);
  store4(static_cast<T *>(k < N ? g.dBm : g.dCm) + o, s);
}

int bwd_tiles(int E, int N, int G) {
  const int CT = 1024 / N;
  return G * ((E / G + CT - 1) / CT);
}

// Tokens per part.  With 8 states shorter ones, the shortest where they are
// few (bf16, B2 L4096 E2048: 263 us at 48, 272 at 32; B1 L512 E2048: 32 us at
// 32, 42 at 48).  With 16, 32 tokens differ from 64 by 5% either way in small
// calls, and 96 are worse there (B1 L512 E2048: 62 us against 46).
int bwd_part_tokens(int B, int L, int E, int N, int G) {
  if (N > 8) return kPart;
  return (int64_t)B * ((L + 47) / 48) * bwd_tiles(E, N, G) < kSMs * 3 ? 32 : 48;
}

// The workspace: floats of each record.
struct BwdSizes {
  size_t h, g, dt, ck, ckdt, cols, bc;
  int S, part;
};
BwdSizes bwd_sizes(int B, int L, int E, int N, int G) {
  BwdSizes z;
  const int pt = z.part = bwd_part_tokens(B, L, E, N, G), K = pt / kScanCheckpoint - 1;
  z.S = L > pt ? (L + pt - 1) / pt : 1;
  const size_t bs = (size_t)B * z.S;
  z.h = bs * E * N;
  z.g = z.h;
  z.dt = bs * E;
  z.ck = L > kScanCheckpoint ? bs * K * E * N : 0;
  z.ckdt = L > kScanCheckpoint ? bs * K * E : 0;
  z.cols = bs * 2 * E;
  z.bc = (size_t)B * bwd_tiles(E, N, G) * L * 2 * N;
  return z;
}

template <typename T, int N>
cudaError_t bwd_typed(const ScanArgs &a, const ScanGrads &g, void *ws, cudaStream_t s) {
  const BwdSizes z = bwd_sizes(a.B, a.L, a.E, N, a.G);
  BwdRecords rec;
  rec.s.h = rec.dA = static_cast<float *>(ws);
  rec.s.g = rec.s.h + z.h;
  rec.s.dt = rec.s.g + z.g;
  rec.s.ck = rec.s.dt + z.dt;
  rec.s.ckdt = rec.s.ck + z.ck;
  rec.cols = rec.s.ckdt + z.ckdt;
  rec.bc = rec.cols + z.cols;
  rec.part = z.part;
  cudaError_t e;
  // one group of tokens needs neither checkpoints nor records
  if (a.L > kScanCheckpoint) {
    e = launch_selective_local(a, g.dy, rec.s, z.S, z.part, sizeof(T) == 4 ? kF32 : kBF16, s);
    if (e != cudaSuccess) return e;
  }
  if (z.S > 1) {
    const int64_t n = (int64_t)a.B * a.E * N;
    e = launch_dependent(scan_bwd_carry_kernel, (unsigned)((n / 2 + kCarryThreads - 1) / kCarryThreads), 2,
                         kCarryThreads, 0, s, a, g.dhN, rec, z.S);
    if (e != cudaSuccess) return e;
  }
  const int tiles = bwd_tiles(a.E, N, a.G);
  constexpr int smem = sizeof(MainSmem<T, N>);
  static_assert((smem + 1024) * (N <= 16 || (N == 32 && sizeof(T) == 2) ? 3 : 2) <= 228 * 1024, "");
  if ((e = allow_smem(scan_bwd_main_kernel<T, N>, smem)) != cudaSuccess) return e;
  unsigned int *timeouts = wait_timeout_counter();
  if (!timeouts) return cudaErrorUnknown;
  using Sh = MainShape<T, N>;
  ScanMaps maps = {};
  if (!make_scan_maps(&maps, a, g.dy, sizeof(T), Sh::CT, Sh::TT)) return cudaErrorInvalidValue;
  const unsigned ctas = (unsigned)((int64_t)a.B * z.S * tiles);
  if (a.L > kScanCheckpoint) {
    e = launch_dependent(scan_bwd_main_kernel<T, N>, ctas, 1, kThreads, smem, s, a, g, maps, rec, z.S, timeouts);
  } else {  // the kernel before is the caller's
    scan_bwd_main_kernel<T, N><<<ctas, kThreads, smem, s>>>(a, g, maps, rec, z.S, timeouts);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  SumBlocks nb;
  nb.bc = ((int64_t)a.B * a.G * a.L * 2 * N / 4 + 255) / 256;
  nb.dA = ((int64_t)a.E * N + kWideCols - 1) / kWideCols;
  const int64_t cols = g.dD || g.ddt_bias ? (2 * (int64_t)a.E + kWideCols - 1) / kWideCols : 0;
  return launch_dependent(scan_bwd_sum_kernel<T>, (unsigned)(nb.bc + nb.dA + cols), 1, 256, 0, s, a, g, rec, z.S,
                          tiles / a.G, nb);
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
  return sizeof(float) * (z.h + z.g + z.dt + z.ck + z.ckdt + z.cols + z.bc);
}

cudaError_t launch_selective_backward(const ScanArgs &a, const ScanGrads &g, Dtype dt, void *ws,
                                      cudaStream_t s) {
  return dt == kF32 ? bwd_states<float>(a, g, ws, s) : bwd_states<__nv_bfloat16>(a, g, ws, s);
}

}  // namespace linattn
