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
// the instructions issued, not memory: per warp and token (512 states) 16
// exponentials (4 cycles each), 32 packed operations (2 cycles each) and what
// feeds them.  Measured (B2 L4096 E2048 N16 in bf16, 132 us): 57% of the issue
// slots and about half of either pipe are used, so beyond the count of
// instructions it is waiting, for results and for shared memory, at the 16
// warps per SM that the registers allow.  Hence (times of alternatives are
// those at which each choice was made):
//   - a thread owns 4 channels x 4 states in registers: per token it reads one
//     16-byte vector of dt, of u = dt x, and two of B and of C (each value
//     twice) from shared memory for 16 state updates, done as packed pairs of
//     channels; the next token's operands are read before this token's are
//     used.  The backward pass's mode, which has more arithmetic per operand,
//     reads B and C once each as 8-byte pairs instead and doubles them in
//     registers: half the shared-memory wavefronts for 16 moves (441 against
//     447 us for the whole backward pass at B2 L4096 E2048 N16 in bf16, but
//     161 against 136 us for the forward pass);
//   - the sum over states crosses N/4 lanes: exchanges that halve a lane's
//     channels leave two parts of y, stored to shared memory, and the threads
//     that write y add them (139 us for the forward pass; four parts, without
//     an exchange at 16 states, cost an SM one of its four CTAs: 157 us);
//   - softplus, the D term and the gate are applied once per (channel, token)
//     when a tile of tokens is staged and when it is stored.
// A tile's inputs come by TMA, one box per tensor, while the previous tile
// computes (copies issued per thread cost a shared-memory wavefront per lane,
// which made them the largest load on that pipe; bulk copies per row kept the
// issuing warp behind the others).
//
// Few channels leave SMs idle, so the tokens split into S parts: the state
// pass leaves every part but the last its end state from zero and its sum of
// dt (the part's decay is exp(A sum dt): no product is kept), and the output
// pass folds the records before its part in front of its own scan.  The parts
// of a ragged batch are laid out over its sequences on the device, which knows
// the lengths.
#include "dependent.cuh"
#include "kernels.h"
#include "mixer_common.cuh"
#include "scan_maps.cuh"

namespace linattn {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxParts = 128;
// A tile's tokens are walked in groups of so many, which a part's last tile
// may leave out (B2 L4096 E2048 N16 in bf16, parts of 216 tokens instead of
// 224: 128.4 us against 131.4; without parts it costs 0.6%).
constexpr int kSteps = 8;
// As many CTAs run whole sequences: 256 of them (B8 L2048 E4096 N16, bf16) take
// 392 us and in parts 467, 192 of them 391 and 350.
constexpr int kWhole = 224;
constexpr int kCheckpoint = kScanCheckpoint;
constexpr int kSlots = 2;    // parts of y, at most

// The passes over the tokens: a part's end state; y; or, for the backward
// pass, a part's end state with checkpoints and its adjoint contribution.
enum { kStates = 0, kOut = 1, kLocal = 2 };

template <typename T, int N, int MODE>
struct Shape {
  // (token, channel) pairs of a tile, at most.  The local pass has one more
  // input to hold: with 2048 pairs one of its four CTAs less fits an SM (472 us
  // for the backward pass against 461).  The others gain by the larger tile (144
  // against 135 us in bf16, 115 against 107 us in fp32).
  static constexpr int kTile = MODE == kLocal ? 1024 : 2048;
  static constexpr int LN = N / 4;         // lanes that share a channel's states
  static constexpr int LC = 32 / LN;       // channel quads per warp
  static constexpr int CPW = LC * 4;       // channels per warp
  static constexpr int CT = CPW * kWarps;  // channels per CTA
  static constexpr int TT = kTile / CT < 8 ? 8 : kTile / CT < 32 ? kTile / CT : 32;  // tokens per tile
  static constexpr int TILE = TT * CT;     // (token, channel) pairs per tile
  static constexpr int QC = CT / 4;        // channel quads per token
  static constexpr int NQ = TILE / 4 / kThreads;  // quads staged per thread
  static constexpr int SLOTS = LN < kSlots ? LN : kSlots;  // parts of y in shared memory
  // the parts of one quad fall into different banks
  static constexpr int SLOT = TILE + 32 / SLOTS;
  static constexpr int BQ = TT * N / 4;    // quads of B (and of C) per tile
  static constexpr int NBQ = (2 * BQ + kThreads - 1) / kThreads;
};

// A tile as loaded.
template <typename T, int N, int MODE>
struct Stage {
  using S = Shape<T, N, MODE>;
  alignas(128) T x[S::TILE];
  alignas(128) T dt[S::TILE];
  alignas(128) T B[S::TT * N];
  alignas(128) T C[MODE != kStates ? S::TT * N : 1];
  alignas(128) T z[MODE != kStates ? S::TILE : 1];
  alignas(128) T dy[MODE == kLocal ? S::TILE : 1];
};

template <typename T, int N, int MODE>
struct Smem {
  using S = Shape<T, N, MODE>;
  Stage<T, N, MODE> stage[2];
  alignas(16) float dt[S::TILE];
  // dt x; in the output pass y's first parts take its place, then the others
  float u[(MODE == kOut ? S::SLOTS : 1) * S::SLOT];
  alignas(16) float g[MODE == kLocal ? S::TILE : 4];  // dy silu(z)
  // [token][N][2], each value twice; kLocal: [token][N], states 4 l and 4 l + 1
  // at 2 l, 4 l + 2 and 4 l + 3 at 2 LN + 2 l
  float B[S::TT * N * (MODE == kLocal ? 1 : 2)];
  alignas(16) float C[MODE == kLocal ? S::TT * N : MODE == kOut ? S::TT * N * 2 : 4];
  uint64_t full[2];
  int abort;
};

// Stores a channel quad's y of one token from its LN state lanes as SLOTS
// parts, after an exchange over lane bits that halves the channels of a lane
// (or, with one left, adds) until that many parts are left.
template <int LN, int SLOTS, int SLOT>
__device__ __forceinline__ void store_parts(float *y, int sl, f2 y01, f2 y23) {
  constexpr unsigned all = 0xffffffffu;
  if constexpr (LN == SLOTS) {
    *reinterpret_cast<ulonglong2 *>(y + sl * SLOT) = make_ulonglong2(y01.v, y23.v);
  } else {
    const bool hi = sl & 1;
    const float2 a = unpack2(hi ? y23 : y01), b = unpack2(hi ? y01 : y23);
    const float k0 = a.x + __shfl_xor_sync(all, b.x, 1), k1 = a.y + __shfl_xor_sync(all, b.y, 1);
    if constexpr (LN == 2 * SLOTS) {
      *reinterpret_cast<float2 *>(y + (sl >> 1) * SLOT + 2 * (sl & 1)) = make_float2(k0, k1);
    } else {
      const bool h2 = sl & 2;
      float k = (h2 ? k1 : k0) + __shfl_xor_sync(all, h2 ? k0 : k1, 2);
      int slot = sl >> 2;
      if constexpr (LN == 8 * SLOTS) {
        k += __shfl_xor_sync(all, k, 4);
        slot = sl >> 3;
      }
      static_assert(LN <= 8 * SLOTS, "");
      y[slot * SLOT + 2 * (sl & 1) + ((sl >> 1) & 1)] = k;
    }
  }
}

// A part of a sequence, and the record of the sequence's first part.
struct Place {
  int b, part, len, part_len, first;
  bool last;
};

// The place of `slot` among the parts of a ragged batch, which share one
// length: the shortest (of four tried, and one that always fits) at which the
// parts of all sequences, one at least for each, fit the slots.  Every warp
// works it out.  With a part length from L alone, slots went empty or a second
// wave was needed.  False for a slot without a part.
__device__ __forceinline__ bool find_place(const int *__restrict__ lens, int B, int L, int slots,
                                           int least, int slot, Place *p) {
  const int lane = threadIdx.x & 31;
  auto clamped = [&](int b) { return min(max(lens[b], 0), L); };
  auto up = [](int n) { return (n + kSteps - 1) / kSteps * kSteps; };
  int total = 0;  // B L < 2^31
  for (int b = lane; b < B; b += 32) total += clamped(b);
  total = __reduce_add_sync(0xffffffffu, total);
  const int lo = max(least, up((total + slots - 1) / slots));
  const int hi = max(lo, up((total + slots - B - 1) / (slots - B)));
  int len = hi;
  for (int k = 0; k < 4; ++k) {
    const int l = up(lo + (hi - lo) / 4 * k);
    int n = 0;
    for (int b = lane; b < B; b += 32) n += max(1, (clamped(b) + l - 1) / l);
    if (__reduce_add_sync(0xffffffffu, n) <= slots) {
      len = l;
      break;
    }
  }
  int before = 0;  // parts of the sequences before
  for (int b0 = 0; b0 < B; b0 += 32) {
    const int b = b0 + lane;
    const int own = b < B ? max(1, (clamped(b) + len - 1) / len) : 0;
    int sum = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    const unsigned here = __ballot_sync(0xffffffffu, slot < before + sum);
    if (here) {
      const int src = __ffs(here) - 1, q = __shfl_sync(0xffffffffu, own, src);
      p->first = before + __shfl_sync(0xffffffffu, sum, src) - q;
      p->b = b0 + src;
      p->part = slot - p->first;
      p->last = p->part == q - 1;
      p->len = clamped(p->b);
      p->part_len = len;
      return true;
    }
    before += __shfl_sync(0xffffffffu, sum, 31);
  }
  return false;
}

// Parts: the last has no record in the state pass; kLocal runs them all.
template <typename T, int N, int MODE>
__global__ void __launch_bounds__(kThreads, 4)
    scan_kernel(const __grid_constant__ ScanArgs a, const __grid_constant__ ScanMaps maps,
                const __grid_constant__ ScanRecords rec, int S, int part_len,
                unsigned int *timeouts) {
  constexpr bool OUT = MODE == kOut, LOCAL = MODE == kLocal;
  using Sh = Shape<T, N, MODE>;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  Smem<T, N, MODE> &sm = *reinterpret_cast<Smem<T, N, MODE> *>(smem_raw);

  const int Eg = a.E / a.G;  // channels per group
  const int gtiles = (Eg + Sh::CT - 1) / Sh::CT, tiles = gtiles * a.G;
  const int tile = blockIdx.x % tiles;
  Place at;
  if (!LOCAL && a.lens && S > 1) {
    if (!find_place(a.lens, a.B, a.L, a.B * S, part_len, blockIdx.x / tiles, &at)) return;
    if (MODE == kStates && at.last) return;
  } else {
    const int nparts = MODE == kStates ? S - 1 : S;
    at.part = (blockIdx.x / tiles) % nparts;
    at.b = blockIdx.x / tiles / nparts;
    at.first = at.b * (LOCAL ? S : S - 1);
    at.len = a.lens ? min(max(a.lens[at.b], 0), a.L) : a.L;
    at.part_len = part_len;
    at.last = at.part == S - 1;
  }
  const int part = at.part, b = at.b;
  if (threadIdx.x == 0) {
    tc::mbar_init(&sm.full[0], 1);
    tc::mbar_init(&sm.full[1], 1);
    tc::mbar_init_fence();
    sm.abort = 0;
  }
  __syncthreads();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int sl = lane & (Sh::LN - 1), lc = lane / Sh::LN;
  const int grp = tile / gtiles;
  const int cg = (tile % gtiles) * Sh::CT;      // first channel within the group
  const int e0 = grp * Eg + cg;                 // first channel
  const int nch = min(Sh::CT, Eg - cg);         // channels of this tile
  const int t0 = part * at.part_len, t1 = min(LOCAL ? a.L : at.len, t0 + at.part_len);

  const bool gated = MODE != kStates && a.z;
  T *y = OUT ? static_cast<T *>(a.y) + (int64_t)b * a.L * a.E + e0 : nullptr;

  // The tile at token tb.  A box may reach behind the part's end, the
  // sequence's or the group's: those rows are cleared when staged, those
  // channels belong to lanes that store nothing.
  auto issue = [&](int tb, int st) {
    if (tid != 0) return;
    Stage<T, N, MODE> &g = sm.stage[st];
    uint64_t *bar = &sm.full[st];
    constexpr uint32_t rows = Sh::TILE * sizeof(T), bc = Sh::TT * N * sizeof(T);
    tc::mbar_arrive_expect_tx(
        bar, (2 + (gated ? 1 : 0) + (LOCAL ? 1 : 0)) * rows + (MODE != kStates ? 2 : 1) * bc);
    tc::tma_load_3d(g.x, &maps.x, e0, tb, b, bar);
    tc::tma_load_3d(g.dt, &maps.dt, e0, tb, b, bar);
    tc::tma_load_3d(g.B, &maps.B, grp * N, tb, b, bar);
    if constexpr (MODE != kStates) {
      tc::tma_load_3d(g.C, &maps.C, grp * N, tb, b, bar);
      if (gated) tc::tma_load_3d(g.z, &maps.z, e0, tb, b, bar);
    }
    if constexpr (LOCAL) tc::tma_load_3d(g.dy, &maps.dy, e0, tb, b, bar);
  };
  if (t0 < t1) issue(t0, 0);

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
      av[c][0] = finite_rate(q.x * kLog2e); av[c][1] = finite_rate(q.y * kLog2e);
      av[c][2] = finite_rate(q.z * kLog2e); av[c][3] = finite_rate(q.w * kLog2e);
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
    // the state before this part: the records of the parts before it, four
    // loaded at a time (one at a time each costs a memory latency)
    constexpr int kFold = 4;
    if (part > 0) wait_for_previous();
    for (int q0 = 0; q0 < part; q0 += kFold) {
      float4 r[kFold][4], sd[kFold];
#pragma unroll
      for (int k = 0; k < kFold; ++k) {
        const int64_t rc = (int64_t)(at.first + q0 + k) * a.E + e0 + c0;
        const bool in = q0 + k < part && c0 < nch;  // widths are multiples of 8
        sd[k] = in ? *reinterpret_cast<const float4 *>(rec.dt + rc) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int c = 0; c < 4; ++c)
          r[k][c] = in ? *reinterpret_cast<const float4 *>(rec.h + (rc + c) * N + n0)
                       : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int k = 0; k < kFold; ++k) {  // a record of zeros leaves h as it is
        const f2 s2[2] = {pack2(sd[k].x, sd[k].y), pack2(sd[k].z, sd[k].w)};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float4 lo = r[k][2 * c], hi = r[k][2 * c + 1];
          h[c][0] = fma2(ex2_2(mul2(s2[c], A[c][0])), h[c][0], pack2(lo.x, hi.x));
          h[c][1] = fma2(ex2_2(mul2(s2[c], A[c][1])), h[c][1], pack2(lo.y, hi.y));
          h[c][2] = fma2(ex2_2(mul2(s2[c], A[c][2])), h[c][2], pack2(lo.z, hi.z));
          h[c][3] = fma2(ex2_2(mul2(s2[c], A[c][3])), h[c][3], pack2(lo.w, hi.w));
        }
      }
    }
  }
  f2 dtsum[2] = {dup2(0.f), dup2(0.f)};
  // the product of the part's decays so far, and its adjoint contribution
  f2 P[2][4], adj[2][4];
  if constexpr (LOCAL)
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        P[c][n] = dup2(1.f);
        adj[c][n] = dup2(0.f);
      }
  // v of this thread's channels and states to p, its first channel's place
  auto store_states = [&](float *p, const f2 (&v)[2][4]) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const float2 q0 = unpack2(v[c][0]), q1 = unpack2(v[c][1]), q2 = unpack2(v[c][2]),
                   q3 = unpack2(v[c][3]);
      if (c0 + 2 * c < nch) {  // widths are multiples of 8
        *reinterpret_cast<float4 *>(p + 2 * c * N) = make_float4(q0.x, q1.x, q2.x, q3.x);
        *reinterpret_cast<float4 *>(p + (2 * c + 1) * N) = make_float4(q0.y, q1.y, q2.y, q3.y);
      }
    }
  };
  auto store_dtsum = [&](float *p) {
    if (sl == 0 && c0 < nch) {
      const float2 q = unpack2(dtsum[0]), r = unpack2(dtsum[1]);
      *reinterpret_cast<float4 *>(p) = make_float4(q.x, q.y, r.x, r.y);
    }
  };

  // per-channel parameters of the staged quads (one column per thread:
  // kThreads is a multiple of QC)
  const int qcol = (tid % Sh::QC) * 4, qrow = tid / Sh::QC;
  constexpr int kRowStep = kThreads / Sh::QC;
  const bool qin = qcol < nch;
  f2 bias[2] = {dup2(0.f), dup2(0.f)}, dskip[2] = {dup2(0.f), dup2(0.f)};
  if (qin && a.dt_bias) load4p(a.dt_bias + e0 + qcol, bias);
  if (OUT && qin && a.D) load4p(a.D + e0 + qcol, dskip);

  struct Operands {
    f2 d[2], u[2], g[2], b[4], c[4];
  };
  auto fetch = [&](int t) {
    Operands o;
    const int s = t * Sh::CT + c0;
    const ulonglong2 dq = *reinterpret_cast<const ulonglong2 *>(&sm.dt[s]);
    const ulonglong2 uq = *reinterpret_cast<const ulonglong2 *>(&sm.u[s]);
    o.d[0] = {dq.x}; o.d[1] = {dq.y};
    o.u[0] = {uq.x}; o.u[1] = {uq.y};
    if constexpr (LOCAL) {
      const ulonglong2 gq = *reinterpret_cast<const ulonglong2 *>(&sm.g[s]);
      o.g[0] = {gq.x}; o.g[1] = {gq.y};
    }
    auto shared4 = [&](const float *arr, f2 (&v)[4]) {
      if constexpr (LOCAL) {
        const float *p = arr + t * N + 2 * sl;
        const float2 lo = *reinterpret_cast<const float2 *>(p);
        const float2 hi = *reinterpret_cast<const float2 *>(p + 2 * Sh::LN);
        v[0] = dup2(lo.x); v[1] = dup2(lo.y);
        v[2] = dup2(hi.x); v[3] = dup2(hi.y);
      } else {
        const ulonglong2 *p = reinterpret_cast<const ulonglong2 *>(arr + (t * N + n0) * 2);
        v[0] = {p[0].x}; v[1] = {p[0].y};
        v[2] = {p[1].x}; v[3] = {p[1].y};
      }
    };
    shared4(sm.B, o.b);
    if constexpr (MODE != kStates) shared4(sm.C, o.c);
    return o;
  };

  int turn = 0;
  for (int tb = t0; tb < t1; tb += Sh::TT, ++turn) {
    const int st = turn & 1, rows = min(Sh::TT, t1 - tb);
    const Stage<T, N, MODE> &g = sm.stage[st];
    // a wait that gives up ends the CTA; the next tile's copies are only
    // issued after this one, so none is in flight but the one that failed
    if (!tc::mbar_wait(&sm.full[st], (turn >> 1) & 1, &sm.abort, timeouts)) {
      tc::mbar_wait_drain(&sm.full[st], (turn >> 1) & 1);
      sm.abort = 1;
    }
#pragma unroll
    for (int i = 0; i < Sh::NQ; ++i) {
      const int r = qrow + i * kRowStep, s = r * Sh::CT + qcol;
      f2 xv[2], dv[2];
      load4p(&g.x[s], xv);
      load4p(&g.dt[s], dv);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        dv[k] = add2(dv[k], bias[k]);
        if (a.softplus) dv[k] = softplus_f2(dv[k]);
        xv[k] = mul2(xv[k], dv[k]);
        // rows behind the end hold nothing and leave the state as it is
        if (r >= rows) dv[k] = xv[k] = dup2(0.f);
      }
      store4p(&sm.dt[s], dv);
      store4p(&sm.u[s], xv);
      if constexpr (LOCAL) {
        f2 gv[2], zv[2];
        load4p(&g.dy[s], gv);
        if (gated) load4p(&g.z[s], zv);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (gated) gv[k] = mul2(gv[k], mul2(zv[k], sigmoid_f2(zv[k])));
          if (r >= rows) gv[k] = dup2(0.f);
        }
        store4p(&sm.g[s], gv);
      }
    }
#pragma unroll
    for (int i = 0; i < Sh::NBQ; ++i) {
      const int v = tid + i * kThreads, which = v / Sh::BQ, q = v % Sh::BQ * 4;
      if (which < (MODE != kStates ? 2 : 1)) {
        float4 w = load4((which ? g.C : g.B) + q);
        if (q / N >= rows) w = make_float4(0.f, 0.f, 0.f, 0.f);
        float *d = which ? sm.C : sm.B;
        if constexpr (LOCAL) {
          d += q / N * N + q % N / 2;
          *reinterpret_cast<float2 *>(d) = make_float2(w.x, w.y);
          *reinterpret_cast<float2 *>(d + 2 * Sh::LN) = make_float2(w.z, w.w);
        } else {
          *reinterpret_cast<float4 *>(d + 2 * q) = make_float4(w.x, w.x, w.y, w.y);
          *reinterpret_cast<float4 *>(d + 2 * q + 4) = make_float4(w.z, w.z, w.w, w.w);
        }
      }
    }
    __syncthreads();
    if (sm.abort) return;
    // the other stage was last read before this barrier
    if (tb + Sh::TT < t1) issue(tb + Sh::TT, st ^ 1);
    Operands nxt = fetch(0);
    auto step = [&](int t) {
      const Operands o = nxt;
      nxt = fetch(t + 1 < Sh::TT ? t + 1 : t);
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const f2 e = ex2_2(mul2(o.d[c], A[c][n]));
          h[c][n] = fma2(e, h[c][n], mul2(o.u[c], o.b[n]));
          if constexpr (LOCAL) {
            P[c][n] = mul2(P[c][n], e);
            adj[c][n] = fma2(P[c][n], mul2(o.g[c], o.c[n]), adj[c][n]);
          }
        }
      if constexpr (OUT) {
        f2 y2[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          y2[c] = mul2(h[c][0], o.c[0]);
#pragma unroll
          for (int n = 1; n < 4; ++n) y2[c] = fma2(h[c][n], o.c[n], y2[c]);
        }
        __syncwarp();  // every lane has read u of this token: y takes its place
        store_parts<Sh::LN, Sh::SLOTS, Sh::SLOT>(&sm.u[t * Sh::CT + c0], sl, y2[0], y2[1]);
      } else {
        dtsum[0] = add2(dtsum[0], o.d[0]);
        dtsum[1] = add2(dtsum[1], o.d[1]);
      }
    };
    if constexpr (LOCAL) {
      static_assert(Sh::TT % kCheckpoint == 0, "");
      for (int t8 = 0; t8 < Sh::TT; t8 += kCheckpoint) {
        const int k = (tb - t0 + t8) / kCheckpoint;
        if (k > 0 && tb + t8 < t1) {
          const int64_t rc = (((int64_t)b * S + part) * (part_len / kCheckpoint - 1) + k - 1) * a.E + e0 + c0;
          store_states(rec.ck + rc * N + n0, h);
          store_dtsum(rec.ckdt + rc);
        }
#pragma unroll
        for (int j = 0; j < kCheckpoint; ++j) step(t8 + j);
      }
    } else {
      #pragma unroll 2
      for (int t8 = 0; t8 < Sh::TT; t8 += kSteps) {
        if (t8 && t8 >= rows) break;
#pragma unroll
        for (int j = 0; j < kSteps; ++j) step(t8 + j);
      }
    }
    __syncthreads();
    if constexpr (OUT) {
#pragma unroll
      for (int i = 0; i < Sh::NQ; ++i) {
        const int r = qrow + i * kRowStep, s = r * Sh::CT + qcol;
        if (qin && r < rows) {
          f2 yv[2], xv[2];
          load4p(&sm.u[s], yv);
#pragma unroll
          for (int k = 1; k < Sh::SLOTS; ++k) {
            f2 q[2];
            load4p(&sm.u[k * Sh::SLOT + s], q);
            yv[0] = add2(yv[0], q[0]);
            yv[1] = add2(yv[1], q[1]);
          }
          load4p(&g.x[s], xv);
          yv[0] = fma2(dskip[0], xv[0], yv[0]);
          yv[1] = fma2(dskip[1], xv[1], yv[1]);
          if (gated) {
            f2 zv[2];
            load4p(&g.z[s], zv);
            // silu(z) first: y z may overflow where silu(z) is zero
#pragma unroll
            for (int k = 0; k < 2; ++k) yv[k] = mul2(yv[k], mul2(zv[k], sigmoid_f2(zv[k])));
          }
          store4p(y + (int64_t)(tb + r) * a.E + qcol, yv);
        }
      }
    }
  }

  // the state after this part: the record, or the final state
  if constexpr (OUT) {
    if (at.last && a.hN) store_states(a.hN + ((int64_t)b * a.E + e0 + c0) * N + n0, h);
  } else {
    const int64_t rc = (LOCAL ? (int64_t)b * S + part : at.first + part) * a.E + e0 + c0;
    store_states(rec.h + rc * N + n0, h);
    store_dtsum(rec.dt + rc);
    if constexpr (LOCAL) store_states(rec.g + rc * N + n0, adj);
  }
}

template <typename T, int N, int MODE>
cudaError_t launch_scan(const ScanArgs &a, const void *dy, const ScanRecords &rec, int S,
                        int part_len, cudaStream_t s) {
  using Sh = Shape<T, N, MODE>;
  ScanMaps maps = {};
  if (!make_scan_maps(&maps, a, dy, sizeof(T), Sh::CT, Sh::TT)) return cudaErrorInvalidValue;
  constexpr int smem = sizeof(Smem<T, N, MODE>);
  unsigned int *timeouts = wait_timeout_counter();
  if (!timeouts) return cudaErrorUnknown;
  cudaError_t e = allow_smem(scan_kernel<T, N, MODE>, smem);
  if (e == cudaSuccess) e = most_shared(scan_kernel<T, N, MODE>);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (int64_t)a.G * ((a.E / a.G + Sh::CT - 1) / Sh::CT);
  const int64_t ctas = (int64_t)a.B * (MODE == kStates && !a.lens ? S - 1 : S) * tiles;
  if (MODE == kOut && S > 1)  // behind the state pass
    return launch_dependent(scan_kernel<T, N, MODE>, (unsigned)ctas, 1, kThreads, smem, s, a, maps, rec, S,
                            part_len, timeouts);
  scan_kernel<T, N, MODE><<<(unsigned)ctas, kThreads, smem, s>>>(a, maps, rec, S, part_len, timeouts);
  return cudaGetLastError();
}

// Tokens of a part, at least: kMaxParts of them hold any sequence.
int max_parts_len(int L, int N) {
  const int least = N > 32 ? N : 32, l = (L + kMaxParts - 1) / kMaxParts;
  return l > least ? (l + kSteps - 1) / kSteps * kSteps : least;
}

template <typename T, int N>
cudaError_t scan_typed(const ScanArgs &a, void *ws, int S, cudaStream_t s) {
  // a ragged batch: the shortest part, the rest is decided on the device
  const int part_len = a.lens && S > 1 ? max_parts_len(a.L, N) : selective_part_len(a.L, S);
  ScanRecords rec = {};
  rec.h = static_cast<float *>(ws);
  rec.dt = rec.h + (size_t)a.B * (a.lens ? S : S - 1) * a.E * N;
  if (S > 1) {
    const cudaError_t e = launch_scan<T, N, kStates>(a, nullptr, rec, S, part_len, s);
    if (e != cudaSuccess) return e;
  }
  return launch_scan<T, N, kOut>(a, nullptr, rec, S, part_len, s);
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

template <typename T>
cudaError_t local_states(const ScanArgs &a, const void *dy, const ScanRecords &rec, int S,
                         int part_len, cudaStream_t s) {
  switch (a.N) {
    case 8: return launch_scan<T, 8, kLocal>(a, dy, rec, S, part_len, s);
    case 16: return launch_scan<T, 16, kLocal>(a, dy, rec, S, part_len, s);
    case 32: return launch_scan<T, 32, kLocal>(a, dy, rec, S, part_len, s);
    case 64: return launch_scan<T, 64, kLocal>(a, dy, rec, S, part_len, s);
  }
  return cudaErrorNotSupported;
}

// CTAs of the output pass that an SM holds: four by registers, fewer by
// shared memory.
template <typename T, int N>
constexpr int resident_ctas() {
  constexpr int n = 227 * 1024 / (sizeof(Smem<T, N, kOut>) + 1024);
  return n < 4 ? n : 4;
}
template <typename T>
int resident(int N) {
  return N == 8 ? resident_ctas<T, 8>() : N == 16 ? resident_ctas<T, 16>()
         : N == 32 ? resident_ctas<T, 32>() : resident_ctas<T, 64>();
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
  float4 A = *reinterpret_cast<const float4 *>(a.A + (int64_t)ec * N + sl * 4);
  A = make_float4(finite_rate(A.x), finite_rate(A.y), finite_rate(A.z), finite_rate(A.w));
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
  // two sequences per thread once that still gives every SM eight CTAs (256 x
  // 4096 channels of 16 states in bf16: 28.9 us, four 29.6, on one machine;
  // 29.6 to 31.6 over three)
  if ((int64_t)nx * a.B >= kSMs * 8 * 2) {
    const int ny = (a.B + 1) / 2;
    scan_step_kernel<T, N, 2><<<dim3(nx, ny < kMaxY ? ny : kMaxY), 256, 0, s>>>(a);
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
  const int l = (L + S - 1) / S;
  return (l + kSteps - 1) / kSteps * kSteps;
}

int selective_parts(int B, int L, int E, int N, int G, Dtype dt, bool ragged) {
  const int CT = 2048 / N;  // channels per CTA
  const int64_t ctas = (int64_t)B * G * ((E / G + CT - 1) / CT);
  if (ctas >= kWhole) return 1;
  // one wave of the output pass
  int64_t S = (int64_t)kSMs * (dt == kF32 ? resident<float>(N) : resident<__nv_bfloat16>(N)) /
              (ctas > 0 ? ctas : 1);
  // parts of at least 32 tokens (B1 L512 E2048 N16 in bf16: 17.4 us; 64: 20.3,
  // 128: 32.9), and three of them: two walk as many tokens one after another
  // as one and its state pass (B16 L64 E1024 G4: 11.6 us, with two parts 14.1)
  const int least = N > 32 ? N : 32, most = L / least < kMaxParts ? L / least : kMaxParts;
  if (most < 3) return 1;
  if (S > most) S = most;
  if (S < 2) return 1;
  if (ragged) return static_cast<int>(S);  // parts, on average over the batch
  const int len = selective_part_len(L, static_cast<int>(S));
  return (L + len - 1) / len;  // no part is empty
}

size_t selective_workspace_bytes(int B, int E, int N, int S, bool ragged) {
  return S > 1 ? sizeof(float) * (size_t)B * (ragged ? S : S - 1) * E * (N + 1) : 0;
}

cudaError_t launch_selective(const ScanArgs &a, Dtype dt, void *ws, int S, cudaStream_t s) {
  return dt == kF32 ? scan_states<float>(a, ws, S, s) : scan_states<__nv_bfloat16>(a, ws, S, s);
}

cudaError_t launch_selective_local(const ScanArgs &a, const void *dy, const ScanRecords &rec, int S,
                                   int part_len, Dtype dt, cudaStream_t s) {
  return dt == kF32 ? local_states<float>(a, dy, rec, S, part_len, s)
                    : local_states<__nv_bfloat16>(a, dy, rec, S, part_len, s);
}

cudaError_t launch_selective_step(const ScanArgs &a, Dtype dt, cudaStream_t s) {
  return dt == kF32 ? step_states<float>(a, s) : step_states<__nv_bfloat16>(a, s);
}

}  // namespace linattn
