// Retention on tcgen05 tensor cores: bf16, Dx = 64 or 128 features, any
// multiple of 32 columns of w.
//
// A CTA works a slice of 32 columns of w of one (batch, head) over a part of the
// tokens, by chunks of 128 tokens.  Columns of the state do not meet, so slices
// give few heads four times the CTAs without a second pass over the tokens; the
// price is that the weights x y^T are computed once per slice.  Per chunk, M = 128
// MMAs with operands as TMA leaves them (no pass over x or y):
//
//   R  = x y^T                      (K = Dx; raw weights, tensor memory)
//   O1 = x [Shi | Slo]              (K = Dx; the state in front, two bf16 values)
//   dS = y^T [w~1 | w~2 | w~3]      (K = tokens; w~ = decayed rows of w as a sum of
//                                    two or three bf16 values side by side)
//   O2 = P w                        (P = R times its powers of the decay, masked, in
//                                    bf16, A operand in tensor memory)
//   o  = scale (g^(.) (O1hi + O1lo) + O2),   S <- g^n S + dS1 + dS2 + dS3
//
// The state itself stays in fp32 registers (a thread has one row of the slice),
// so dS needs nothing of the chunk before and only the sum S is a chain.  Values
// side by side cost little: an MMA of N = 32 columns is bound by reading A from
// shared memory (128 x 16 values for 128 x 32 x 16 products), not by the
// products.
//
// Warp roles (18 warps):
//   0-7    P: powers of the decay, mask, bf16 (a lane quadrant and two of its
//          four blocks of 32 columns each); then half of the output columns of
//          the quadrant's tokens
//   8-11   state: registers, its bf16 values for the MMA (thread = row)
//   12-15  w~ (thread = token), and zeros behind a ragged sequence's end
//   16     TMA: lane 0 the x ring, lane 1 the y ring, lane 2 the w ring
//   17     TMEM owner and MMA issuer
// Every wait is bounded; a CTA that gives up counts the failure in device
// memory, drains its copies and MMAs, frees tensor memory and exits.
#include "common.cuh"
#include "mixer_common.cuh"
#include "retention.cuh"
#include "tc_common.cuh"

namespace linattn {
namespace {

using namespace tc;

constexpr int kC = 128;  // tokens per chunk
constexpr int kThreads = 576;
constexpr int kWarpS = 8, kWarpW = 12, kWarpTma = 16, kWarpMma = 17;
constexpr int kAhead = 2;        // chunks between a tile's prefetch into L2 and its load
constexpr int kBox = kC * 128;  // 128 tokens x 64 features, 128-byte swizzle
constexpr int kAtom = kC * 64;  // 128 tokens x 32 columns, 64-byte swizzle

// Shared memory, from a 1024-byte aligned base: slots of x and y, slots of w,
// w~ (one buffer; two in the pass that only sums states), the state's bf16
// values, the weights of a chunk's blocks, barriers.
template <int DX, int SW, int NS, bool STATE>
struct Lay {
  static constexpr int kTile = DX / 64 * kBox;
  static constexpr int kWTile = SW / 32 * kAtom;
  // a slot: x, then y
  static constexpr int kYAt = STATE ? 0 : kTile, kSlot = kYAt + kTile;
  // loads take 2000 cycles and more from issue to landing when all SMs stream, so
  // as many slots as fit
  static constexpr int kSlots = STATE ? 4 : 2, kWSlots = STATE || SW == 32 ? 4 : 2;
  static constexpr int kW = kSlots * kSlot;
  static constexpr int kWt = kW + kWSlots * kWTile;
  static constexpr int kWtBuf = NS * kWTile;
  static constexpr int kSop = kWt + (STATE ? 2 : 1) * kWtBuf;
  static constexpr int kSopAtom = DX * 64;
  // weights of a block of 32 x 32 on the diagonal and of the one beside it, rows
  // of kLdT floats (16-byte accesses of 8 rows meet every bank once)
  static constexpr int kLdT = 36;
  static constexpr int kTab = kSop + (STATE ? 0 : 2 * (SW / 32) * kSopAtom);
  static constexpr int kBar = kTab + (STATE ? 0 : 2 * 32 * kLdT * 4);
  static constexpr int kNumBars = 32;
  static constexpr int kMisc = kBar + kNumBars * 8;
  static constexpr int kAlloc = kMisc + 16 + 1024;
  static_assert(kAlloc <= 227 * 1024, "shared memory");
  // Tensor memory columns: two buffers of raw weights, in each block of 32
  // columns then P as bf16 pairs in the first 16; O1 with both values of the state
  // side by side; O2; dS (twice in the pass that only sums states).
  static constexpr uint32_t cR = 0, cO1 = 256, cO2 = cO1 + 2 * SW;
  static constexpr uint32_t cD = STATE ? 0 : cO2 + SW, cD2 = NS * SW;
  static_assert(cD + (STATE ? 2 : 1) * NS * SW <= 512, "tensor memory");
};

// Where a barrier is one and not a pair, each of its phases is seen by every
// waiter before the next can end.
enum Bar : int {
  kXYFull = 0,    // [4] tiles of x and y landed
  kXYEmpty = 4,   // [4] slot free (MMA commit)
  kWFull = 8,     // [4]
  kWEmpty = 12,   // [4]
  kRFull = 16,    // [2] raw weights computed
  kDFull = 18,    // [2] dS computed
  kWReady = 20,   // [2] w~ written (main pass: one)
  kDRead = 22,    // [2] the pass that only sums states: dS read
  kOGo = 24,      // the state's bf16 values written, outputs of the chunk before read
  kPReady = 25,   // P written
  kOFull = 26,    // O1, O2 complete
  kDrain = 27,
};

struct TcRole {
  CUtensorMap m[3];  // x, y, w
  uint8_t at[3][4];  // places of head, token and batch among each map's outer dimensions
};
struct TcParams {
  RetArgs a;
  TcRole map[kRetRoles];
  int parts, cpp, slices;
  unsigned int *timeouts;
};

// warp_wait of tc_common.cuh for a kernel of many waiting warps with much code: a
// plain try first (15 cycles where the phase is over, 50 with a hint), then the
// hardware holds the warp until the phase ends or the hint (nanoseconds) runs out,
// so that waiting warps leave the issue slots to the others; one function for all
// waits that take longer.
__device__ __forceinline__ bool held(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(1000000u)
      : "memory");
  return ok != 0;
}
__device__ __noinline__ bool held_longer(uint32_t bar, uint32_t parity, volatile int *abort, unsigned int *timeouts) {
  const long long t0 = clock64();
  bool ok;
  while (!(ok = held(bar, parity)) && !*abort) {
    if (clock64() - t0 > kWaitCycles) {
      *abort = 1;
      atomicAdd(timeouts, 1u);
      break;
    }
  }
  return ok;
}
__device__ __forceinline__ bool held_wait(uint64_t *bar, uint32_t parity, volatile int *abort, unsigned int *timeouts) {
  const uint32_t at = smem_u32(bar);
  bool ok = mbar_try_wait(bar, parity);
  if (!ok) ok = held_longer(at, parity, abort, timeouts);
  return __all_sync(0xffffffffu, ok);
}

// Of a descriptor only the address in its low word changes from step to step.
struct Desc {
  uint32_t lo, hi;
  __device__ __forceinline__ explicit Desc(uint64_t d) : lo(static_cast<uint32_t>(d)), hi(static_cast<uint32_t>(d >> 32)) {}
};
template <bool ADD>
__device__ __forceinline__ void mma_ss(uint32_t d, const Desc &a, uint32_t a_off, const Desc &b, uint32_t b_off,
                                       uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 x, y;\n setp.ne.b32 p, %6, 0;\n mov.b64 x, {%1, %2};\n mov.b64 y, {%3, %4};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %5, p;\n}\n" ::"r"(d),
      "r"(a.lo + a_off), "r"(a.hi), "r"(b.lo + b_off), "r"(b.hi), "r"(idesc), "n"(ADD ? 1 : 0)
      : "memory");
}
template <bool ADD>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, const Desc &b, uint32_t b_off, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 y;\n setp.ne.b32 p, %5, 0;\n mov.b64 y, {%2, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b.lo + b_off), "r"(b.hi), "r"(idesc), "n"(ADD ? 1 : 0)
      : "memory");
}
// The lane that issues a group of MMAs, the same every time.  A branch around the
// group, in a warp the compiler knows to agree on its role: 10 instructions an
// MMA, against 35 with the election inside each.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n selp.u32 %0, 1, 0, e;\n}\n" : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t *v) {
  float f[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) f[i] = __uint_as_float(v[i]);
  tmem_st16(taddr, f);
}

// A pair of fp32 values as NS pairs of bf16 values that add up to them (each
// remainder is exact).
template <int NS>
__device__ __forceinline__ void split2(f2 v, uint32_t *out) {
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const float2 x = unpack2(v);
    out[s] = pack_bf16x2(x.x, x.y);
    if (s + 1 < NS)
      v = add2(v, pack2(__uint_as_float((out[s] << 16) ^ 0x80000000u), __uint_as_float((out[s] & 0xffff0000u) ^ 0x80000000u)));
  }
}

template <int DX, int SW, int NS, bool STATE>
__global__ void __launch_bounds__(kThreads, 1) retention_tc_kernel(const __grid_constant__ TcParams p) {
  using Ly = Lay<DX, SW, NS, STATE>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                            ~static_cast<uintptr_t>(1023));
  uint64_t *bar = reinterpret_cast<uint64_t *>(sm + Ly::kBar);
  float *tab = reinterpret_cast<float *>(sm + Ly::kTab);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + Ly::kMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + Ly::kMisc + 4);

  const RetRole &r = p.a.role[blockIdx.z];
  const TcRole &map = p.map[blockIdx.z];
  const int np = STATE ? p.parts - 1 : p.parts;
  const int slice = blockIdx.x % p.slices, part = blockIdx.x / p.slices % np;
  const int64_t bh = blockIdx.x / p.slices / np;
  const int e0 = slice * SW;
  if (e0 >= r.Dw) return;
  const int b = static_cast<int>(bh / p.a.H), h = static_cast<int>(bh % p.a.H);
  // the shuffle tells the compiler that a warp agrees on its role
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int tokens = ret_tokens(p.a.lens, b, p.a.L);
  const int n = (tokens + kC - 1) / kC;
  const bool last_part = part == p.parts - 1;
  const int c0 = min(n, part * p.cpp), nc = (last_part ? n : min(n, c0 + p.cpp)) - c0;
  const bool keep = STATE || (last_part && r.end);  // the state behind the last chunk is wanted
  const float lg = p.a.lg.g[h];
  // chunk c of the part: its first token and how many it has
  auto first = [&](int c) { return (r.reverse ? n - 1 - c0 - c : c0 + c) * kC; };
  auto size = [&](int c) { return min(kC, tokens - first(c)); };

  if (!STATE)
    for (int i = tid; i < 2 * 32 * 32; i += kThreads) {
      const int row = i >> 5 & 31, e = i & 31, gap = 32 * (i >> 10) + (r.reverse ? e - row : row - e);
      tab[(i >> 5) * Ly::kLdT + e] = gap >= 0 ? exp2f(lg * static_cast<float>(gap)) : 0.f;
    }
  if (tid == 32 * kWarpTma) {
    for (int s = 0; s < 16; ++s) mbar_init(&bar[kXYFull + s], 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar[kRFull + s], 1);
      mbar_init(&bar[kDFull + s], 1);
      mbar_init(&bar[kWReady + s], STATE ? 12 : 4);
      mbar_init(&bar[kDRead + s], 4);
    }
    mbar_init(&bar[kOGo], 12);
    mbar_init(&bar[kPReady], 8);
    mbar_init(&bar[kOFull], 1);
    mbar_init(&bar[kDrain], 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == kWarpMma) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == kWarpTma) {
    if (lane < 2) {  // lane 0: x and y, lane 1: w
      auto map_of = [&](int i) { return &map.m[i]; };
      prefetch_tmap(map_of(lane == 0 ? 1 : 2));
      if (lane == 0 && !STATE) prefetch_tmap(map_of(0));
      uint64_t *fullb = &bar[lane == 0 ? kXYFull : kWFull], *emptyb = &bar[lane == 0 ? kXYEmpty : kWEmpty];
      const int hx = h / r.xg, hy = h / r.yg, hw = h / r.wg;
      const int sharers = r.Dw / SW;
      // f(map, column, outer coordinates) for each box of a tile of tensor i
      auto boxes = [&](int i, int head, int t, auto &&f) {
        const uint8_t *at = map.at[i];
        auto place = [&](int j) { return at[0] == j ? head : (at[1] == j ? t : b); };
        const int y = place(0), z = place(1), w = place(2);
#pragma unroll 1
        for (int j = 0; j < (i == 2 ? SW / 32 : DX / 64); ++j) f(j, i == 2 ? e0 + 32 * j : 64 * j, y, z, w);
      };
      const int slots = lane == 0 ? Ly::kSlots : Ly::kWSlots;
      int issued = 0;
      for (int c = 0; c < nc; ++c) {
        const int sl = c % slots;
        if (!mbar_wait(&emptyb[sl], ((c / slots) & 1) ^ 1, abort_flag, p.timeouts)) break;
        // The slots hold less than the memory's latency: later tiles come into L2
        // ahead, the boxes of x and y shared out among the slices that read them.
        const int t0 = first(c), tp = first(c + kAhead);
        const bool ahead = c + kAhead < nc;
        if (lane == 0) {
          mbar_arrive_expect_tx(&fullb[sl], Ly::kSlot);
          for (int i = STATE ? 1 : 0; i < 2; ++i) {
            uint8_t *dst = sm + sl * Ly::kSlot + (i == 0 ? 0 : Ly::kYAt);
            boxes(i, i == 0 ? hx : hy, t0, [&](int j, int x, int y, int z, int w) {
              tma_load_4d(dst + j * kBox, map_of(i), x, y, z, w, &fullb[sl]);
            });
          }
          for (int i = STATE ? 1 : 0; ahead && i < 2; ++i)
            boxes(i, i == 0 ? hx : hy, tp, [&](int j, int x, int y, int z, int w) {
              if ((i * (DX / 64) + j) % sharers == slice) tma_prefetch_4d(map_of(i), x, y, z, w);
            });
        } else {
          mbar_arrive_expect_tx(&fullb[sl], Ly::kWTile);
          boxes(2, hw, t0, [&](int j, int x, int y, int z, int w) {
            tma_load_4d(sm + Ly::kW + sl * Ly::kWTile + j * kAtom, map_of(2), x, y, z, w, &fullb[sl]);
          });
          if (ahead)
            boxes(2, hw, tp, [&](int, int x, int y, int z, int w) { tma_prefetch_4d(map_of(2), x, y, z, w); });
        }
        issued = c + 1;
      }
      if (*abort_flag)  // let every issued copy land before the CTA exits
        for (int c = issued > slots ? issued - slots : 0; c < issued; ++c)
          mbar_wait_drain(&fullb[c % slots], (c / slots) & 1);
    }
    __syncwarp();
  } else if (warp == kWarpMma) {
    constexpr uint32_t ID_R = idesc_bf16(128, 128, false, false);
    constexpr uint32_t ID_O1 = idesc_bf16(128, 2 * SW, false, true);
    constexpr uint32_t ID_D = idesc_bf16(DX, NS * SW, true, true);
    constexpr uint32_t ID_O2 = idesc_bf16(128, SW, false, true);
    const uint32_t base = smem_u32(sm);
    // rows as K-major operands (K = features) and y^T as A (M = features in
    // 64-wide atoms, K = tokens); w, w~ and the state with columns in atoms of 32
    auto rows = [&](int at) { return Desc(smem_desc(base + at, 16, 1024, kSw128)); };
    auto atoms = [&](int at, int atom) { return Desc(smem_desc(base + at, atom, 512, kSw64)); };
    auto step = [](int kk) { return static_cast<uint32_t>((kk >> 2) * (kBox >> 4) + (kk & 3) * 2); };
    auto slot = [](int c) { return c % Ly::kSlots; };
    auto landed = [&](int c) { return held_wait(&bar[kXYFull + slot(c)], (c / Ly::kSlots) & 1, abort_flag, p.timeouts); };
    auto tiles = [&](int c) {  // x and y of chunk c have landed
      return landed(c) &&
             // rows behind the end have to be zero first
             (size(c) == kC || held_wait(&bar[kWReady], c & 1, abort_flag, p.timeouts));
    };
    auto tiles_state = [&](int c) {  // y has landed, dS of two chunks ago has been read
      return landed(c) && (c < 2 || held_wait(&bar[kDRead + (c & 1)], ((c - 2) >> 1) & 1, abort_flag, p.timeouts));
    };
    auto weigh = [&](int c) {  // R of chunk c
      const Desc x = rows(slot(c) * Ly::kSlot), y = rows(slot(c) * Ly::kSlot + Ly::kYAt);
      const uint32_t d = tmem + Ly::cR + 128 * (c & 1);
      if (elect_one()) {
        mma_ss<false>(d, x, 0, y, 0, ID_R);
#pragma unroll
        for (int kk = 1; kk < DX / 16; ++kk) mma_ss<true>(d, x, step(kk), y, step(kk), ID_R);
        mma_commit(&bar[kRFull + (c & 1)]);
      }
      __syncwarp();
    };
    bool ok = true;
    if (!STATE && nc > 0) {
      ok = tiles(0);
      tc_fence_after();
      if (ok) weigh(0);
    }
    // Per chunk O1, dS, R of the next chunk and O2, so that each group's consumers
    // work behind other groups: P behind O2 and O1 and dS of the next chunk, the
    // state behind R and O2, the outputs' read (before the next O1) behind nothing.
    for (int c = 0; ok && c < nc; ++c) {
      const int sl = c & 1;
      const uint32_t ph = (c >> 1) & 1;
      if (!STATE) {
        if (!held_wait(&bar[kOGo], c & 1, abort_flag, p.timeouts)) break;
        tc_fence_after();
        const Desc x = rows(slot(c) * Ly::kSlot), sop = atoms(Ly::kSop, Ly::kSopAtom);
        if (elect_one()) {
          mma_ss<false>(tmem + Ly::cO1, x, 0, sop, 0, ID_O1);
#pragma unroll
          for (int kk = 1; kk < DX / 16; ++kk) mma_ss<true>(tmem + Ly::cO1, x, step(kk), sop, kk * 64, ID_O1);
        }
        __syncwarp();
      } else if (!tiles_state(c)) {
        break;
      }
      if (!held_wait(&bar[kWReady + (STATE ? sl : 0)], STATE ? ph : c & 1, abort_flag, p.timeouts)) break;
      tc_fence_after();
      const Desc yt(smem_desc(base + slot(c) * Ly::kSlot + Ly::kYAt, kBox, 1024, kSw128));
      const Desc wt = atoms(Ly::kWt + (STATE ? sl * Ly::kWtBuf : 0), kAtom);
      const uint32_t d = tmem + (STATE && sl ? Ly::cD2 : Ly::cD);
      if (elect_one()) {
        if (keep || c + 1 < nc) {
          mma_ss<false>(d, yt, 0, wt, 0, ID_D);
#pragma unroll
          for (int kk = 1; kk < kC / 16; ++kk) mma_ss<true>(d, yt, kk * 128, wt, kk * 64, ID_D);
        }
        mma_commit(&bar[kDFull + sl]);
        mma_commit(&bar[kXYEmpty + slot(c)]);
        if (STATE) mma_commit(&bar[kWEmpty + c % Ly::kWSlots]);
      }
      __syncwarp();
      if (!STATE) {
        if (c + 1 < nc) {
          if (!tiles(c + 1)) break;
          tc_fence_after();
          weigh(c + 1);
        }
        if (!held_wait(&bar[kPReady], c & 1, abort_flag, p.timeouts)) break;
        tc_fence_after();
        const Desc w = atoms(Ly::kW + c % Ly::kWSlots * Ly::kWTile, kAtom);
        const uint32_t pr = tmem + Ly::cR + 128 * sl;
        if (elect_one()) {
          mma_ts<false>(tmem + Ly::cO2, pr, w, 0, ID_O2);
#pragma unroll
          for (int kk = 1; kk < kC / 16; ++kk)
            mma_ts<true>(tmem + Ly::cO2, pr + 32 * (kk >> 1) + 8 * (kk & 1), w, kk * 64, ID_O2);
          mma_commit(&bar[kOFull]);
          mma_commit(&bar[kWEmpty + c % Ly::kWSlots]);
        }
        __syncwarp();
      }
    }
    // every MMA issued has completed before TMEM is released
    if (elect_one()) {
      mma_commit(&bar[kDrain]);
      mbar_wait_drain(&bar[kDrain], 0);
    }
    __syncwarp();
  } else if (warp >= kWarpW || (STATE && warp < kWarpS)) {
    // a third of the columns each where the warps that weigh have nothing to do
    const int t = tid & (kC - 1), group = STATE && warp >= kWarpW ? 2 : warp >> 2 & 1, groups = STATE ? 3 : 1;
    for (int c = 0; c < nc; ++c) {
      const int ws = c % Ly::kWSlots, xs = c % Ly::kSlots, nv = size(c);
      const float f = t < nv ? exp2f(lg * static_cast<float>(r.reverse ? t + 1 : nv - 1 - t)) : 0.f;
      // the buffer is free once the sum over the chunk that used it is done
      const int before = c - (STATE ? 2 : 1);
      if (!held_wait(&bar[kWFull + ws], (c / Ly::kWSlots) & 1, abort_flag, p.timeouts) ||
          (nv < kC && !held_wait(&bar[kXYFull + xs], (c / Ly::kSlots) & 1, abort_flag, p.timeouts)) ||
          (before >= 0 && !held_wait(&bar[kDFull + (before & 1)], (before >> 1) & 1, abort_flag, p.timeouts)))
        break;
      uint8_t *wrow = sm + Ly::kW + ws * Ly::kWTile;
      uint8_t *wt = sm + Ly::kWt + (STATE ? (c & 1) * Ly::kWtBuf : 0);
      if (t < nv) {
#pragma unroll 2
        for (int q = STATE ? group : 0; q < SW / 8; q += groups) {
          const int at = (q >> 2) * kAtom + sw64_off(t, 16 * (q & 3));
          const uint4 x = *reinterpret_cast<const uint4 *>(wrow + at);
          const uint32_t u[4] = {x.x, x.y, x.z, x.w};
          uint32_t s[4][NS];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            split2<NS>(mul2(dup2(f), pack2(__uint_as_float(u[k] << 16), __uint_as_float(u[k] & 0xffff0000u))), s[k]);
#pragma unroll
          for (int j = 0; j < NS; ++j)
            *reinterpret_cast<uint4 *>(wt + j * Ly::kWTile + at) = make_uint4(s[0][j], s[1][j], s[2][j], s[3][j]);
        }
      } else {
        const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll 1
        for (int q = STATE ? group : 0; q < SW / 8; q += groups) {
          const int at = (q >> 2) * kAtom + sw64_off(t, 16 * (q & 3));
          *reinterpret_cast<uint4 *>(wrow + at) = z;
          for (int j = 0; j < NS; ++j) *reinterpret_cast<uint4 *>(wt + j * Ly::kWTile + at) = z;
        }
#pragma unroll 1
        for (int q = STATE ? group : 0; q < DX / 8; q += groups)
          *reinterpret_cast<uint4 *>(sm + xs * Ly::kSlot + Ly::kYAt + (q >> 3) * kBox + sw128_off(t, 16 * (q & 7))) = z;
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[kWReady + (STATE ? c & 1 : 0)]);
    }
  } else if (warp >= kWarpS) {
    // row d of the state: all 32 lanes of a quadrant, or (64 features) 16
    const int qd = warp - kWarpS;
    const int d = DX == 128 ? 32 * qd + lane : 16 * qd + (lane & 15);
    const bool mine = DX == 128 || lane < 16;
    const int64_t size_of = static_cast<int64_t>(DX) * r.Dw;
    float *rec = r.rec + bh * (p.parts - 1) * size_of;
    f2 S[SW / 2];
#pragma unroll
    for (int e = 0; e < SW / 2; ++e) S[e] = dup2(0.f);
    if (!STATE) {
      const int here = ret_before(part * p.cpp, n, tokens, kC, r.reverse);
      if (r.start) {
        const float f = exp2f(lg * static_cast<float>(here)) * r.start_scale;
        const float *from = r.start + bh * size_of + static_cast<int64_t>(d) * r.start_rs +
                            static_cast<int64_t>(e0) * r.start_cs;
#pragma unroll
        for (int e = 0; e < SW / 2; ++e)
          S[e] = pack2(f * from[static_cast<int64_t>(2 * e) * r.start_cs], f * from[static_cast<int64_t>(2 * e + 1) * r.start_cs]);
      }
      for (int j = 0; j < part; ++j) {
        const f2 f = dup2(exp2f(lg * static_cast<float>(here - ret_before((j + 1) * p.cpp, n, tokens, kC, r.reverse))));
        const float4 *from = reinterpret_cast<const float4 *>(rec + j * size_of + d * r.Dw + e0);
#pragma unroll
        for (int e = 0; e < SW / 4; ++e) {
          const float4 v = from[e];
          S[2 * e] = fma2(f, pack2(v.x, v.y), S[2 * e]);
          S[2 * e + 1] = fma2(f, pack2(v.z, v.w), S[2 * e + 1]);
        }
      }
    }
    bool ok = true;
    for (int c = 0; c <= nc; ++c) {
      if (c > 0 && (c < nc || keep)) {  // S <- g^n S + dS of chunk c - 1
        const int l = c - 1;
        const f2 g = dup2(exp2f(lg * static_cast<float>(size(l))));
        if (!held_wait(&bar[kDFull + (l & 1)], (l >> 1) & 1, abort_flag, p.timeouts)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t at = tmem_addr(tmem, 32 * qd, STATE && (l & 1) ? Ly::cD2 : Ly::cD);
#pragma unroll
        for (int j = 0; j < SW / 16; ++j) {
          float x[NS][16];
#pragma unroll
          for (int k = 0; k < NS; ++k) tmem_ld16(at + SW * k + 16 * j, x[k]);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            f2 v = pack2(x[NS - 1][2 * e], x[NS - 1][2 * e + 1]);
#pragma unroll
            for (int k = NS - 2; k >= 0; --k) v = add2(v, pack2(x[k][2 * e], x[k][2 * e + 1]));
            S[8 * j + e] = fma2(g, S[8 * j + e], v);
          }
        }
        tc_fence_before();
      }
      if (STATE) {
        __syncwarp();
        if (c > 0 && c < nc && lane == 0) mbar_arrive(&bar[kDRead + ((c - 1) & 1)]);
      } else if (c < nc) {
        if (mine) {
#pragma unroll
          for (int q = 0; q < SW / 8; ++q) {
            uint32_t s[4][2];
#pragma unroll
            for (int k = 0; k < 4; ++k) split2<2>(S[4 * q + k], s[k]);
#pragma unroll
            for (int j = 0; j < 2; ++j)
              *reinterpret_cast<uint4 *>(sm + Ly::kSop + (j * (SW / 32) + (q >> 2)) * Ly::kSopAtom +
                                         sw64_off(d, 16 * (q & 3))) = make_uint4(s[0][j], s[1][j], s[2][j], s[3][j]);
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[kOGo]);
      }
    }
    if (keep && ok && mine) {
      float4 *to = reinterpret_cast<float4 *>((STATE ? rec + part * size_of : r.end + bh * size_of) + d * r.Dw + e0);
      const f2 f = dup2(STATE ? 1.f : r.end_scale);
#pragma unroll
      for (int e = 0; e < SW / 4; ++e) {
        const float2 lo = unpack2(mul2(f, S[2 * e])), hi = unpack2(mul2(f, S[2 * e + 1]));
        to[e] = make_float4(lo.x, lo.y, hi.x, hi.y);
      }
    }
  } else if (!STATE) {
    // P: rows of quadrant qd, blocks of 32 columns h2 and h2 + 2; output columns
    // [SW / 2 h2, + SW / 2)
    const int qd = warp & 3, h2 = warp >> 2, t = 32 * qd + lane;
    const bool rev = r.reverse;
    const uint32_t quad = tmem_addr(tmem, 32 * qd, 0);
    uint8_t *out = static_cast<uint8_t *>(r.o);
    const int wide = r.o_f32 ? 4 : 2;  // bytes of an output
    const int64_t unit = b * r.os.b + h * r.os.h + e0 + SW / 2 * h2;
    if (lane == 0 && nc > 0) mbar_arrive(&bar[kOGo]);  // no outputs in front of the first chunk
    for (int c = -1; c < nc; ++c) {
      if (c >= 0) {  // outputs of chunk c
        const int nv = size(c);
        const float f = r.out_scale * exp2f(lg * static_cast<float>(rev ? nv - 1 - t : t + 1));
        uint8_t *at = out + (unit + (first(c) + t) * r.os.t) * wide;
        if (!held_wait(&bar[kOFull], c & 1, abort_flag, p.timeouts)) break;
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < SW / 32; ++j) {
          float hi[16], lo[16], v[16];
          const uint32_t col = SW / 2 * h2 + 16 * j;
          tmem_ld16(quad + Ly::cO1 + col, hi);
          tmem_ld16(quad + Ly::cO1 + SW + col, lo);
          tmem_ld16(quad + Ly::cO2 + col, v);
          tmem_wait_ld();
          if (j == SW / 32 - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_relaxed(&bar[kOGo]);
          }
          if (t < nv) {
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = fmaf(f, hi[e] + lo[e], r.out_scale * v[e]);
            if (r.o_f32) {
              float4 *to = reinterpret_cast<float4 *>(at + 64 * j);
#pragma unroll
              for (int e = 0; e < 4; ++e) to[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
            } else {
              uint4 *to = reinterpret_cast<uint4 *>(at + 32 * j);
#pragma unroll
              for (int e = 0; e < 2; ++e)
                to[e] = make_uint4(pack_bf16x2(v[8 * e], v[8 * e + 1]), pack_bf16x2(v[8 * e + 2], v[8 * e + 3]),
                                   pack_bf16x2(v[8 * e + 4], v[8 * e + 5]), pack_bf16x2(v[8 * e + 6], v[8 * e + 7]));
            }
          }
        }
      }
      const int l = c + 1;  // weights of the next chunk
      if (l == nc) break;
      if (!held_wait(&bar[kRFull + (l & 1)], (l >> 1) & 1, abort_flag, p.timeouts)) break;
      tc_fence_after();
      const uint32_t raw = quad + Ly::cR + 128 * (l & 1);
#pragma unroll 1
      for (int g = h2; g < 4; g += 2) {
        const int away = rev ? g - qd : qd - g;
        uint32_t pk[16];
        if (away >= 0) {
          const float4 *w4 = reinterpret_cast<const float4 *>(tab + ((away > 0 ? 32 : 0) + lane) * Ly::kLdT);
          float a[32];
          tmem_ld32(raw + 32 * g, a);
          tmem_wait_ld();
          if (away > 1) {
            const f2 far = dup2(exp2f(lg * static_cast<float>(32 * (away - 1))));
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 v = unpack2(mul2(far, pack2(a[2 * e], a[2 * e + 1])));
              a[2 * e] = v.x, a[2 * e + 1] = v.y;
            }
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4 w = w4[e];
            const float2 lo = unpack2(mul2(pack2(w.x, w.y), pack2(a[4 * e], a[4 * e + 1])));
            const float2 hi = unpack2(mul2(pack2(w.z, w.w), pack2(a[4 * e + 2], a[4 * e + 3])));
            pk[2 * e] = pack_bf16x2(lo.x, lo.y);
            pk[2 * e + 1] = pack_bf16x2(hi.x, hi.y);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) pk[e] = 0u;
        }
        tmem_st16u(raw + 32 * g, pk);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[kPReady]);
    }
    if (p.a.fill && last_part)
      for (int i = tokens + t; i < p.a.L; i += kC) {
        uint4 *to = reinterpret_cast<uint4 *>(out + (unit + i * r.os.t) * wide);
        for (int e = 0; e < wide * SW / 32; ++e) to[e] = make_uint4(0, 0, 0, 0);
      }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) tmem_dealloc(tmem, 512);
}

template <int DX, int SW, int NS, bool STATE>
cudaError_t pass(const TcParams &p, int64_t units, cudaStream_t s) {
  auto k = retention_tc_kernel<DX, SW, NS, STATE>;
  const int bytes = Lay<DX, SW, NS, STATE>::kAlloc;
  const cudaError_t e = allow_smem(k, bytes);
  if (e != cudaSuccess) return e;
  const int np = STATE ? p.parts - 1 : p.parts;
  k<<<dim3(static_cast<unsigned>(units * np), 1, p.a.roles), kThreads, bytes, s>>>(p);
  return cudaGetLastError();
}

template <int DX, int SW, int NS>
cudaError_t go(const TcParams &p, int64_t units, cudaStream_t s) {
  if (p.parts > 1) {
    const cudaError_t e = pass<DX, SW, NS, true>(p, units, s);
    if (e != cudaSuccess) return e;
  }
  return pass<DX, SW, NS, false>(p, units, s);
}

int64_t columns(const RetArgs &a) {
  int64_t n = 0;
  for (int i = 0; i < a.roles; ++i) n += static_cast<int64_t>(a.B) * a.H * a.role[i].Dw;
  return n;
}

// Slices of 64 columns compute the raw weights half as often as slices of 32,
// but are half as many.  Three values of w~ do not fit beside them.
int slice_width(const RetArgs &a) {
  for (int i = 0; i < a.roles; ++i)
    if (a.role[i].Dw % 64 != 0 || a.role[i].end) return 32;
  return columns(a) / 64 >= kSMs - 24 ? 64 : 32;
}

}  // namespace

bool ret_tc_supported(const RetArgs &a, Dtype dt) {
  if (dt != kBF16) return false;
  for (int i = 0; i < a.roles; ++i)
    if ((a.role[i].Dx != 64 && a.role[i].Dx != 128) || a.role[i].Dw % 32 != 0) return false;
  return true;
}

int ret_parts_tc(const RetArgs &a) {
  const int64_t units = columns(a) / slice_width(a);
  const int chunks = (a.L + kC - 1) / kC;
  // Parts cost a pass over y and w for their records (about half of a chunk's
  // time) and a launch (about four chunks' time).
  int64_t parts = kSMs / (units > 0 ? units : 1);
  if (parts > 16) parts = 16;
  if (parts > chunks / 4) parts = chunks / 4;
  if (parts < 2 || 1.5 * chunks / parts + 4 > chunks) return 1;
  return static_cast<int>(parts);
}

cudaError_t launch_retention_tc(const RetArgs &a, int parts, cudaStream_t s) {
  const int chunks = (a.L + kC - 1) / kC, SW = slice_width(a);
  unsigned int *timeouts = wait_timeout_counter();
  if (!timeouts) return cudaErrorNotSupported;
  // one launch for the roles of each number of features
  for (const int DX : {64, 128}) {
    TcParams p = {};
    p.a = a;
    p.a.roles = 0;
    p.parts = parts;
    p.cpp = (chunks + parts - 1) / parts;
    p.timeouts = timeouts;
    bool exact = false;
    for (int i = 0; i < a.roles; ++i) {
      const RetRole &r = a.role[i];
      if (r.Dx != DX) continue;
      TcRole &m = p.map[p.a.roles];
      auto encode = [&](int i, const void *base, int width, int group, const RetStrides &s, int box) {
        return make_tmap_heads(&m.m[i], base, width, a.H / group, a.L, a.B, s.h, s.t, s.b, box, kC, m.at[i]);
      };
      if (!encode(0, r.x, DX, r.xg, r.xs, 64) || !encode(1, r.y, DX, r.yg, r.ys, 64) ||
          !encode(2, r.w, r.Dw, r.wg, r.ws, 32))
        return cudaErrorNotSupported;
      p.a.role[p.a.roles++] = r;
      if (r.Dw / SW > p.slices) p.slices = r.Dw / SW;
      exact |= r.end != nullptr;
    }
    if (!p.a.roles) continue;
    const int64_t units = static_cast<int64_t>(a.B) * a.H * p.slices;
    if (units * parts >= (1LL << 31)) return cudaErrorNotSupported;
    cudaError_t e;
    if (SW == 64) e = DX == 64 ? go<64, 64, 1>(p, units, s) : go<128, 64, 1>(p, units, s);
    else if (exact) e = DX == 64 ? go<64, 32, 3>(p, units, s) : go<128, 32, 3>(p, units, s);
    else e = DX == 64 ? go<64, 32, 1>(p, units, s) : go<128, 32, 1>(p, units, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace linattn
