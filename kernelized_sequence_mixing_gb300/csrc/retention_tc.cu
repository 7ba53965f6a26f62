// Retention on tcgen05 tensor cores: bf16, Dx = 128 or up to 64 features (fewer are
// filled up with zeros as they land), any multiple of 32 columns of w.
//
// A CTA works a slice of SW = 32 or 64 columns of w of one (batch, head) over a part
// of the tokens, by chunks of 128 tokens.  Columns of the state do not meet, so
// slices give few heads more CTAs without a second pass over the tokens; the price
// is that the weights x y^T are computed once per slice.  Per chunk, M = 128
// MMAs with operands as TMA leaves them (no pass over x or y):
//
//   R  = x y^T                      (K = Dx; raw weights, tensor memory)
//   O1 = x [Shi | Slo]              (K = Dx; the state in front, two bf16 values)
//   dS = y^T w~                     (K = tokens; w~ = decayed rows of w)
//   O2 = P w                        (P = R times its powers of the decay, masked, in
//                                    bf16, A operand in tensor memory)
//   o  = scale (g^(.) (O1hi + O1lo) + O2),   S <- g^n S + dS
//
// The state itself stays in fp32 registers (a thread has one row of the slice),
// so dS needs nothing of the chunk before and only the sum S is a chain.  Values
// side by side cost little: an MMA of N = 32 columns is bound by reading A from
// shared memory (128 x 16 values for 128 x 32 x 16 products), not by the
// products.
//
// Warp roles (19 warps):
//   0-7    P: powers of the decay, mask, bf16 (a lane quadrant and two of its
//          four blocks of 32 columns each); with slices of 64 columns also the
//          output rows, half the columns each
//   8-11   state: registers, its bf16 values for the MMA (thread = row)
//   12-15  w~ (thread = token), and zeros behind a ragged sequence's end; with
//          slices of 32 columns also the output rows
//   16     TMA: rings of x, y and w
//   17     TMEM owner, issues R and O2
//   18     issues O1 and dS: one warp's instructions for all four (some 500 a
//          chunk) take longer than the products
// Every wait is bounded; a CTA that gives up counts the failure in device
// memory, drains its copies and MMAs, frees tensor memory and exits.
//
// Two passes where the tokens are cut into parts: one sums each part's own state
// (no x, no weights, no outputs), the other starts from those sums.  A returned
// state is the sum of all parts' records, built from decayed rows as three bf16
// values (fp32 accuracy); states for outputs make do with one (but where the roles of
// a launch share that pass with one that returns its state, all have three).
//
// Bound by no unit but by the chain of waits of one CTA an SM (weights, P, O2, outputs;
// dS, state, O1): about 2400 cycles a chunk of 128 features and 32 columns against 700
// of products.  On an SM that works (128 of 152 at B2 H16) the tensor pipe is busy 41%
// of the time, its reading of operands 48%, the pipe of shared memory 49%, and half of
// the issue slots are taken.  Measured: B2 L16384 H16 D128
// forward 162 us (3.3 TB/s of q, k, v, o; 0.49 of the copy rate); B1 L65536 H8|4 D128
// with the final state 199 us; backward B4 L4096 H8 D64 63 us.
#include <type_traits>

#include "common.cuh"
#include "dependent.cuh"
#include "mixer_common.cuh"
#include "retention.cuh"
#include "tc_common.cuh"

namespace linattn {
namespace {

using namespace tc;

constexpr int kC = 128;  // tokens per chunk
constexpr int kThreads = 608;
constexpr int kWarpS = 8, kWarpW = 12, kWarpTma = 16, kWarpMma = 17;  // and 18
constexpr int kBox = kC * 128;  // 128 tokens x 64 features, 128-byte swizzle
constexpr int kAtom = kC * 64;  // 128 tokens x 32 columns, 64-byte swizzle

// Shared memory, from a 1024-byte aligned base: slots of x and y, slots of w,
// w~ (one buffer; two in the pass that only sums states), the state's bf16
// values, the weights of a chunk's blocks, barriers.
template <int DX, int SW, int NS, bool STATE>
struct Lay {
  static constexpr int kTile = DX / 64 * kBox;
  static constexpr int kWTile = SW / 32 * kAtom;
  // Loads take 2000 cycles and more from issue to landing when all SMs stream, so
  // as many slots as fit; y is held longer than x, w longest.
  static constexpr bool kTight = DX == 128 && SW == 64 && NS == 3;
  static constexpr int kXSlots = 2, kYSlots = STATE ? (kTight ? 3 : 4) : (SW == 32 ? 3 : 2);
  static constexpr int kWSlots = STATE ? (kTight ? 2 : 4) : (SW == 32 ? 4 : 2);
  static constexpr int kX = 0;
  static constexpr int kY = STATE ? 0 : kXSlots * kTile;
  static constexpr int kW = kY + kYSlots * kTile;
  static constexpr int kWt = kW + kWSlots * kWTile;
  static constexpr int kWtBuf = NS * kWTile;
  static constexpr int kSop = kWt + (STATE ? 2 : 1) * kWtBuf;
  static constexpr int kSopAtom = DX * 64;
  // weights of a block of 32 x 32 on the diagonal and of the one beside it, rows
  // of kLdT floats (16-byte accesses of 8 rows meet every bank once)
  static constexpr int kLdT = 36;
  static constexpr int kTab = kSop + (STATE ? 0 : 2 * (SW / 32) * kSopAtom);
  static constexpr int kBar = kTab + (STATE ? 0 : 2 * 32 * kLdT * 4);
  static constexpr int kNumBars = 44;
  static constexpr int kMisc = kBar + kNumBars * 8;
  static constexpr int kAlloc = kMisc + 16 + 1024;
  static_assert(kAlloc <= 227 * 1024, "shared memory");
  // Tensor memory columns: two buffers of raw weights, in each block of 32
  // columns then P as bf16 pairs in the first 16; kO buffers of O1, with both
  // values of the state side by side, and O2; dS, of each value of w~ (twice in the
  // pass that only sums states).
  static constexpr int kO = SW == 32 ? 2 : 1;
  static constexpr uint32_t cR = 0, cO = 256, cOBuf = 3 * SW;
  static constexpr uint32_t cD = STATE ? 0 : cO + kO * cOBuf, cD2 = NS * SW;
  static_assert(cD + (STATE ? 2 : 1) * NS * SW <= 512, "tensor memory");
};

// Each phase of a barrier is seen by every waiter before the phase after next of
// the same barrier can end; the numbers of barriers follow from how far the roles
// can run ahead of one another.
enum Bar : int {
  kXFull = 0,     // [4] tile landed
  kXEmpty = 4,    // [4] slot free (commits of both issuing warps, of one where states are summed)
  kYFull = 8,     // [4]
  kYEmpty = 12,   // [4]
  kWFull = 16,    // [4]
  kWEmpty = 20,   // [4]
  kRFull = 24,    // [2] raw weights computed
  kDFull = 26,    // [2] dS computed
  kWReady = 28,   // [4] w~ written: the warp that issues O2 waits for it late
  kDRead = 32,    // [2] the pass that only sums states: dS read
  kPReady = 34,   // [2] P written
  kOFull = 36,    // [2] O1, O2 complete
  kORead = 38,    // [2] O1, O2 read
  kSReady = 40,   // the state's bf16 values written
  kDrain = 41,    // [2]
};

struct TcRole {
  CUtensorMap m[3];  // x, y, w
};
struct TcParams {
  RetArgs a;
  TcRole map[kRetRoles];
  int parts, cpp, slices, records;  // records: of the role of this launch that has most
  bool sectors;
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

// N MMAs along K, D[tmem] = (ADD: +=) sum of A[smem] B[smem]^T, the operands'
// addresses (in the descriptors' low words, in units of 16 bytes) going on by a
// step each; a step of 0: K-major rows of 64 features, by 2 and, behind each four,
// to the next box.  All lanes come here and the leader issues, by predicate: with
// a branch of one lane around them the operands go through vector registers and an
// MMA takes 50 cycles to issue however small it is, against 16 (a loop, not
// unrolled, cannot feed the tensor pipe either).
template <int N, bool ADD, int A_STEP, int B_STEP>
__device__ __forceinline__ void mma_group(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
  const uint32_t alo = static_cast<uint32_t>(a), blo = static_cast<uint32_t>(b);
  const uint32_t ahi = static_cast<uint32_t>(a >> 32), bhi = static_cast<uint32_t>(b >> 32);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t row = (i >> 2) * (kBox >> 4) + (i & 3) * 2;
    asm volatile(
        "{\n .reg .pred p, e;\n .reg .b64 x, y;\n setp.ne.b32 p, %6, 0;\n setp.ne.b32 e, %7, 0;\n"
        " mov.b64 x, {%1, %2};\n mov.b64 y, {%3, %4};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %5, p;\n}\n" ::"r"(d),
        "r"(alo + (A_STEP ? i * A_STEP : row)), "r"(ahi), "r"(blo + (B_STEP ? i * B_STEP : row)), "r"(bhi), "r"(idesc),
        "r"(ADD || i > 0 ? 1u : 0u), "r"(leader)
        : "memory");
  }
}
// The same with A in tensor memory, P: 16 values of K in 8 columns, 32 in the first
// half of each 32 columns.
template <int N, int B_STEP>
__device__ __forceinline__ void mma_group_p(uint32_t leader, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc) {
  const uint32_t blo = static_cast<uint32_t>(b), bhi = static_cast<uint32_t>(b >> 32);
#pragma unroll
  for (int i = 0; i < N; ++i)
    asm volatile(
        "{\n .reg .pred p, e;\n .reg .b64 y;\n setp.ne.b32 p, %5, 0;\n setp.ne.b32 e, %6, 0;\n mov.b64 y, {%2, %3};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n}\n" ::"r"(d),
        "r"(a + 32 * (i >> 1) + 8 * (i & 1)), "r"(blo + i * B_STEP), "r"(bhi), "r"(idesc), "r"(i > 0 ? 1u : 0u),
        "r"(leader)
        : "memory");
}
__device__ __forceinline__ void commit(uint32_t leader, uint64_t *bar) {
  asm volatile(
      "{\n .reg .pred e;\n setp.ne.b32 e, %1, 0;\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar)),
      "r"(leader)
      : "memory");
}
__device__ __forceinline__ void expect_tx(uint32_t leader, uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n .reg .pred e;\n setp.ne.b32 e, %2, 0;\n"
      " @e mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;\n}\n" ::"r"(bar),
      "r"(bytes), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void load_tile(uint32_t leader, uint32_t dst, const CUtensorMap *map, int token, int atom,
                                          int head, int batch, uint32_t bar) {
  asm volatile(
      "{\n .reg .pred e;\n setp.ne.b32 e, %7, 0;\n"
      " @e cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {0, %2, %3, %4, %5}], [%6];\n}\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(token), "r"(atom), "r"(head), "r"(batch), "r"(bar), "r"(leader)
      : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n selp.u32 %0, 1, 0, e;\n}\n" : "=r"(r));
  return r;
}
// A value that all lanes agree on, and the compiler knows it.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

__device__ __forceinline__ void tmem_st8u(uint32_t taddr, const uint32_t *v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
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

  const RetRole &r = p.a.role[blockIdx.y];
  const TcRole &map = p.map[blockIdx.y];
  const int np = STATE ? p.records : p.parts;
  const int slice = blockIdx.x % p.slices, part = blockIdx.x / p.slices % np;
  const int64_t bh = blockIdx.x / p.slices / np;
  const int e0 = slice * SW;
  // the last part's record serves the end state alone
  if (e0 >= r.Dw || (STATE && part >= r.records)) return;
  const int b = static_cast<int>(bh / p.a.H), h = static_cast<int>(bh % p.a.H);
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const int tokens = uniform(ret_tokens(p.a.lens, b, p.a.L));
  const int n = (tokens + kC - 1) / kC;
  const bool last_part = part == p.parts - 1;
  const int c0 = min(n, part * p.cpp), nc = (last_part ? n : min(n, c0 + p.cpp)) - c0;
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
    for (int s = 0; s < kRFull; ++s) {
      const bool both = !STATE && ((s >= kXEmpty && s < kYFull) || (s >= kYEmpty && s < kWFull));
      mbar_init(&bar[s], both ? 2 : 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar[kRFull + s], 1);
      mbar_init(&bar[kDFull + s], 1);
      mbar_init(&bar[kWReady + s], STATE ? 12 : 4);
      mbar_init(&bar[kWReady + 2 + s], STATE ? 12 : 4);
      mbar_init(&bar[kDRead + s], 4);
      mbar_init(&bar[kPReady + s], 8);
      mbar_init(&bar[kOFull + s], 2);
      mbar_init(&bar[kORead + s], SW == 32 ? 4 : 8);  // the warps that write outputs
    }
    mbar_init(&bar[kSReady], 4);
    mbar_init(&bar[kDrain], 1);
    mbar_init(&bar[kDrain + 1], 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == kWarpMma) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  // the pass behind comes up as this one's CTAs end; before the first bounded wait
  // all of it waits for the records
  if (STATE) let_next_start();
  else wait_for_previous();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*tmem_slot);

  // Output columns [col, col + 16 N) of the rows of a lane quadrant.
  auto outputs = [&](int c, int qd, int col, auto pieces) {
    constexpr int N = decltype(pieces)::value;
    const int nv = size(c), t = 32 * qd + lane, wide = r.o_f32 ? 4 : 2;
    const float f = r.out_scale * exp2f(lg * static_cast<float>(r.reverse ? nv - 1 - t : t + 1));
    uint8_t *at = static_cast<uint8_t *>(r.o) + (b * r.os.b + h * r.os.h + e0 + col + (first(c) + t) * r.os.t) * wide;
    if (!held_wait(&bar[kOFull + (c & 1)], (c >> 1) & 1, abort_flag, p.timeouts)) return false;
    tc_fence_after();
    const uint32_t o = tmem_addr(tmem, 32 * qd, Ly::cO + (Ly::kO == 2 && (c & 1) ? Ly::cOBuf : 0u) + col);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      float hi[16], lo[16], v[16];
      tmem_ld16(o + 16 * j, hi);
      tmem_ld16(o + 16 * j + SW, lo);
      tmem_ld16(o + 16 * j + 2 * SW, v);
      tmem_wait_ld();
      if (j == N - 1) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_relaxed(&bar[kORead + (c & 1)]);
      }
      if (t < nv) {
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = fmaf(f, hi[e] + lo[e], r.out_scale * v[e]);
        if (r.o_f32) {
          float4 *to = reinterpret_cast<float4 *>(at + 64 * j);
#pragma unroll
          for (int e = 0; e < 4; ++e) to[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        } else {
          uint32_t pk[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) pk[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
          // whole 32-byte sectors where the rows lie on them (191 us against 210)
          if (p.sectors) {
            st_global_v8(at + 32 * j, pk);
          } else {
            uint4 *to = reinterpret_cast<uint4 *>(at + 32 * j);
            to[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
            to[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
          }
        }
      }
    }
    return true;
  };
  // Zeros behind a sequence's end.
  auto fill = [&](int t, int col, int cols) {
    if (!p.a.fill || !last_part) return;
    const int wide = r.o_f32 ? 4 : 2;
    uint8_t *out = static_cast<uint8_t *>(r.o) + (b * r.os.b + h * r.os.h + e0 + col) * wide;
    for (int i = tokens + t; i < p.a.L; i += kC) {
      uint4 *to = reinterpret_cast<uint4 *>(out + i * r.os.t * wide);
      for (int e = 0; e < cols * wide / 16; ++e) to[e] = make_uint4(0, 0, 0, 0);
    }
  };
  // Outputs are the work of the warps that have time for it: with slices of 32
  // columns those of w~, with 64 those of P, half the columns each.
  constexpr bool kOutW = SW == 32;

  if (warp == kWarpTma) {
    // The warp as one for all rings, the leader's copies by predicate (see
    // mma_group).  Each wait is for groups that need earlier loads alone: in turn x
    // of chunk c and, where they have more slots, y and w of later chunks.
    const uint32_t leader = elect_one();
    struct Ring {
      const CUtensorMap *m;
      uint64_t *full;
      int sm, head, slots, bytes, atom, ahead;
    };
    const Ring rings[3] = {
        {&map.m[0], &bar[kXFull], Ly::kX, h / r.xg, Ly::kXSlots, Ly::kTile, 0, 0},
        {&map.m[1], &bar[kYFull], Ly::kY, h / r.yg, Ly::kYSlots, Ly::kTile, 0, STATE ? 0 : Ly::kYSlots - Ly::kXSlots},
        {&map.m[2], &bar[kWFull], Ly::kW, h / r.wg, Ly::kWSlots, Ly::kWTile, e0 / 32,
         STATE ? 0 : Ly::kWSlots - Ly::kXSlots}};
    constexpr int kFirst = STATE ? 1 : 0;
    int issued[3] = {0, 0, 0};
    auto load = [&](const Ring &g, int c) {
      const int sl = c % g.slots;
      if (!held_wait(g.full + 4 + sl, ((c / g.slots) & 1) ^ 1, abort_flag, p.timeouts)) return false;
      const uint32_t full = smem_u32(g.full + sl);
      __syncwarp();
      expect_tx(leader, full, g.bytes);
      load_tile(leader, smem_u32(sm + g.sm + sl * g.bytes), g.m, first(c), g.atom, g.head, b, full);
      return true;
    };
    bool ok = true;
    for (int c = 0; ok && c < nc; ++c)
#pragma unroll
      for (int i = kFirst; i < 3; ++i)
#pragma unroll 1
        for (; ok && issued[i] <= c + rings[i].ahead && issued[i] < nc; ++issued[i])
          if (!load(rings[i], issued[i])) {
            ok = false;
            break;
          }
    if (*abort_flag)  // let every issued copy land before the CTA exits
#pragma unroll
      for (int i = kFirst; i < 3; ++i)
        for (int c = max(0, issued[i] - rings[i].slots); c < issued[i]; ++c)
          mbar_wait_drain(rings[i].full + c % rings[i].slots, (c / rings[i].slots) & 1);
    __syncwarp();
  } else if (warp >= kWarpMma) {
    const uint32_t base = smem_u32(sm);
    // rows as K-major operands (K = features) and y^T as A (M = features in
    // 64-wide atoms, K = tokens); w, w~ and the state with columns in atoms of 32
    auto rows = [&](int at) { return smem_desc(base + at, 16, 1024, kSw128); };
    auto atoms = [&](int at, int atom) { return smem_desc(base + at, atom, 512, kSw64); };
    auto xs = [](int c) { return c % Ly::kXSlots; };
    auto ys = [](int c) { return c % Ly::kYSlots; };
    auto x_landed = [&](int c) { return held_wait(&bar[kXFull + xs(c)], (c / Ly::kXSlots) & 1, abort_flag, p.timeouts); };
    auto y_landed = [&](int c) { return held_wait(&bar[kYFull + ys(c)], (c / Ly::kYSlots) & 1, abort_flag, p.timeouts); };
    auto w_ready = [&](int c) { return held_wait(&bar[kWReady + (c & 3)], (c >> 2) & 1, abort_flag, p.timeouts); };
    // the outputs that were in the buffer have been read
    auto o_free = [&](int c) {
      const int l = c - Ly::kO;
      return l < 0 || held_wait(&bar[kORead + (l & 1)], (l >> 1) & 1, abort_flag, p.timeouts);
    };
    auto o_at = [&](int c) { return tmem + Ly::cO + (Ly::kO == 2 && (c & 1) ? Ly::cOBuf : 0u); };
    const uint32_t leader = elect_one();
    if (warp == kWarpMma) {
      // R of a chunk ahead of O2 of the one before, so that P works behind O2
      if (!STATE) {
        constexpr uint32_t ID_R = idesc_bf16(128, 128, false, false), ID_O2 = idesc_bf16(128, SW, false, true);
#pragma unroll 1
        for (int c = 0; c <= nc; ++c) {
          if (c < nc) {
            // rows behind the end have to be zero first
            if (!x_landed(c) || !y_landed(c) || (size(c) < kC && !w_ready(c))) break;
            tc_fence_after();
            __syncwarp();
            mma_group<DX / 16, false, 0, 0>(leader, tmem + Ly::cR + 128 * (c & 1), rows(Ly::kX + xs(c) * Ly::kTile),
                                            rows(Ly::kY + ys(c) * Ly::kTile), ID_R);
            commit(leader, &bar[kRFull + (c & 1)]);
            commit(leader, &bar[kXEmpty + xs(c)]);
            commit(leader, &bar[kYEmpty + ys(c)]);
          }
          if (c > 0) {
            const int l = c - 1;
            if (!w_ready(l) || !o_free(l) || !held_wait(&bar[kPReady + (l & 1)], (l >> 1) & 1, abort_flag, p.timeouts))
              break;
            tc_fence_after();
            __syncwarp();
            mma_group_p<kC / 16, 64>(leader, o_at(l) + 2 * SW, tmem + Ly::cR + 128 * (l & 1),
                                     atoms(Ly::kW + l % Ly::kWSlots * Ly::kWTile, kAtom), ID_O2);
            commit(leader, &bar[kOFull + (l & 1)]);
            commit(leader, &bar[kWEmpty + l % Ly::kWSlots]);
          }
        }
      }
    } else {
      constexpr uint32_t ID_O1 = idesc_bf16(128, 2 * SW, false, true);
      constexpr uint32_t ID_D = idesc_bf16(DX, NS * SW, true, true);
#pragma unroll 1
      for (int c = 0; c < nc; ++c) {
        const int sl = c & 1;
        if (!STATE) {
          if (!x_landed(c) || !o_free(c) || !held_wait(&bar[kSReady], c & 1, abort_flag, p.timeouts)) break;
          tc_fence_after();
          __syncwarp();
          mma_group<DX / 16, false, 0, 64>(leader, o_at(c), rows(Ly::kX + xs(c) * Ly::kTile), atoms(Ly::kSop, Ly::kSopAtom),
                                           ID_O1);
          commit(leader, &bar[kOFull + sl]);
          commit(leader, &bar[kXEmpty + xs(c)]);
        } else if (c > 1 && !held_wait(&bar[kDRead + sl], ((c - 2) >> 1) & 1, abort_flag, p.timeouts)) {
          break;  // dS of two chunks ago has been read
        }
        if (!y_landed(c) || !w_ready(c)) break;
        tc_fence_after();
        __syncwarp();
        if (STATE || c + 1 < nc) {
          const uint64_t yt = smem_desc(base + Ly::kY + ys(c) * Ly::kTile, kBox, 1024, kSw128);
          const uint64_t wt = atoms(Ly::kWt + (STATE ? sl * Ly::kWtBuf : 0), kAtom);
          const uint32_t d = tmem + Ly::cD + (STATE && sl ? Ly::cD2 : 0u);
          mma_group<kC / 16, false, 128, 64>(leader, d, yt, wt, ID_D);
        }
        commit(leader, &bar[kDFull + sl]);
        commit(leader, &bar[kYEmpty + ys(c)]);
        if (STATE) commit(leader, &bar[kWEmpty + c % Ly::kWSlots]);
      }
    }
    // every MMA issued has completed before TMEM is released
    commit(leader, &bar[kDrain + warp - kWarpMma]);
    mbar_wait_drain(&bar[kDrain + warp - kWarpMma], 0);
    __syncwarp();
  } else if (warp >= kWarpW || (STATE && warp < kWarpS)) {
    // a third of the columns each where the warps that weigh have nothing to do
    const int t = tid & (kC - 1), group = STATE && warp >= kWarpW ? 2 : warp >> 2 & 1, groups = STATE ? 3 : 1;
    for (int c = 0; c <= nc; ++c) {
      if (c == nc) {
        if (!STATE && kOutW && c > 0) outputs(c - 1, warp - kWarpW, 0, std::integral_constant<int, SW / 16>{});
        break;
      }
      const int ws = c % Ly::kWSlots, ys = c % Ly::kYSlots, nv = size(c);
      const float f = t < nv ? exp2f(lg * static_cast<float>(r.reverse ? t + 1 : nv - 1 - t)) : 0.f;
      // the buffer is free once the sum over the chunk that used it is done
      const int before = c - (STATE ? 2 : 1);
      if (!held_wait(&bar[kWFull + ws], (c / Ly::kWSlots) & 1, abort_flag, p.timeouts) ||
          (nv < kC && !held_wait(&bar[kYFull + ys], (c / Ly::kYSlots) & 1, abort_flag, p.timeouts)) ||
          (before >= 0 && !held_wait(&bar[kDFull + (before & 1)], (before >> 1) & 1, abort_flag, p.timeouts)))
        break;
      uint8_t *wrow = sm + Ly::kW + ws * Ly::kWTile;
      uint8_t *wt = sm + Ly::kWt + (STATE ? (c & 1) * Ly::kWtBuf : 0);
      if (t < nv) {
#pragma unroll 1
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
          *reinterpret_cast<uint4 *>(sm + Ly::kY + ys * Ly::kTile + (q >> 3) * kBox + sw128_off(t, 16 * (q & 7))) = z;
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[kWReady + (c & 3)]);
      if (!STATE && kOutW && c > 0 && !outputs(c - 1, warp - kWarpW, 0, std::integral_constant<int, SW / 16>{})) break;
    }
    if (!STATE && kOutW) fill(t, 0, SW);
  } else if (warp >= kWarpS) {
    // row d of the state: all 32 lanes of a quadrant, or (64 features) 16
    const int qd = warp - kWarpS;
    const int d = DX == 128 ? 32 * qd + lane : 16 * qd + (lane & 15);
    const bool mine = DX == 128 || lane < 16;
    const bool stored = mine && (DX == 128 || d < r.Dx);  // rows behind Dx stay zero
    const int64_t size_of = static_cast<int64_t>(r.Dx) * r.Dw;
    float *rec = r.rec + bh * r.records * size_of;
    f2 S[SW / 2];
#pragma unroll
    for (int e = 0; e < SW / 2; ++e) S[e] = dup2(0.f);
    if (!STATE && stored) {
      const int here = ret_before(part * p.cpp, n, tokens, kC, r.reverse);
      if (r.start) {
        const float f = exp2f(lg * static_cast<float>(here)) * r.start_scale;
        const float *from = r.start + bh * r.state + static_cast<int64_t>(d) * r.start_rs +
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
      if (last_part && r.end) {
        // the end state: this part's start and its record, whose sums are exact to
        // fp32 (w~ as three values), while this pass makes do with one
        const f2 f = dup2(exp2f(lg * static_cast<float>(tokens - here)) * r.end_scale), one = dup2(r.end_scale);
        const float4 *from = reinterpret_cast<const float4 *>(rec + part * size_of + d * r.Dw + e0);
        float4 *to = reinterpret_cast<float4 *>(r.end + bh * r.state + d * r.Dw + e0);
#pragma unroll
        for (int e = 0; e < SW / 4; ++e) {
          const float4 v = from[e];
          const float2 lo = unpack2(fma2(one, pack2(v.x, v.y), mul2(f, S[2 * e])));
          const float2 hi = unpack2(fma2(one, pack2(v.z, v.w), mul2(f, S[2 * e + 1])));
          to[e] = make_float4(lo.x, lo.y, hi.x, hi.y);
        }
      }
    }
    __syncwarp();
    bool ok = true;
    for (int c = 0; c <= nc; ++c) {
      if (c > 0 && (c < nc || STATE)) {  // S <- g^n S + dS of chunk c - 1
        const int l = c - 1;
        const f2 g = dup2(exp2f(lg * static_cast<float>(size(l))));
        if (!held_wait(&bar[kDFull + (l & 1)], (l >> 1) & 1, abort_flag, p.timeouts)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t at = tmem_addr(tmem, 32 * qd, Ly::cD + (STATE && (l & 1) ? Ly::cD2 : 0u));
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
        if (lane == 0) mbar_arrive(&bar[kSReady]);
      }
    }
    if (STATE && ok && stored) {
      float4 *to = reinterpret_cast<float4 *>(rec + part * size_of + d * r.Dw + e0);
#pragma unroll
      for (int e = 0; e < SW / 4; ++e) {
        const float2 lo = unpack2(S[2 * e]), hi = unpack2(S[2 * e + 1]);
        to[e] = make_float4(lo.x, lo.y, hi.x, hi.y);
      }
    }
  } else if (!STATE) {
    // P: rows of quadrant qd, blocks of 32 columns h2 and h2 + 2
    const int qd = warp & 3, h2 = warp >> 2, t = 32 * qd + lane;
    const bool rev = r.reverse;
    const uint32_t quad = tmem_addr(tmem, 32 * qd, 0);
    // the next chunk's weights first: O2 of this one waits for its own
    for (int c = -1; c < nc; ++c) {
      const int l = c + 1;  // weights of the next chunk
      if (l < nc) {
        if (!held_wait(&bar[kRFull + (l & 1)], (l >> 1) & 1, abort_flag, p.timeouts)) break;
        tc_fence_after();
        const uint32_t raw = quad + Ly::cR + 128 * (l & 1);
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {  // half of a block: 16 columns
          const int g = h2 + (i & 2), half = i & 1, away = rev ? g - qd : qd - g;
          uint32_t pk[8];
          if (away >= 0) {
            const float4 *w4 = reinterpret_cast<const float4 *>(tab + ((away > 0 ? 32 : 0) + lane) * Ly::kLdT + 16 * half);
            const f2 far = dup2(away > 1 ? exp2f(lg * static_cast<float>(32 * (away - 1))) : 1.f);
            float a[16];
            tmem_ld16(raw + 32 * g + 16 * half, a);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float4 w = w4[e];
              const float2 lo = unpack2(mul2(mul2(far, pack2(w.x, w.y)), pack2(a[4 * e], a[4 * e + 1])));
              const float2 hi = unpack2(mul2(mul2(far, pack2(w.z, w.w)), pack2(a[4 * e + 2], a[4 * e + 3])));
              pk[2 * e] = pack_bf16x2(lo.x, lo.y);
              pk[2 * e + 1] = pack_bf16x2(hi.x, hi.y);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) pk[e] = 0u;
          }
          // the second half's P lies over the first half's raw weights, read already
          tmem_st8u(raw + 32 * g + 8 * half, pk);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[kPReady + (l & 1)]);
      }
      if (!kOutW && c >= 0 && !outputs(c, qd, SW / 2 * h2, std::integral_constant<int, SW / 32>{})) break;
    }
    if (!kOutW) fill(t, SW / 2 * h2, SW / 2);
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
  const unsigned grid = static_cast<unsigned>(units * (STATE ? p.records : p.parts));
  if (!STATE && p.records > 0) return launch_dependent(k, grid, p.a.roles, kThreads, bytes, s, p);
  k<<<dim3(grid, p.a.roles), kThreads, bytes, s>>>(p);
  return cudaGetLastError();
}

template <int DX, int SW>
cudaError_t go(const TcParams &p, bool exact, int64_t units, cudaStream_t s) {
  if (p.records > 0) {
    const cudaError_t e = exact ? pass<DX, SW, 3, true>(p, units, s) : pass<DX, SW, 1, true>(p, units, s);
    if (e != cudaSuccess) return e;
  }
  return pass<DX, SW, 1, false>(p, units, s);
}

// How a call is cut: slices of SW columns and parts of the tokens.
struct Cut {
  int SW, parts;
};

// The cut that is done first by a model of one CTA per SM: a chunk takes 1 unit of
// time with slices of 32 columns and 1.6 with 64 (2440 and 3850 cycles of 128
// features), in the pass that sums states 0.4 and 0.5, and a CTA 4 units to begin
// and end.
Cut cut_of(const RetArgs &a) {
  const int chunks = (a.L + kC - 1) / kC;
  bool wide = true, end = false;
  for (int i = 0; i < a.roles; ++i) {
    wide &= a.role[i].Dw % 64 == 0;
    end |= a.role[i].end != nullptr;
  }
  Cut best = {32, 1};
  double least = 1e300;
  for (int SW = 32; SW <= (wide ? 64 : 32); SW += 32) {
    int64_t units = 0;
    for (int i = 0; i < a.roles; ++i) units += static_cast<int64_t>(a.B) * a.H * (a.role[i].Dw / SW);
    for (int parts = 1; parts <= 16 && (parts == 1 || parts * 4 <= chunks); ++parts) {
      const int cpp = (chunks + parts - 1) / parts, sums = end ? parts : parts - 1;
      auto waves = [&](int64_t n) { return static_cast<double>((n + kSMs - 1) / kSMs); };
      double t = waves(units * parts) * (cpp * (SW == 32 ? 1.0 : 1.6) + 4);
      if (sums > 0) t += waves(units * sums) * (cpp * (SW == 32 ? 0.4 : 0.5) + 4);
      if (t < least) least = t, best = {SW, parts};
    }
  }
  return best;
}

}  // namespace

bool ret_tc_supported(const RetArgs &a, Dtype dt) {
  if (dt != kBF16) return false;
  for (int i = 0; i < a.roles; ++i)
    if ((a.role[i].Dx > 64 && a.role[i].Dx != 128) || a.role[i].Dw % 32 != 0) return false;
  return true;
}

int ret_parts_tc(const RetArgs &a) { return cut_of(a).parts; }

cudaError_t launch_retention_tc(const RetArgs &a, int parts, cudaStream_t s) {
  const int chunks = (a.L + kC - 1) / kC, SW = cut_of(a).SW;
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
    p.sectors = true;
    bool end = false;
    for (int i = 0; i < a.roles; ++i) {
      const RetRole &r = a.role[i];
      if ((r.Dx <= 64 ? 64 : 128) != DX) continue;
      TcRole &m = p.map[p.a.roles];
      auto encode = [&](int i, const void *base, int width, int group, const RetStrides &s, int atom, int atoms) {
        return make_tmap_atoms(&m.m[i], base, width, a.H / group, a.L, a.B, s.h, s.t, s.b, atom, atoms, kC);
      };
      if (!encode(0, r.x, r.Dx, r.xg, r.xs, 64, DX / 64) || !encode(1, r.y, r.Dx, r.yg, r.ys, 64, DX / 64) ||
          !encode(2, r.w, r.Dw, r.wg, r.ws, 32, SW / 32))
        return cudaErrorNotSupported;
      p.a.role[p.a.roles++] = r;
      if (r.Dw / SW > p.slices) p.slices = r.Dw / SW;
      if (r.records > p.records) p.records = r.records;
      end |= r.end != nullptr;
      p.sectors &= reinterpret_cast<uintptr_t>(r.o) % 32 == 0 && (r.os.b | r.os.t | r.os.h) % 16 == 0;
    }
    if (!p.a.roles) continue;
    const int64_t units = static_cast<int64_t>(a.B) * a.H * p.slices;
    if (units * parts >= (1LL << 31)) return cudaErrorNotSupported;
    cudaError_t e;
    if (SW == 64) e = DX == 64 ? go<64, 64>(p, end, units, s) : go<128, 64>(p, end, units, s);
    else e = DX == 64 ? go<64, 32>(p, end, units, s) : go<128, 32>(p, end, units, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace linattn
