// Beam search over decode states: the n best continuations of each request,
// and the states' reordering.
//
// Selection.  A continuation (k, v) of request b scores
//   scores[k] + logits[k][v] - log sum_u exp(logits[k][u]),
// computed as the score less the log of the sum relative to the row's maximum, plus
// the logit's distance from the maximum.  Within a beam the order of continuations is
// the order of its logits, so one pass over the logits serves: each CTA takes a piece
// of a row that fits its registers and leaves the piece's maximum, its sum of
// exponentials relative to that, and its n largest logits in order (ties: lowest index
// first).  A second kernel, one CTA per request, joins the sums in 64 bits and takes the n
// best of the sorted lists.  Bound by HBM (the logits are read once) with one
// exponential per logit beside it (16 a clock and SM).
//
// The n largest of a piece: the n-th largest of the maxima of 32 or 128 groups of
// threads bounds the n-th largest value from below, and what is not below that
// bound is collected, in expectation little more than n values (with the maxima of
// all 256 threads, ranked by all of them, a piece took five times as long).  Many equal
// logits can be more than the buffer holds; then the list is taken value by
// value (n rounds of a maximum over the CTA).
//
// Measured, 256 requests x 4 beams x 32000 bf16, n = 8 (65.5 MB of logits, 9.6 us
// at the copy rate): 33 us, of them 25 in the pieces (32% of DRAM, half of the issue
// slots: five CTAs an SM, each a chain of load, maximum, bound, collection) and the
// rest in the join, 256 CTAs of which each waits at its barriers.  One request x 4 x
// 131071 fp32: 12 us in a graph, 26 launched one by one.
//
// Reordering.  A thread has one position (16 bytes where sizes allow) of the
// states of all K beams of a request: it loads the parents' before it stores
// any, so the states move in place, without a second buffer and without a
// barrier; beams that keep their own state are neither read nor written.  Bound by
// HBM: 32 x 4 beams, 361 MB in 59-64 us (83-90% of the copy rate).
#include <float.h>

#include "common.cuh"
#include "dependent.cuh"
#include "kernels.h"
#include "mixer_common.cuh"

namespace linattn {
namespace {

constexpr int kThreads = 256;
constexpr int kKept = 512;  // values collected of a piece

// Values in the order of their logits: larger keys first.  A NaN sorts anywhere
// (its row has no continuations).
__device__ __forceinline__ bool ahead(float a, int ia, float b, int ib) { return a > b || (a == b && ia < ib); }

// What a piece leaves: its n largest logits and their places (n padded to an
// even number), its maximum and its sum.
struct Piece {
  float *value;  // [pieces][n]
  int *index;    // [pieces][n]
  float2 *sum;   // [pieces] (maximum, sum of exp(x - maximum))
};

struct SelectParams {
  BeamArgs a;
  Piece out;
  int pieces;  // of a row
};

// 16 bytes of logits: how many, the pattern of -inf, their values, and how they are
// loaded from where a row off the 16-byte boundary has them (each word of 4 bytes;
// four lanes share a sector, which L1 holds between the loads).  over: the words
// reach over the group's ends, by one value of the row each way.  some: the first n
// values of a group alone, one by one.
template <typename T>
struct vec16;
template <>
struct vec16<float> {
  static constexpr int kN = 4;
  static constexpr uint32_t kNone = 0xff800000u;
  static __device__ __forceinline__ void get(const uint4 &v, float *x) {
    x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ bool over(const float *) { return false; }
  static __device__ __forceinline__ uint4 load(const float *p, bool aligned) {
    if (aligned) return __ldcs(reinterpret_cast<const uint4 *>(p));
    const uint32_t *w = reinterpret_cast<const uint32_t *>(p);
    return make_uint4(__ldg(w), __ldg(w + 1), __ldg(w + 2), __ldg(w + 3));
  }
  static __device__ __noinline__ uint4 some(const float *p, int n) {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(p);
    return make_uint4(w[0], n > 1 ? w[1] : kNone, n > 2 ? w[2] : kNone, n > 3 ? w[3] : kNone);
  }
};
template <>
struct vec16<__nv_bfloat16> {
  static constexpr int kN = 8;
  static constexpr uint32_t kNone = 0xff80ff80u;
  static __device__ __forceinline__ void get(const uint4 &v, float *x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ bool over(const __nv_bfloat16 *p) { return reinterpret_cast<uintptr_t>(p) % 4 != 0; }
  static __device__ __forceinline__ uint4 load(const __nv_bfloat16 *p, bool aligned) {
    if (!over(p)) return vec16<float>::load(reinterpret_cast<const float *>(p), aligned);
    const uint32_t *w = reinterpret_cast<const uint32_t *>(p - 1);
    uint32_t a[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) a[i] = __ldg(w + i);
    return make_uint4(__funnelshift_r(a[0], a[1], 16), __funnelshift_r(a[1], a[2], 16),
                      __funnelshift_r(a[2], a[3], 16), __funnelshift_r(a[3], a[4], 16));
  }
  static __device__ __noinline__ uint4 some(const __nv_bfloat16 *p, int n) {
    const uint16_t *w = reinterpret_cast<const uint16_t *>(p);
    uint32_t a[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      a[i] = (2 * i < n ? w[2 * i] : kNone & 0xffffu) | (2 * i + 1 < n ? w[2 * i + 1] : kNone & 0xffffu) << 16;
    return make_uint4(a[0], a[1], a[2], a[3]);
  }
};

// The groups of a row off the 16-byte boundary, from the aligned 16 bytes in which
// they begin: each lane takes what is missing from the next lane, lane 31 from the
// first lane of the next warp (edge[8 g]).  WS whole words in front of the group and
// `bits`, 0 or 16, more.
template <int WS, int G>
__device__ __forceinline__ void shift_groups(uint4 (&raw)[G], const uint4 *edge, int lane, int bits) {
#pragma unroll
  for (int g = 0; g < G; ++g) {
    uint32_t w[8] = {raw[g].x, raw[g].y, raw[g].z, raw[g].w};
#pragma unroll
    for (int j = 0; j <= WS; ++j) {
      w[4 + j] = __shfl_down_sync(~0u, w[j], 1);
      if (lane == 31) w[4 + j] = reinterpret_cast<const uint32_t *>(edge + 8 * g)[j];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) w[WS + j] = __funnelshift_r(w[WS + j], w[WS + j + 1], bits);
    raw[g] = make_uint4(w[WS], w[WS + 1], w[WS + 2], w[WS + 3]);
  }
}

// A piece is VALUES values per thread, in groups of 16 bytes dealt out to the
// threads in turn from the row's first value on, wherever that lies: rows of the
// same logits have the same sums to the last bit, so that equal beams tie.
template <typename T, int VALUES>
__global__ void __launch_bounds__(kThreads, 5) beams_piece_kernel(const __grid_constant__ SelectParams p) {
  constexpr int kN = vec16<T>::kN, kGroups = VALUES / kN;
  __shared__ float top[128];
  __shared__ float kept[kKept];
  __shared__ int place[kKept];
  // rows off the boundary: bf16 by aligned loads and a shift (64 x 16 x 50257, cold:
  // 64 us, in words 70), fp32 in words (73; the shift spills: 86).  In a graph 56.5 us
  // and 64.0, against 52.3 and 53.7 of V = 50256
  constexpr bool kShift = sizeof(T) == 2;
  __shared__ uint4 edges[kShift ? 8 * kGroups + 1 : 1];  // what each warp's first lane loads
  __shared__ float warp_max[kThreads / 32], warp_sum[kThreads / 32], bound;
  __shared__ int count;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int piece = blockIdx.x % p.pieces;
  const int64_t row = blockIdx.x / p.pieces;
  const T *x = static_cast<const T *>(p.a.logits) + row * p.a.ld;
  const int skew = static_cast<int>(reinterpret_cast<uintptr_t>(x) % 16);  // bytes behind the boundary
  const int V = p.a.V, n = p.a.n;
  const int base = piece * (kThreads * VALUES);  // of this piece in the row (V is at most 2^30)
  if (tid == 0) count = 0;
  // all loads under way before the first value is used
  uint4 raw[kGroups];
  auto at = [&](int g) { return base + (g * kThreads + tid) * kN; };
  if (skew == 0 && base + kThreads * VALUES <= V) {
#pragma unroll
    for (int g = 0; g < kGroups; ++g) raw[g] = __ldcs(reinterpret_cast<const uint4 *>(x + at(g)));
  } else if (kShift && skew != 0 && (base > 0 || row > 0) && base + kThreads * VALUES + kN <= V) {
    // from the boundary in front of the piece to the one behind it: all of the tensor
    if constexpr (kShift) {
      const T *from = x - skew / static_cast<int>(sizeof(T));
      if (tid == 0) edges[8 * kGroups] = __ldg(reinterpret_cast<const uint4 *>(from + base + kThreads * VALUES));
#pragma unroll
      for (int g = 0; g < kGroups; ++g) raw[g] = __ldcs(reinterpret_cast<const uint4 *>(from + at(g)));
      if (lane == 0)
#pragma unroll
        for (int g = 0; g < kGroups; ++g) edges[8 * g + warp] = raw[g];
      __syncthreads();
      const int bits = skew % 4 * 8;
      if (skew < 4) shift_groups<0>(raw, edges + warp + 1, lane, bits);
      else if (skew < 8) shift_groups<1>(raw, edges + warp + 1, lane, bits);
      else if (skew < 12) shift_groups<2>(raw, edges + warp + 1, lane, bits);
      else shift_groups<3>(raw, edges + warp + 1, lane, bits);
    }
  } else {
    // a piece at the row's end, or in words: groups across the row's end (loaded in
    // words that reach over theirs: at either end) value by value, behind the others
    const bool over = vec16<T>::over(x);
    auto whole = [&](int g) { return at(g) >= over && at(g) + kN + over <= V; };
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      raw[g] = make_uint4(vec16<T>::kNone, vec16<T>::kNone, vec16<T>::kNone, vec16<T>::kNone);
      if (whole(g)) raw[g] = vec16<T>::load(x + at(g), skew == 0);
    }
#pragma unroll
    for (int g = 0; g < kGroups; ++g)
      if (!whole(g) && at(g) < V) raw[g] = vec16<T>::some(x + at(g), V - at(g));
  }
  float v[VALUES], most[kGroups], m = -INFINITY;
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    vec16<T>::get(raw[g], v + g * kN);
    most[g] = v[g * kN];
#pragma unroll
    for (int i = 1; i < kN; ++i) most[g] = fmaxf(most[g], v[g * kN + i]);
    m = fmaxf(m, most[g]);
  }
  // maxima of groups of 8 threads (n up to 32) or 2: 32 or 128 groups
  const bool few = n <= 32;
  float gm = fmaxf(m, __shfl_xor_sync(~0u, m, 1));
  if (few) {
    gm = fmaxf(gm, __shfl_xor_sync(~0u, gm, 2));
    gm = fmaxf(gm, __shfl_xor_sync(~0u, gm, 4));
  }
  if ((tid & (few ? 7 : 1)) == 0) top[tid >> (few ? 3 : 1)] = gm;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) gm = fmaxf(gm, __shfl_xor_sync(~0u, gm, o));
  if (lane == 0) warp_max[warp] = gm;
  __syncthreads();
  float all = warp_max[0];
#pragma unroll
  for (int i = 1; i < kThreads / 32; ++i) all = fmaxf(all, warp_max[i]);
  float least;
  if (few) {
    // every warp sorts the 32 maxima over its lanes: no warp waits for another
    float own = top[lane];
#pragma unroll
    for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
      for (int j = k >> 1; j > 0; j >>= 1) {
        const float other = __shfl_xor_sync(~0u, own, j);
        const bool larger = ((lane & j) == 0) == ((lane & k) == 0 || k == 32);
        own = larger ? fmaxf(own, other) : fminf(own, other);
      }
    least = __shfl_sync(~0u, own, n - 1);
  } else {
    if (tid < 128) {  // rank of a group's maximum among the groups'
      const float own = top[tid];
      int rank = 0;
      for (int i = 0; i < 128; ++i) rank += ahead(top[i], i, own, tid);
      if (rank == n - 1) bound = own;
    }
    __syncthreads();
    least = bound;
  }
  least = fmaxf(least, -FLT_MAX);  // -inf is no continuation
  f2 sums = dup2(0.f);
  if (all > -INFINITY) {
    // the difference first: it is exact where it matters, near the maximum
    const f2 off = dup2(-all), l2e = dup2(kLog2e);
#pragma unroll
    for (int i = 0; i < VALUES; i += 2) sums = add2(sums, ex2_2(mul2(add2(pack2(v[i], v[i + 1]), off), l2e)));
  }
  float sum = sum2(sums);
  if (!(all > -INFINITY)) {
#pragma unroll
    for (int i = 0; i < VALUES; ++i)
      if (v[i] != v[i]) sum = v[i];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
  if (lane == 0) warp_sum[warp] = sum;
  if (m >= least) {  // few threads
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      if (!(most[g] >= least)) continue;
#pragma unroll
      for (int i = 0; i < kN; ++i)
        if (v[g * kN + i] >= least) {
          const int to = atomicAdd(&count, 1);
          if (to < kKept) {
            kept[to] = v[g * kN + i];
            place[to] = at(g) + i;
          }
        }
    }
  }
  __syncthreads();
  float *value = p.out.value + static_cast<int64_t>(blockIdx.x) * n;
  int *index = p.out.index + static_cast<int64_t>(blockIdx.x) * n;
  const int found = count;
  if (found <= kKept) {
    for (int i = tid; i < found; i += kThreads) {
      const float a = kept[i];
      const int ia = place[i];
      int r = 0;
      for (int j = 0; j < found; ++j) r += ahead(kept[j], place[j], a, ia);
      if (r < n) {
        value[r] = a;
        index[r] = ia;
      }
    }
    for (int i = found + tid; i < n; i += kThreads) {
      value[i] = -INFINITY;
      index[i] = -1;
    }
  } else {
    // value by value: the largest behind the last one taken
    float last = INFINITY;
    int at_last = -1;
    for (int r = 0; r < n; ++r) {
      float best = -INFINITY;
      int at_best = 0x7fffffff;
#pragma unroll
      for (int g = 0; g < kGroups; ++g)
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          const int here = at(g) + i;
          const float a = v[g * kN + i];
          if (ahead(last, at_last, a, here) && ahead(a, here, best, at_best)) best = a, at_best = here;
        }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float a = __shfl_xor_sync(~0u, best, o);
        const int there = __shfl_xor_sync(~0u, at_best, o);
        if (ahead(a, there, best, at_best)) best = a, at_best = there;
      }
      __syncthreads();
      if (lane == 0) kept[warp] = best, place[warp] = at_best;
      __syncthreads();
      last = kept[0], at_last = place[0];
#pragma unroll
      for (int i = 1; i < kThreads / 32; ++i)
        if (ahead(kept[i], place[i], last, at_last)) last = kept[i], at_last = place[i];
      if (tid == 0) {
        value[r] = last;
        index[r] = last > -INFINITY ? at_last : -1;
      }
    }
  }
  if (tid == 0) {
    float t = 0.f;
    for (int i = 0; i < kThreads / 32; ++i) t += warp_sum[i];
    p.out.sum[blockIdx.x] = make_float2(all, t);
  }
  let_next_start();
}

// A score as an integer of the same order (fp64 comparisons are slow here).
__device__ __forceinline__ int64_t key_of(double v) {
  const int64_t k = __double_as_longlong(v + 0.0);
  return k < 0 ? k ^ INT64_MAX : k;
}
__device__ __forceinline__ double score_of(int64_t key) { return __longlong_as_double(key < 0 ? key ^ INT64_MAX : key); }

// log t to about 2^-23, absolutely: the fp32 logarithm, off by its own rounding,
// and one step of Newton's method (64-bit logarithms take microseconds here).
__device__ __forceinline__ double log_of(double t) {
  const float tf = static_cast<float>(t), y = logf(tf);
  return static_cast<double>(y) + fmaf(tf, expf(-y), -1.f);
}

constexpr int kCand = 1024;  // candidates of a request that are ranked at once
constexpr int kMaxBeams = 32;
constexpr int kHeld = 2048;  // entries of lists that shared memory holds

// A continuation: its score's key, and beam and token as one number of the
// order in which ties go.
struct Cand {
  int64_t key, at;
};
__device__ __forceinline__ bool ahead(const Cand &a, const Cand &b) {
  return a.key > b.key || (a.key == b.key && a.at < b.at);
}

// The n best of a request's lists.  Rows first: the log of each row's sum relative
// to its maximum, and with it the offset score - log in 64 bits (-inf for a row that
// offers nothing), to which a logit's distance from the maximum is added (a row of
// the type's lowest value would swallow score and log, were they added to the
// logits).  Then the first entries of the lists, one per thread, of which the
// n-th largest bounds the n-th best continuation; and the candidates that are
// not below it, ranked.
__global__ void __launch_bounds__(kThreads) beams_join_kernel(const __grid_constant__ SelectParams p) {
  __shared__ double offset[kMaxBeams], lse[kMaxBeams];
  __shared__ float most[kMaxBeams];
  __shared__ uint8_t done[kMaxBeams];
  __shared__ Cand cand[kCand];
  __shared__ int64_t heads[kThreads];
  __shared__ Cand best[kThreads / 32];
  __shared__ int64_t bound;
  __shared__ int count;
  __shared__ float held_value[kHeld];
  __shared__ int held_index[kHeld];
  const int K = p.a.K, n = p.a.n, pieces = p.pieces, lists = K * pieces;
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t first = static_cast<int64_t>(b) * lists;
  const int64_t nothing = key_of(-INFINITY);
  if (tid == 0) count = 0;
  // what the pass before does not write, ahead of the wait for it
  const float own_score = tid < K ? p.a.scores[static_cast<int64_t>(b) * K + tid] : 0.f;
  const bool own_done = tid < K && p.a.finished && p.a.finished[static_cast<int64_t>(b) * K + tid];
  wait_for_previous();
  const bool held = lists * n <= kHeld;
  if (held)
    for (int i = tid; i < lists * n; i += kThreads) {
      held_value[i] = p.out.value[first * n + i];
      held_index[i] = p.out.index[first * n + i];
    }
  if (tid < K) done[tid] = own_done;
  for (int k = warp; k < K; k += kThreads / 32) {
    const float2 *s = p.out.sum + first + static_cast<int64_t>(k) * pieces;
    float m = -INFINITY;
    for (int i = lane; i < pieces; i += 32) m = fmaxf(m, s[i].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
    double t = 0.0;
    for (int i = lane; i < pieces; i += 32) {
      const float2 x = s[i];
      // a piece of -inf alone adds nothing, one with NaN its NaN
      t += x.x > -INFINITY ? x.y * expf(x.x - m) : x.y;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(~0u, t, o);
    if (lane == 0) lse[k] = log_of(t), most[k] = m;
  }
  __syncthreads();
  if (tid < K) {
    const double l = own_done ? 0.0 : lse[tid];
    if (own_done) most[tid] = 0.f;
    offset[tid] = isfinite(own_score) && isfinite(l) && isfinite(most[tid]) ? own_score - l : -INFINITY;
  }
  __syncthreads();
  // entry i of list l (a finished beam has one, its end token at no cost, in
  // its first list)
  auto entry = [&](int l, int i) -> Cand {
    const int k = l / pieces;
    const double off = offset[k];
    if (!(off > -INFINITY)) return {nothing, INT64_MAX};
    const int64_t row = static_cast<int64_t>(k) << 32;
    if (done[k]) return l == k * pieces && i == 0 ? Cand{key_of(off), row | p.a.eos} : Cand{nothing, INT64_MAX};
    const int in = l * n + i;
    const int v = held ? held_index[in] : p.out.index[first * n + in];
    if (v < 0) return {nothing, INT64_MAX};
    const double below = static_cast<double>(held ? held_value[in] : p.out.value[first * n + in]) - most[k];
    return {key_of(off + below), row | v};
  };
  // one entry per thread: so deep into the lists that there are 4 n, or the best
  // head of several lists
  int64_t mine = nothing;
  int some = kThreads;
  if (lists < kThreads) {
    const int deep = min(min(n, (4 * n + lists - 1) / lists), kThreads / lists);
    some = max(lists * deep, n);
    if (tid < lists * deep) mine = entry(tid % lists, tid / lists).key;
  } else {
    for (int l = tid; l < lists; l += kThreads) {
      const int64_t h = entry(l, 0).key;
      if (h > mine) mine = h;
    }
  }
  heads[tid] = mine;
  __syncthreads();
  if (tid < some) {
    int rank = 0;
    for (int i = 0; i < some; ++i) rank += heads[i] > mine || (heads[i] == mine && i < tid);
    if (rank == n - 1) bound = mine;
  }
  __syncthreads();
  const int64_t least = bound;
  for (int l = tid; l < lists; l += kThreads)
    for (int i = 0; i < n; ++i) {
      const Cand c = entry(l, i);
      if (c.key == nothing || c.key < least) break;
      const int to = atomicAdd(&count, 1);
      if (to < kCand) cand[to] = c;
    }
  __syncthreads();
  const int found = count;
  const int64_t out = static_cast<int64_t>(b) * n;
  auto put = [&](int r, const Cand &c) {
    const bool any = c.key != nothing;
    p.a.out_scores[out + r] = static_cast<float>(score_of(c.key));
    p.a.parents[out + r] = any ? static_cast<int>(c.at >> 32) : -1;
    p.a.tokens[out + r] = any ? static_cast<int>(c.at & 0xffffffff) : -1;
  };
  if (found <= kCand) {
    for (int i = tid; i < found; i += kThreads) {
      const Cand c = cand[i];
      int r = 0;
      for (int j = 0; j < found; ++j) r += ahead(cand[j], c);
      if (r < n) put(r, c);
    }
    for (int i = found + tid; i < n; i += kThreads) put(i, {nothing, 0});
    return;
  }
  // more equal scores than the buffer holds: one continuation after another
  Cand last = {INT64_MAX, -1};
  for (int r = 0; r < n; ++r) {
    Cand mx = {nothing, INT64_MAX};
    for (int l = tid; l < lists; l += kThreads)
      for (int i = 0; i < n; ++i) {
        const Cand c = entry(l, i);
        if (c.key == nothing) break;
        if (ahead(last, c) && ahead(c, mx)) mx = c;
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const Cand c = {__shfl_xor_sync(~0u, mx.key, o), __shfl_xor_sync(~0u, mx.at, o)};
      if (ahead(c, mx)) mx = c;
    }
    __syncthreads();
    if (lane == 0) best[warp] = mx;
    __syncthreads();
    last = best[0];
    for (int i = 1; i < kThreads / 32; ++i)
      if (ahead(best[i], last)) last = best[i];
    if (tid == 0) put(r, last);
  }
}

// Values per thread: long pieces where there are rows enough to fill the card,
// short ones where the pieces of a few rows have to.
int values_of(int64_t rows, int V) { return rows * ((V + 8191) / 8192) >= 2 * kSMs ? 32 : 8; }

int pieces_of(int64_t rows, int V) {
  const int piece = kThreads * values_of(rows, V);
  return (V + piece - 1) / piece;
}

// --- reordering ---

struct ReorderParams {
  void *state[kReorderStates];
  int64_t words[kReorderStates];  // of a beam
  const int *parents;
  int B, K;
};

template <typename W, int KMAX>
__global__ void __launch_bounds__(kThreads) reorder_kernel(const __grid_constant__ ReorderParams p) {
  __shared__ int parent[KMAX];
  const int K = p.K;
  const int64_t words = p.words[blockIdx.z];
  for (int b = blockIdx.y; b < p.B; b += gridDim.y) {
    int from = threadIdx.x;
    if (threadIdx.x < K) {
      const int named = p.parents[static_cast<int64_t>(b) * K + threadIdx.x];
      if (named >= 0 && named < K) from = named;
      parent[threadIdx.x] = from;
    }
    const bool moves = __syncthreads_or(from != threadIdx.x);
    W *state = static_cast<W *>(p.state[blockIdx.z]) + static_cast<int64_t>(b) * K * words;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; moves && i < words;
         i += static_cast<int64_t>(gridDim.x) * kThreads) {
      W v[KMAX];
#pragma unroll
      for (int k = 0; k < KMAX; ++k)
        if (k < K && parent[k] != k) v[k] = state[parent[k] * words + i];
#pragma unroll
      for (int k = 0; k < KMAX; ++k)
        if (k < K && parent[k] != k) state[k * words + i] = v[k];
    }
    __syncthreads();  // the next request's parents
  }
}

template <typename W>
cudaError_t reorder(const ReorderParams &p, int count, int B, int64_t most, cudaStream_t s) {
  int64_t x = (most + kThreads - 1) / kThreads;
  // a few waves of CTAs at most: a thread then walks several positions
  const int64_t enough = (32 * kSMs + static_cast<int64_t>(B) * count - 1) / (static_cast<int64_t>(B) * count);
  if (x > enough) x = enough;
  const dim3 grid(static_cast<unsigned>(x), static_cast<unsigned>(B < 65535 ? B : 65535), static_cast<unsigned>(count));
  if (p.K <= 4) reorder_kernel<W, 4><<<grid, kThreads, 0, s>>>(p);
  else if (p.K <= 8) reorder_kernel<W, 8><<<grid, kThreads, 0, s>>>(p);
  else if (p.K <= 16) reorder_kernel<W, 16><<<grid, kThreads, 0, s>>>(p);
  else reorder_kernel<W, 32><<<grid, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

size_t beams_workspace_bytes(int B, int K, int V, int n) {
  const int64_t rows = static_cast<int64_t>(B) * K;
  return static_cast<size_t>(rows * pieces_of(rows, V)) * (sizeof(float2) + 8 * static_cast<size_t>(n));
}

cudaError_t launch_select_beams(const BeamArgs &a, Dtype dt, void *ws, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(a.B) * a.K;
  SelectParams p = {a, {}, pieces_of(rows, a.V)};
  const int64_t all = rows * p.pieces;
  if (all >= (1LL << 31)) return cudaErrorNotSupported;
  p.out.sum = static_cast<float2 *>(ws);
  p.out.value = reinterpret_cast<float *>(p.out.sum + all);
  p.out.index = reinterpret_cast<int *>(p.out.value + all * a.n);
  const bool big = values_of(rows, a.V) == 32;
  const unsigned grid = static_cast<unsigned>(all);
  if (dt == kF32) {
    if (big) beams_piece_kernel<float, 32><<<grid, kThreads, 0, s>>>(p);
    else beams_piece_kernel<float, 8><<<grid, kThreads, 0, s>>>(p);
  } else {
    if (big) beams_piece_kernel<__nv_bfloat16, 32><<<grid, kThreads, 0, s>>>(p);
    else beams_piece_kernel<__nv_bfloat16, 8><<<grid, kThreads, 0, s>>>(p);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_dependent(beams_join_kernel, static_cast<unsigned>(a.B), 1, kThreads, 0, s, p);
}

cudaError_t launch_reorder_states(void *const *states, const int64_t *bytes, int count, const int *parents, int B,
                                  int K, cudaStream_t s) {
  // 16-byte words where a state's size and place allow them, else 4-byte ones,
  // else bytes; one launch for each of these that occurs
  ReorderParams p = {};
  p.parents = parents;
  p.B = B;
  p.K = K;
  for (const int w : {16, 4, 1}) {
    int m = 0;
    int64_t most = 0;
    for (int i = 0; i < count; ++i) {
      int own = 16;
      while (own > 1 && (bytes[i] % own != 0 || reinterpret_cast<uintptr_t>(states[i]) % own != 0))
        own = own == 16 ? 4 : 1;
      if (own != w || bytes[i] == 0) continue;
      p.state[m] = states[i];
      p.words[m] = bytes[i] / w;
      if (p.words[m] > most) most = p.words[m];
      ++m;
    }
    if (m) {
      const cudaError_t e = w == 16  ? reorder<uint4>(p, m, B, most, s)
                            : w == 4 ? reorder<uint32_t>(p, m, B, most, s)
                                     : reorder<uint8_t>(p, m, B, most, s);
      if (e != cudaSuccess) return e;
    }
  }
  return cudaSuccess;
}

}  // namespace linattn
