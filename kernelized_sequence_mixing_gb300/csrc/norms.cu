// RMS norms around a mixing block, forward and backward (fp32 arithmetic).
//
// After the block, per (b, t, h) row of D values (the heads of a causal
// linear-attention pass, or the groups of a state space block):
//   gate after:  o = p rsqrt(mean p^2 + eps) w act(g),   p = y
//   gate first:  o = p rsqrt(mean p^2 + eps) w,          p = y act(g)
// with act = SiLU.  y is read where the block left it ([B][H][L][D] or
// [B][L][H][D]) and o is written token-major, as the projection behind it
// reads it.  Ahead of the next block, per row of E values:
//   r = residual + scale x,   o = r rsqrt(mean r^2 + eps) w
// (the norm takes the fp32 sum, not the rounded r that is written beside it).
//
// Backward.  With n = p rstd and dn = do w (act(g)):
//   dp = rstd (dn - n mean(dn n)) = rstd dn - p rstd^3 sum(dn p) / D,
// so one joint reduction of sum p^2 and sum dn p serves a row (rstd^3 alone
// leaves the fp32 range long before its product with the sum does).
//
// Bound by memory: every value is read once into registers and written once.
// A row belongs to a power of two of lanes, 8 values a lane at a time: part
// of a warp up to D = 128, a warp up to 1024, a CTA beyond.  The backward
// passes keep a row group on one head, so the weight gradient stays in
// registers over all its rows and leaves as one record per CTA; the records
// are added in their order.
#include <type_traits>

#include "dependent.cuh"
#include "kernels.h"
#include "mixer_common.cuh"

namespace linattn {
namespace {

constexpr int kThreads = 256;

enum { kGateAfter = 0, kGateFirst = 1, kResidual = 2 };

struct RowArgs {
  const void *in1, *in2;  // y and gate, or x and residual (backward: r and nothing)
  const void *in3, *in4;  // backward: do; dr
  const float *w;
  void *out1, *out2;      // o and r; backward: dy and dgate, or dresidual and dx
  float *rec;             // backward: [slots][H][D] weight gradients, or null
  unsigned tokens;        // B L (residual: rows); tokens x H < 2^31
  int H, D, L;
  float eps, scale;
  bool heads_first;
  int hs;                 // a CTA's rows are 2^hs heads (which divide H) of its tokens
};

// Where token j (of batch entry b, at t in it) of head h lies: in y, and in the
// token-major tensors.  Rows count less than 2^31.
struct Row {
  unsigned j, b, t;
  int h;
  __device__ __forceinline__ int64_t off(const RowArgs &a) const {
    return (int64_t)(j * a.H + h) * a.D;
  }
  __device__ __forceinline__ int64_t y_off(const RowArgs &a) const {
    return a.heads_first ? ((int64_t)(b * a.H + h) * a.L + t) * a.D : off(a);
  }
};

// Sum over a row's LANES lanes (LANES = kThreads: the CTA; `sh` has room for
// two rounds, `round` alternates so that one barrier per sum is enough).
template <int LANES, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float (*sh)[K][kThreads / 32], int &round) {
#pragma unroll
  for (int o = (LANES < 32 ? LANES : 32) / 2; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if constexpr (LANES > 32) {
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) sh[round][k][warp] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < LANES / 32; ++i) s += sh[round][k][i];
      v[k] = s;
    }
    round ^= 1;
  }
}

// CTAs go over the head blocks first.  The divisions are the CTA's: a thread
// steps from its first token.
template <typename T, int MODE, int LANES, int VPT>
__global__ void __launch_bounds__(kThreads) norm_kernel(const __grid_constant__ RowArgs a) {
  constexpr int GPC = kThreads / LANES;
  constexpr int R = VPT == 1 && LANES < 256 ? 2 : 1;  // rows per group, loaded together
  __shared__ float sh[2][1][kThreads / 32];
  int round = 0;
  const float invD = 1.f / a.D;
  const int lane = threadIdx.x % LANES, grp = threadIdx.x / LANES;
  raw8<T> rp[R][VPT], rg[R][VPT];
  int64_t off[R];
  bool live[R];
  const unsigned hblocks = (unsigned)a.H >> a.hs;
  const unsigned tb = hblocks == 1 ? blockIdx.x : blockIdx.x / hblocks;
  const unsigned j0 = tb * (GPC * R >> a.hs);
  const unsigned b0 = MODE == kResidual ? 0u : j0 / (unsigned)a.L, i0 = j0 - b0 * (unsigned)a.L;
  const int h = static_cast<int>(((blockIdx.x - tb * hblocks) << a.hs) + (grp & ((1 << a.hs) - 1)));
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const unsigned step = (grp >> a.hs) + r * (GPC >> a.hs);
    Row row = {j0 + step, b0, i0 + step, h};
    if (MODE != kResidual)
      while (row.t >= (unsigned)a.L) {
        row.t -= a.L;
        ++row.b;
      }
    live[r] = row.j < a.tokens;
    off[r] = live[r] ? row.off(a) : 0;
    const T *in1 = static_cast<const T *>(a.in1) +
                   (MODE == kResidual || !live[r] ? off[r] : row.y_off(a));
    const T *in2 = static_cast<const T *>(a.in2) + off[r];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = (v * LANES + lane) * 8;
      rp[r][v].zero();
      rg[r][v].zero();
      if (live[r] && c < a.D) {
        rp[r][v].load(in1 + c);
        if (MODE != kResidual || a.in2) rg[r][v].load(in2 + c);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    f2 p[VPT][4], g[VPT][4], s2 = dup2(0.f);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      rp[r][v].getp(p[v]);
      rg[r][v].getp(g[v]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (MODE == kResidual) {
          p[v][i] = fma2(dup2(a.scale), p[v][i], g[v][i]);
        } else {
          g[v][i] = mul2(g[v][i], sigmoid_f2(g[v][i]));
          if (MODE == kGateFirst) p[v][i] = mul2(p[v][i], g[v][i]);
        }
        s2 = fma2(p[v][i], p[v][i], s2);
      }
    }
    float s[1] = {sum2(s2)};
    row_sum<LANES, 1>(s, sh, round);
    const f2 rstd = dup2(rsqrtf(fmaf(s[0], invD, a.eps)));
    if (!live[r]) continue;
    T *o = static_cast<T *>(a.out1) + off[r];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = (v * LANES + lane) * 8;
      if (c < a.D) {
        if (MODE == kResidual) store8p(static_cast<T *>(a.out2) + off[r] + c, p[v]);
        f2 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = dup2(1.f);
        if (a.w) load8p(a.w + (int64_t)h * a.D + c, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          w[i] = mul2(w[i], mul2(p[v][i], rstd));
          if (MODE == kGateAfter) w[i] = mul2(w[i], g[v][i]);
        }
        store8p(o + c, w);
      }
    }
  }
}

// 2^hs heads per CTA; its row groups stride over the tokens.
template <typename T, int MODE, int LANES, int VPT>
__global__ void __launch_bounds__(kThreads)
    norm_bwd_kernel(const __grid_constant__ RowArgs a, int slots) {
  let_next_start();
  constexpr int GPC = kThreads / LANES;
  __shared__ float sh[2][2][kThreads / 32];
  int round = 0;
  const int lane = threadIdx.x % LANES, grp = threadIdx.x / LANES;
  const unsigned hblocks = (unsigned)a.H >> a.hs, slot = blockIdx.x / hblocks;
  const int h0 = static_cast<int>((blockIdx.x - slot * hblocks) << a.hs);
  const int h = h0 + (grp & ((1 << a.hs) - 1));
  const unsigned tpc = GPC >> a.hs;  // tokens of a turn
  f2 w[VPT][4], dw[VPT][4];
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = (v * LANES + lane) * 8;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[v][i] = dup2(1.f);
      dw[v][i] = dup2(0.f);
    }
    if (a.w && c < a.D) load8p(a.w + (int64_t)h * a.D + c, w[v]);
  }
  const float invD = 1.f / a.D;
  // a turn's rows as they lie in memory, loaded one turn ahead where a row is
  // one vector per lane
  struct Rows {
    raw8<T> y[VPT], g[VPT], d[VPT];  // g: the gate, or dr
    int64_t off, yoff;
    bool live;
  };
  const unsigned stride = slots * tpc;
  Row row = {slot * tpc + (grp >> a.hs), 0u, 0u, h};
  unsigned stride_b = 0, stride_t = 0;
  if (MODE != kResidual) {
    row.b = row.j / (unsigned)a.L;
    row.t = row.j - row.b * (unsigned)a.L;
    stride_b = stride / (unsigned)a.L;
    stride_t = stride - stride_b * (unsigned)a.L;
  }
  auto fetch = [&](Rows &r) {  // the next row of this group
    r.live = row.j < a.tokens;
    r.off = r.live ? row.off(a) : 0;
    r.yoff = MODE == kResidual || !r.live ? r.off : row.y_off(a);
    row.j += stride;
    if (MODE != kResidual) {
      row.b += stride_b;
      row.t += stride_t;
      if (row.t >= (unsigned)a.L) {
        row.t -= a.L;
        ++row.b;
      }
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = (v * LANES + lane) * 8;
      r.y[v].zero();
      r.g[v].zero();
      r.d[v].zero();
      if (r.live && c < a.D) {
        r.y[v].load(static_cast<const T *>(a.in1) + r.yoff + c);
        r.d[v].load(static_cast<const T *>(a.in3) + r.off + c);
        if (MODE == kResidual) {
          if (a.in4) r.g[v].load(static_cast<const T *>(a.in4) + r.off + c);
        } else {
          r.g[v].load(static_cast<const T *>(a.in2) + r.off + c);
        }
      }
    }
  };
  constexpr bool kPrefetch = VPT == 1;
  Rows cur, nxt;
  if (kPrefetch) fetch(nxt);
  // every group of the CTA makes the same number of turns (the sums cross
  // lanes of several groups)
  for (unsigned j0 = slot * tpc; j0 < a.tokens; j0 += stride) {
    if (kPrefetch) {
      cur = nxt;
      fetch(nxt);
    } else {
      fetch(cur);
    }
    f2 s0 = dup2(0.f), s1 = dup2(0.f);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      f2 y[4], g[4], d[4];
      cur.y[v].getp(y);
      cur.g[v].getp(g);
      cur.d[v].getp(d);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f2 p = y[i], dn = mul2(d[i], w[v][i]);
        if (MODE != kResidual) {
          const f2 act = mul2(g[i], sigmoid_f2(g[i]));
          if (MODE == kGateFirst) p = mul2(p, act);
          else dn = mul2(dn, act);
        }
        s0 = fma2(p, p, s0);
        s1 = fma2(dn, p, s1);
      }
    }
    float s[2] = {sum2(s0), sum2(s1)};
    row_sum<LANES, 2>(s, sh, round);
    const float rs = rsqrtf(fmaf(s[0], invD, a.eps));
    const f2 rstd = dup2(rs), k = dup2(-rs * (rs * (rs * (s[1] * invD))));
    if (cur.live) {
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int c = (v * LANES + lane) * 8;
        if (c < a.D) {
          f2 y[4], g[4], d[4], o1[4], o2[4];
          cur.y[v].getp(y);
          cur.g[v].getp(g);
          cur.d[v].getp(d);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (MODE == kResidual) {
              const f2 n = mul2(y[i], rstd);
              dw[v][i] = fma2(d[i], n, dw[v][i]);
              o1[i] = add2(g[i], fma2(rstd, mul2(d[i], w[v][i]), mul2(k, y[i])));
              o2[i] = mul2(dup2(a.scale), o1[i]);
            } else {
              const f2 sg = sigmoid_f2(g[i]), act = mul2(g[i], sg);
              // silu'(g) = s (1 + g (1 - s))
              const f2 dact = mul2(sg, fma2(g[i], fma2(sg, dup2(-1.f), dup2(1.f)), dup2(1.f)));
              if (MODE == kGateFirst) {
                const f2 p = mul2(y[i], act);
                const f2 dp = fma2(rstd, mul2(d[i], w[v][i]), mul2(k, p));
                dw[v][i] = fma2(d[i], mul2(p, rstd), dw[v][i]);
                o1[i] = mul2(dp, act);
                o2[i] = mul2(mul2(dp, y[i]), dact);
              } else {
                const f2 da = mul2(d[i], act), n = mul2(y[i], rstd);
                dw[v][i] = fma2(da, n, dw[v][i]);
                o1[i] = fma2(rstd, mul2(da, w[v][i]), mul2(k, y[i]));
                o2[i] = mul2(mul2(d[i], n), mul2(w[v][i], dact));
              }
            }
          }
          store8p(static_cast<T *>(a.out1) + cur.yoff + c, o1);
          if (MODE != kResidual || a.out2) store8p(static_cast<T *>(a.out2) + cur.off + c, o2);
        }
      }
    }
  }
  if (!a.rec) return;
  float *rec = a.rec + ((int64_t)slot * a.H + h0) * a.D;
  if constexpr (GPC == 1) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = (v * LANES + lane) * 8;
      if (c < a.D) store8p(rec + c, dw[v]);
    }
  } else {
    // each head's groups, in group order
    __shared__ float part[GPC][LANES * 8];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      __syncthreads();
      store8p(&part[grp][lane * 8], dw[v]);
      __syncthreads();
      const int hb = 1 << a.hs;
      for (int i = threadIdx.x; i < hb * LANES * 8; i += kThreads) {
        const int hh = i / (LANES * 8), k = i % (LANES * 8), c = v * LANES * 8 + k;
        if (c < a.D) {
          float q = part[hh][k];
          for (int g = hh + hb; g < GPC; g += hb) q += part[g][k];
          rec[(int64_t)hh * a.D + c] = q;
        }
      }
    }
  }
}

// Lanes per row: 8 values each up to a warp, then up to 4 vectors per lane,
// then the CTA.
template <typename F>
cudaError_t by_width(int D, F &&f) {
  if (D <= 32) return f(std::integral_constant<int, 4>{}, std::integral_constant<int, 1>{});
  if (D <= 64) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 1>{});
  if (D <= 128) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{});
  if (D <= 256) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 1>{});
  if (D <= 512) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 2>{});
  if (D <= 1024) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 4>{});
  if (D <= 2048) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 1>{});
  if (D <= 4096) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
  return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 4>{});
}

int lanes_of(int D) { return D <= 32 ? 4 : D <= 64 ? 8 : D <= 128 ? 16 : D <= 1024 ? 32 : 256; }

// Heads of a CTA's rows, as a power of two: up to four, as many as divide H
// and fit its groups.
int head_shift(int H, int D) {
  const int gpc = kThreads / lanes_of(D);
  int s = 2;
  while ((1 << s) > gpc || H % (1 << s)) --s;
  return s;
}

// CTAs per head block of a backward pass: about two per SM over all blocks, no
// more than there are rows for.  More of them hide more latency but leave more
// records to add: B4 H8 L4096 D64 takes 16.0, 17.0 and 19.3 us with two, four
// and six, 8191 rows of 2048 take 35.9, 37.8 and 35.2 (bf16, both kernels,
// replayed in a graph: the first case's 84 MB stay in L2 there; its main kernel
// takes 20.6 us with cold caches).
int bwd_slots(int64_t tokens, int H, int D) {
  const int hs = head_shift(H, D), tpc = (kThreads / lanes_of(D)) >> hs, blocks = H >> hs;
  const int64_t most = (tokens + tpc - 1) / tpc;
  int64_t n = (kSMs * 2 + blocks - 1) / blocks;
  if (n > most) n = most;
  return n < 1 ? 1 : static_cast<int>(n);
}

template <typename T, int MODE>
cudaError_t run_rows(const RowArgs &a, cudaStream_t s) {
  return by_width(a.D, [&](auto lanes, auto vpt) {
    constexpr int LANES = decltype(lanes)::value, VPT = decltype(vpt)::value;
    constexpr int R = VPT == 1 && LANES < 256 ? 2 : 1;
    const int tpc = (kThreads / LANES * R) >> a.hs;  // tokens per CTA
    const int64_t ctas = ((int64_t)a.tokens + tpc - 1) / tpc * (a.H >> a.hs);
    norm_kernel<T, MODE, LANES, VPT><<<(unsigned)ctas, kThreads, 0, s>>>(a);
    return cudaGetLastError();
  });
}

template <typename T, int MODE>
cudaError_t run_rows_bwd(const RowArgs &a, float *dw, cudaStream_t s) {
  const int slots = bwd_slots(a.tokens, a.H, a.D);
  cudaError_t e = by_width(a.D, [&](auto lanes, auto vpt) {
    constexpr int LANES = decltype(lanes)::value, VPT = decltype(vpt)::value;
    norm_bwd_kernel<T, MODE, LANES, VPT><<<(unsigned)(slots * (a.H >> a.hs)), kThreads, 0, s>>>(a, slots);
    return cudaGetLastError();
  });
  if (e != cudaSuccess || !dw) return e;
  return launch_column_sum(a.rec, slots, a.H * a.D, dw, a.H * a.D, nullptr, s);
}

RowArgs gate_rows(const NormGateArgs &n) {
  RowArgs a = {};
  a.in1 = n.y;
  a.in2 = n.gate;
  a.w = n.w;
  a.out1 = n.out;
  a.tokens = (unsigned)n.B * (unsigned)n.L;
  a.H = n.H;
  a.D = n.D;
  a.L = n.L;
  a.hs = head_shift(n.H, n.D);
  a.eps = n.eps;
  a.heads_first = n.heads_first;
  return a;
}

RowArgs residual_rows(const NormResidualArgs &n) {
  RowArgs a = {};
  a.w = n.w;
  a.tokens = (unsigned)n.rows;
  a.H = 1;
  a.D = n.E;
  a.L = 1;
  a.hs = 0;
  a.eps = n.eps;
  a.scale = n.scale;
  return a;
}

}  // namespace

cudaError_t launch_norm_gate(const NormGateArgs &n, Dtype dt, cudaStream_t s) {
  const RowArgs a = gate_rows(n);
  if (dt == kF32)
    return n.gate_first ? run_rows<float, kGateFirst>(a, s) : run_rows<float, kGateAfter>(a, s);
  return n.gate_first ? run_rows<__nv_bfloat16, kGateFirst>(a, s)
                      : run_rows<__nv_bfloat16, kGateAfter>(a, s);
}

size_t norm_gate_backward_workspace_bytes(int B, int H, int L, int D) {
  return sizeof(float) * (size_t)bwd_slots((int64_t)B * L, H, D) * H * D;
}

cudaError_t launch_norm_gate_backward(const NormGateArgs &n, const NormGateGrads &g, Dtype dt,
                                      void *ws, cudaStream_t s) {
  RowArgs a = gate_rows(n);
  a.in3 = g.dout;
  a.out1 = g.dy;
  a.out2 = g.dgate;
  a.rec = g.dw ? static_cast<float *>(ws) : nullptr;
  if (dt == kF32)
    return n.gate_first ? run_rows_bwd<float, kGateFirst>(a, g.dw, s)
                        : run_rows_bwd<float, kGateAfter>(a, g.dw, s);
  return n.gate_first ? run_rows_bwd<__nv_bfloat16, kGateFirst>(a, g.dw, s)
                      : run_rows_bwd<__nv_bfloat16, kGateAfter>(a, g.dw, s);
}

cudaError_t launch_norm_residual(const NormResidualArgs &n, Dtype dt, cudaStream_t s) {
  RowArgs a = residual_rows(n);
  a.in1 = n.x;
  a.in2 = n.residual;
  a.out1 = n.o;
  a.out2 = n.r;
  return dt == kF32 ? run_rows<float, kResidual>(a, s) : run_rows<__nv_bfloat16, kResidual>(a, s);
}

size_t norm_residual_backward_workspace_bytes(int64_t rows, int E) {
  return sizeof(float) * (size_t)bwd_slots(rows, 1, E) * E;
}

cudaError_t launch_norm_residual_backward(const NormResidualArgs &n, const NormResidualGrads &g,
                                          Dtype dt, void *ws, cudaStream_t s) {
  RowArgs a = residual_rows(n);
  a.in1 = n.r;
  a.in3 = g.dout;
  a.in4 = g.dr;
  a.out1 = g.dresidual;
  a.out2 = g.dx;
  a.rec = g.dw ? static_cast<float *>(ws) : nullptr;
  return dt == kF32 ? run_rows_bwd<float, kResidual>(a, g.dw, s)
                    : run_rows_bwd<__nv_bfloat16, kResidual>(a, g.dw, s);
}

}  // namespace linattn
