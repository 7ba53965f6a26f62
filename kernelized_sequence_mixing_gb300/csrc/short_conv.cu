// Short causal depthwise convolution ahead of the selective scan: a prompt,
// one token, and the backward pass (fp32 arithmetic).
//
//   pre_t[e] = bias[e] + sum_(k < W) w[e][k] x_(t - W + 1 + k)[e],  W in 2..4,
//   y_t = silu(pre_t)  (or pre_t),
// with the rows before the first token taken from `state` (or zeros).
//
// Bound by memory: x is read once and y written once.  A thread owns a few
// consecutive channels (16 bytes of them in the forward pass, one packed pair
// in the backward pass, whose windows and sums need the registers) and a run
// of consecutive tokens; the last W - 1 rows stay in registers as a sliding
// window, so only the first W - 1 rows of a run are read twice (from L2), and
// the next tokens' loads are issued a group ahead.
#include "dependent.cuh"
#include "kernels.h"
#include "mixer_common.cuh"

namespace linattn {
namespace {

constexpr int kThreads = 128;

// Pairs of channels as they lie in memory.
template <typename T, int P> struct rawp;  // P pairs
template <> struct rawp<__nv_bfloat16, 2> {
  uint2 a;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { a = *reinterpret_cast<const uint2 *>(p); }
  __device__ __forceinline__ void store(__nv_bfloat16 *p) const { *reinterpret_cast<uint2 *>(p) = a; }
  __device__ __forceinline__ void zero() { a = make_uint2(0u, 0u); }
  __device__ __forceinline__ void get(f2 (&x)[2]) const {
    x[0] = bf16x2_to_f2(a.x);
    x[1] = bf16x2_to_f2(a.y);
  }
};
template <> struct rawp<__nv_bfloat16, 4> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { a = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void store(__nv_bfloat16 *p) const { *reinterpret_cast<uint4 *>(p) = a; }
  __device__ __forceinline__ void zero() { a = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(f2 (&x)[4]) const {
    x[0] = bf16x2_to_f2(a.x);
    x[1] = bf16x2_to_f2(a.y);
    x[2] = bf16x2_to_f2(a.z);
    x[3] = bf16x2_to_f2(a.w);
  }
};
template <> struct rawp<float, 2> {
  float4 a;
  __device__ __forceinline__ void load(const float *p) { a = *reinterpret_cast<const float4 *>(p); }
  __device__ __forceinline__ void store(float *p) const { *reinterpret_cast<float4 *>(p) = a; }
  __device__ __forceinline__ void zero() { a = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(f2 (&x)[2]) const {
    x[0] = pack2(a.x, a.y);
    x[1] = pack2(a.z, a.w);
  }
};
template <> struct rawp<__nv_bfloat16, 1> {
  uint32_t a;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { a = *reinterpret_cast<const uint32_t *>(p); }
  __device__ __forceinline__ void zero() { a = 0u; }
  __device__ __forceinline__ void get(f2 (&x)[1]) const { x[0] = bf16x2_to_f2(a); }
};
template <> struct rawp<float, 1> {
  float2 a;
  __device__ __forceinline__ void load(const float *p) { a = *reinterpret_cast<const float2 *>(p); }
  __device__ __forceinline__ void zero() { a = make_float2(0.f, 0.f); }
  __device__ __forceinline__ void get(f2 (&x)[1]) const { x[0] = pack2(a.x, a.y); }
};
__device__ __forceinline__ void store_pair(__nv_bfloat16 *p, f2 v) {
  const float2 q = unpack2(v);
  *reinterpret_cast<uint32_t *>(p) = f32_to_bf16x2(q.x, q.y);
}
__device__ __forceinline__ void store_pair(float *p, f2 v) {
  *reinterpret_cast<float2 *>(p) = unpack2(v);
}
__device__ __forceinline__ void store_pairs(__nv_bfloat16 *p, const f2 (&v)[2]) {
  const float2 q = unpack2(v[0]), r = unpack2(v[1]);
  *reinterpret_cast<uint2 *>(p) = make_uint2(f32_to_bf16x2(q.x, q.y), f32_to_bf16x2(r.x, r.y));
}
__device__ __forceinline__ void store_pairs(float *p, const f2 (&v)[2]) {
  const float2 q = unpack2(v[0]), r = unpack2(v[1]);
  *reinterpret_cast<float4 *>(p) = make_float4(q.x, q.y, r.x, r.y);
}
__device__ __forceinline__ void store_pairs(__nv_bfloat16 *p, const f2 (&v)[4]) {
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 q = unpack2(v[i]);
    x[2 * i] = q.x;
    x[2 * i + 1] = q.y;
  }
  store8(p, x);
}
// Pairs of channels per thread of the forward pass: 16 bytes.
template <typename T> constexpr int kPairs = 8 / sizeof(T);
template <int P>
__device__ __forceinline__ void load_bias(const float *bias, int e, f2 (&out)[P]) {
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const float2 q = bias ? *reinterpret_cast<const float2 *>(bias + e + 2 * p) : make_float2(0.f, 0.f);
    out[p] = pack2(q.x, q.y);
  }
}
__device__ __forceinline__ f2 silu2(f2 v) { return mul2(v, sigmoid_f2(v)); }

// Row t < 0 of a sequence (before its first token): state row t + W - 1, or
// zeros.
template <typename T, int W, int P>
__device__ __forceinline__ rawp<T, P> early_row(const T *state, int t, int E) {
  rawp<T, P> r;
  if (state) r.load(state + (int64_t)(t + W - 1) * E);
  else r.zero();
  return r;
}

// The taps of 2P consecutive channels as pairs: w [E][W], from channel e.
template <int W, int P>
__device__ __forceinline__ void load_taps(const float *w, int e, f2 (&out)[W][P]) {
  float q[2 * P * W];
  if constexpr (P >= 2) {  // 4 W floats per two pairs: 16-byte aligned
#pragma unroll
    for (int i = 0; i < P * W / 2; ++i) {
      const float4 v = *reinterpret_cast<const float4 *>(w + (int64_t)e * W + 4 * i);
      q[4 * i] = v.x; q[4 * i + 1] = v.y; q[4 * i + 2] = v.z; q[4 * i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float2 v = *reinterpret_cast<const float2 *>(w + (int64_t)e * W + 2 * i);
      q[2 * i] = v.x; q[2 * i + 1] = v.y;
    }
  }
#pragma unroll
  for (int k = 0; k < W; ++k)
#pragma unroll
    for (int p = 0; p < P; ++p) out[k][p] = pack2(q[2 * p * W + k], q[(2 * p + 1) * W + k]);
}

// CTAs of the forward pass that fit an SM; one more would spill (B4 L4096
// E4096 W4 in bf16: 47 us at four, 79 at five; fp32: 85 at five, 87 at six).
template <typename T> constexpr int kResident = sizeof(T) == 2 ? 4 : 5;

template <typename T, int W>
__global__ void __launch_bounds__(kThreads, kResident<T>)
    conv_kernel(const __grid_constant__ ConvArgs a, int run_len, int runs) {
  constexpr int P = kPairs<T>;
  const unsigned cols = a.E / (2 * P);
  const int64_t idx = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t total = (int64_t)a.B * runs * cols;
  if (idx >= total) return;
  int e, run;
  int64_t b;
  if (total < ((int64_t)1 << 32)) {  // 32-bit divisions
    const unsigned i = static_cast<unsigned>(idx), br = i / cols;
    e = static_cast<int>(i - br * cols) * 2 * P;
    b = br / static_cast<unsigned>(runs);
    run = static_cast<int>(br - static_cast<unsigned>(b) * runs);
  } else {
    const int64_t br = idx / cols;
    e = static_cast<int>(idx - br * cols) * 2 * P;
    b = br / runs;
    run = static_cast<int>(br - b * runs);
  }
  const int len = a.lens ? min(max(a.lens[b], 0), a.L) : a.L;
  const int t0 = run * run_len, t1 = min(len, t0 + run_len);
  const T *x = static_cast<const T *>(a.x) + b * a.L * a.ldx + e;
  const T *st = a.state ? static_cast<const T *>(a.state) + b * (W - 1) * a.E + e : nullptr;
  T *y = static_cast<T *>(a.y) + b * a.L * a.E + e;

  if (run == runs - 1 && a.state_out) {
    // the last W - 1 rows of the sequence, bit for bit
    T *so = static_cast<T *>(a.state_out) + b * (W - 1) * a.E + e;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
      const int t = len - (W - 1) + k;
      rawp<T, P> r;
      if (t >= 0) r.load(x + t * a.ldx);
      else r = early_row<T, W, P>(st, t, a.E);
      r.store(so + (int64_t)k * a.E);
    }
  }
  if (t0 >= t1) return;

  f2 w[W][P], bias[P], win[W][P];  // win[k] = row t - W + 1 + k
  auto enter = [&](const rawp<T, P> &r) {
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
#pragma unroll
      for (int p = 0; p < P; ++p) win[k][p] = win[k + 1][p];
    r.get(win[W - 1]);
  };
  auto out_row = [&](T *p) {
    f2 o[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      o[i] = bias[i];
#pragma unroll
      for (int k = 0; k < W; ++k) o[i] = fma2(w[k][i], win[k][i], o[i]);
      if (a.silu) o[i] = silu2(o[i]);
    }
    store_pairs(p, o);
  };
  constexpr int kAhead = 4;
  const T *xp = x + t0 * a.ldx;
  T *yp = y + (int64_t)t0 * a.E;
  int t = t0;
  rawp<T, P> nxt[kAhead];
  auto fetch = [&] {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      nxt[j].load(xp);
      xp += a.ldx;
    }
  };
  if (t + kAhead <= t1) fetch();
  load_taps<W, P>(a.w, e, w);
  load_bias<P>(a.bias, e, bias);
#pragma unroll
  for (int k = 0; k < W - 1; ++k) {
    const int s = t0 - (W - 1) + k;
    rawp<T, P> r;
    if (s >= 0) r.load(x + s * a.ldx);
    else r = early_row<T, W, P>(st, s, a.E);
    r.get(win[k + 1]);
  }
  for (; t + kAhead <= t1; t += kAhead) {
    rawp<T, P> cur[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) cur[j] = nxt[j];
    if (t + 2 * kAhead <= t1) fetch();
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      enter(cur[j]);
      out_row(yp);
      yp += a.E;
    }
  }
  xp = x + t * a.ldx;
  for (; t < t1; ++t) {
    rawp<T, P> r;
    r.load(xp);
    xp += a.ldx;
    enter(r);
    out_row(yp);
    yp += a.E;
  }
}

// One token: a thread keeps its channels' taps for the sequences of its slice.
template <typename T, int W>
__global__ void __launch_bounds__(128) conv_step_kernel(const __grid_constant__ ConvArgs a) {
  const int e = (blockIdx.x * 128 + threadIdx.x) * 4;
  if (e >= a.E) return;
  f2 w[W][2], bias[2];
  load_taps<W, 2>(a.w, e, w);
  load_bias<2>(a.bias, e, bias);
  for (int64_t b = blockIdx.y; b < a.B; b += gridDim.y) {
    T *st = static_cast<T *>(a.state_out) + b * (W - 1) * a.E + e;
    rawp<T, 2> r[W];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) r[k].load(st + (int64_t)k * a.E);
    r[W - 1].load(static_cast<const T *>(a.x) + b * a.ldx + e);
    f2 o[2] = {bias[0], bias[1]};
#pragma unroll
    for (int k = 0; k < W; ++k) {
      f2 x[2];
      r[k].get(x);
#pragma unroll
      for (int p = 0; p < 2; ++p) o[p] = fma2(w[k][p], x[p], o[p]);
      if (k > 0) r[k].store(st + (int64_t)(k - 1) * a.E);
    }
    if (a.silu)
#pragma unroll
      for (int p = 0; p < 2; ++p) o[p] = silu2(o[p]);
    store_pairs(static_cast<T *>(a.y) + b * a.E + e, o);
  }
}

// Backward.  With dpre_t = dy_t silu'(pre_t):
//   dx_s = sum_k w[k] dpre_(s + W - 1 - k)   (s < 0: the gradient of `state`),
//   dw[k] = sum_t dpre_t x_(t - W + 1 + k),   dbias = sum_t dpre_t.
// A thread walks the tokens of its runs with windows of x and of dpre; at
// token t it knows dpre_(t-W+1..t), which is all that dx_(t-W+1) needs.  A run
// of dx rows [s0, s1) reads W - 1 tokens of dpre beyond s1, recomputed by the
// next run too; the sums count a token only in the run that owns it.  A CTA
// is 32 pairs of channels x 4 runs at a time; its sums meet in shared memory
// and leave as one record, and a second kernel adds the records in their
// order, so the result does not depend on scheduling.
constexpr int kBwdCols = 32, kBwdRows = 4;
// CTAs that fit an SM: the loads ahead (2 W per thread) take the registers.
// Three taps in fp32 spill 8 bytes as it is, the others nothing.  One more
// would spill (B4 L4096 E4096, W = 4, fp32: 128 us at four, 185 at
// five; bf16: 89 at five, 95 at six), one less leaves a part of the SM idle.
constexpr int bwd_resident(int elem_bytes, int W) { return (elem_bytes == 4 ? 8 : 9) - W; }

template <typename T, int W>
__global__ void __launch_bounds__(kBwdCols * kBwdRows, bwd_resident(sizeof(T), W))
    conv_bwd_kernel(const __grid_constant__ ConvArgs a, const __grid_constant__ ConvGrads g,
                    float *__restrict__ rec, int run_len, int runs) {
  let_next_start();
  const int tx = threadIdx.x % kBwdCols, ty = threadIdx.x / kBwdCols;
  const int e = (blockIdx.x * kBwdCols + tx) * 2;
  const bool in = e < a.E;
  f2 w[W][1], bias = dup2(0.f), dw[W], db = dup2(0.f);
#pragma unroll
  for (int k = 0; k < W; ++k) w[k][0] = dw[k] = dup2(0.f);
  if (in) {
    load_taps<W, 1>(a.w, e, w);
    if (a.bias) bias = pack2(a.bias[e], a.bias[e + 1]);
  }
  const int64_t total = (int64_t)a.B * runs;
  for (int64_t r = (int64_t)blockIdx.y * kBwdRows + ty; in && r < total;
       r += (int64_t)gridDim.y * kBwdRows) {
    const int64_t b = r / runs;
    const int run = static_cast<int>(r - b * runs);
    const int s0 = run * run_len, s1 = min(a.L, s0 + run_len);
    const T *x = static_cast<const T *>(a.x) + b * a.L * a.ldx + e;
    const T *dy = static_cast<const T *>(g.dy) + b * a.L * a.E + e;
    T *dx = static_cast<T *>(g.dx) + b * a.L * a.E + e;
    const T *st = a.state ? static_cast<const T *>(a.state) + b * (W - 1) * a.E + e : nullptr;
    f2 xw[W], dp[W];  // xw[k] = row t-W+1+k; dp[k] = dpre of t-W+1+k
#pragma unroll
    for (int k = 0; k < W; ++k) xw[k] = dp[k] = dup2(0.f);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
      const int t = s0 - (W - 1) + k;
      rawp<T, 1> q;
      if (t >= 0) q.load(x + t * a.ldx);
      else q = early_row<T, W, 1>(st, t, a.E);
      f2 v[1];
      q.get(v);
      xw[k + 1] = v[0];
    }
    // one token on: its row and upstream gradient into the windows
    auto enter = [&](const rawp<T, 1> &xr, const rawp<T, 1> &gr) {
#pragma unroll
      for (int k = 0; k < W - 1; ++k) {
        xw[k] = xw[k + 1];
        dp[k] = dp[k + 1];
      }
      f2 v[1];
      xr.get(v);
      xw[W - 1] = v[0];
      gr.get(v);
      f2 d = v[0];
      if (a.silu) {
        f2 p = bias;
#pragma unroll
        for (int k = 0; k < W; ++k) p = fma2(w[k][0], xw[k], p);
        // silu'(p) = s (1 + p (1 - s))
        const f2 s = sigmoid_f2(p);
        d = mul2(d, mul2(s, fma2(p, fma2(s, dup2(-1.f), dup2(1.f)), dup2(1.f))));
      }
      dp[W - 1] = d;
    };
    auto add_sums = [&] {
      db = add2(db, dp[W - 1]);
#pragma unroll
      for (int k = 0; k < W; ++k) dw[k] = fma2(dp[W - 1], xw[k], dw[k]);
    };
    auto dx_row = [&] {  // of the window's first token
      // dpre_(s + W - 1 - k) = dp[W - 1 - k]
      f2 o = mul2(w[0][0], dp[W - 1]);
#pragma unroll
      for (int k = 1; k < W; ++k) o = fma2(w[k][0], dp[W - 1 - k], o);
      return o;
    };
    // the first W - 1 tokens: their dx rows belong to the run before, or are
    // the state's
    int t = s0;
#pragma unroll
    for (int k = 0; k < W - 1; ++k, ++t) {
      rawp<T, 1> xr, gr;
      xr.zero();
      gr.zero();
      if (t < a.L) {
        xr.load(x + t * a.ldx);
        gr.load(dy + (int64_t)t * a.E);
      }
      enter(xr, gr);
      if (t >= a.L) dp[W - 1] = dup2(0.f);
      if (t < s1) add_sums();
      if (run == 0 && g.dstate) store_pair(static_cast<T *>(g.dstate) + (b * (W - 1) + k) * a.E + e, dx_row());
    }
    // whole groups of the run's own tokens, loads a group ahead
    constexpr int kAhead = 2 * W;  // a multiple of W: the windows turn in place
    const T *xp = x + t * a.ldx, *gp = dy + (int64_t)t * a.E;
    T *op = dx + (int64_t)s0 * a.E;
    if (t + kAhead <= s1) {
      rawp<T, 1> xn[kAhead], gn[kAhead];
      auto fetch = [&] {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          xn[j].load(xp);
          gn[j].load(gp);
          xp += a.ldx;
          gp += a.E;
        }
      };
      fetch();
      for (; t + kAhead <= s1; t += kAhead) {
        rawp<T, 1> xq[kAhead], gq[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          xq[j] = xn[j];
          gq[j] = gn[j];
        }
        if (t + 2 * kAhead <= s1) fetch();
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          enter(xq[j], gq[j]);
          add_sums();
          store_pair(op, dx_row());
          op += a.E;
        }
      }
    }
    // what is left, and the W - 1 tokens behind the run
    xp = x + t * a.ldx;
    gp = dy + (int64_t)t * a.E;
    for (; t < s1 + W - 1; ++t) {
      rawp<T, 1> xr, gr;
      xr.zero();
      gr.zero();
      if (t < a.L) {
        xr.load(xp);
        gr.load(gp);
        xp += a.ldx;
        gp += a.E;
      }
      enter(xr, gr);
      if (t >= a.L) dp[W - 1] = dup2(0.f);
      if (t < s1) add_sums();
      if (t - (W - 1) >= s0) {
        store_pair(op, dx_row());
        op += a.E;
      }
    }
  }
  // sums of the CTA's runs, in row order; a record is dw [E][W], then dbias [E]
  __shared__ float2 sh[kBwdRows][kBwdCols];
  float *out = rec + (int64_t)blockIdx.y * (W + 1) * a.E;
#pragma unroll
  for (int k = 0; k <= W; ++k) {
    __syncthreads();
    sh[ty][tx] = unpack2(k < W ? dw[k % W] : db);
    __syncthreads();
    if (ty == 0 && in) {
      float2 q = sh[0][tx];
      for (int j = 1; j < kBwdRows; ++j) {
        q.x += sh[j][tx].x;
        q.y += sh[j][tx].y;
      }
      const int stride = k < W ? W : 1;
      float *o = k < W ? out + (int64_t)e * W + k : out + (int64_t)a.E * W + e;
      o[0] = q.x;
      o[stride] = q.y;
    }
  }
}

// Backward pass: a run per warp row such that all the CTAs are resident at
// once (a CTA has four rows), of at least 29 tokens (the W - 1 walked twice are
// then a tenth at most).  More sequences than such rows give up to four times
// as many CTAs, and beyond that a row takes several sequences.  Holding them to
// the resident CTAs measured the same within 4% either way (bf16 B256 L128
// E4096 W4: 181 us, held 187; B512 L64: 206 and 206; fp32 B300 L64 E8192 W4:
// 356, held 349).
struct BwdPlan {
  int run_len, runs, ny;
};
BwdPlan conv_bwd_plan(int B, int L, int E, int W, int elem_bytes) {
  const int nx = (E / 2 + kBwdCols - 1) / kBwdCols;
  int rows = kSMs * bwd_resident(elem_bytes, W) / nx * kBwdRows;  // rows of runs that fit at once
  if (rows < kBwdRows) rows = kBwdRows;
  const int per = rows / B > 0 ? rows / B : 1;  // runs per sequence
  BwdPlan p;
  p.run_len = (L + per - 1) / per;
  if (p.run_len < 29) p.run_len = 29;
  p.runs = (L + p.run_len - 1) / p.run_len;
  const int64_t need = ((int64_t)B * p.runs + kBwdRows - 1) / kBwdRows;
  p.ny = need < rows ? static_cast<int>(need) : rows;
  return p;
}

template <typename T, int W>
cudaError_t conv_fwd_typed(const ConvArgs &a, cudaStream_t s) {
  // Runs of at most 128 tokens (the taps and the W - 1 early rows cost a thread
  // about five tokens' work), in whole groups of 4, as many as fill the waves
  // of CTAs that this takes.
  const int cols = a.E / (2 * kPairs<T>);
  const int64_t wave = (int64_t)kSMs * kResident<T> * kThreads, lanes = (int64_t)a.B * cols;
  const int64_t least = lanes * ((a.L + 127) / 128), waves = least > wave ? (least + wave - 1) / wave : 1;
  const int64_t per = waves * wave / lanes;  // runs per sequence
  int64_t len = per > 0 ? (a.L + per - 1) / per : a.L;
  len = (len + 3) / 4 * 4;
  const int run_len = static_cast<int>(len < 8 ? 8 : len > 128 ? 128 : len);
  const int runs = a.L > 0 ? (a.L + run_len - 1) / run_len : 1;
  const int64_t n = (int64_t)a.B * runs * cols;
  conv_kernel<T, W><<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, s>>>(a, run_len, runs);
  return cudaGetLastError();
}
template <typename T, int W>
cudaError_t conv_step_typed(const ConvArgs &a, cudaStream_t s) {
  const int nx = (a.E / 4 + 127) / 128;
  // about eight CTAs per SM; beyond that a CTA takes several sequences
  int ny = (kSMs * 8 + nx - 1) / nx;
  if (ny > a.B) ny = a.B;
  conv_step_kernel<T, W><<<dim3(nx, ny), 128, 0, s>>>(a);
  return cudaGetLastError();
}
template <typename T, int W>
cudaError_t conv_bwd_typed(const ConvArgs &a, const ConvGrads &g, void *ws, cudaStream_t s) {
  const BwdPlan p = conv_bwd_plan(a.B, a.L, a.E, W, sizeof(T));
  const int nx = (a.E / 2 + kBwdCols - 1) / kBwdCols;
  float *rec = static_cast<float *>(ws);
  conv_bwd_kernel<T, W><<<dim3(nx, p.ny), kBwdCols * kBwdRows, 0, s>>>(a, g, rec, p.run_len, p.runs);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_column_sum(rec, p.ny, (int64_t)(W + 1) * a.E, g.dw, (int64_t)W * a.E, g.dbias, s);
}

template <typename T>
cudaError_t conv_widths(const ConvArgs &a, const ConvGrads *g, bool step, void *ws, cudaStream_t s) {
  switch (a.W) {
#define LA_CONV_W(w)                                               \
  case w:                                                          \
    return g ? conv_bwd_typed<T, w>(a, *g, ws, s)                  \
             : step ? conv_step_typed<T, w>(a, s) : conv_fwd_typed<T, w>(a, s);
    LA_CONV_W(2)
    LA_CONV_W(3)
    LA_CONV_W(4)
#undef LA_CONV_W
  }
  return cudaErrorNotSupported;
}

}  // namespace

cudaError_t launch_conv(const ConvArgs &a, Dtype dt, cudaStream_t s) {
  return dt == kF32 ? conv_widths<float>(a, nullptr, false, nullptr, s)
                    : conv_widths<__nv_bfloat16>(a, nullptr, false, nullptr, s);
}
cudaError_t launch_conv_step(const ConvArgs &a, Dtype dt, cudaStream_t s) {
  return dt == kF32 ? conv_widths<float>(a, nullptr, true, nullptr, s)
                    : conv_widths<__nv_bfloat16>(a, nullptr, true, nullptr, s);
}
size_t conv_backward_workspace_bytes(int B, int L, int E, int W, Dtype dt) {
  return sizeof(float) * (size_t)conv_bwd_plan(B, L, E, W, dt == kF32 ? 4 : 2).ny * (W + 1) * E;
}
cudaError_t launch_conv_backward(const ConvArgs &a, const ConvGrads &g, Dtype dt, void *ws,
                                 cudaStream_t s) {
  return dt == kF32 ? conv_widths<float>(a, &g, false, ws, s)
                    : conv_widths<__nv_bfloat16>(a, &g, false, ws, s);
}

}  // namespace linattn
