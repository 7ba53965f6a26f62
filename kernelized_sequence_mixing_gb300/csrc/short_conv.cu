// Short causal depthwise convolution ahead of the selective scan: a prompt,
// one token, and the backward pass (fp32 arithmetic).
//
//   pre_t[e] = bias[e] + sum_(k < W) w[e][k] x_(t - W + 1 + k)[e],  W in 2..4,
//   y_t = silu(pre_t)  (or pre_t),
// with the rows before the first token taken from `state` (or zeros).
//
// Bound by memory: x is read once and y written once.  A thread owns a vector
// of channels (8 in the forward pass, 4 in the backward pass, whose
// accumulators need the registers) and a run of consecutive tokens; the last
// W - 1 rows stay in registers as a sliding window, so only the first W - 1
// rows of a run are read twice (from L2).
#include "kernels.h"
#include "mixer_common.cuh"

namespace linattn {
namespace {

constexpr int kThreads = 256;
constexpr int kRun = 16;  // tokens per thread of the forward pass

// Row t of sequence b before its first token: state row t + W - 1, or zeros.
template <typename T, int W>
__device__ __forceinline__ void state_row8(const ConvArgs &a, int64_t b, int t, int e, float (&x)[8]) {
  if (a.state) {
    load8(static_cast<const T *>(a.state) + (b * (W - 1) + t + W - 1) * a.E + e, x);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.f;
  }
}

template <typename T, int W>
__global__ void __launch_bounds__(kThreads) conv_kernel(const __grid_constant__ ConvArgs a, int runs) {
  const int cols = a.E / 8;
  const int64_t idx = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (idx >= (int64_t)a.B * runs * cols) return;
  const int e = static_cast<int>(idx % cols) * 8;
  const int64_t br = idx / cols;
  const int run = static_cast<int>(br % runs);
  const int64_t b = br / runs;
  const int len = a.lens ? min(max(a.lens[b], 0), a.L) : a.L;
  const int t0 = run * kRun, t1 = min(len, t0 + kRun);
  const T *x = static_cast<const T *>(a.x) + b * a.L * a.ldx + e;
  T *y = static_cast<T *>(a.y) + b * a.L * a.E + e;

  if (run == runs - 1 && a.state_out) {
    // the last W - 1 rows of the sequence, bit for bit
    T *so = static_cast<T *>(a.state_out) + b * (W - 1) * a.E + e;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
      const int t = len - (W - 1) + k;
      raw8<T> r;
      if (t >= 0) r.load(x + t * a.ldx);
      else if (a.state) r.load(static_cast<const T *>(a.state) + (b * (W - 1) + t + W - 1) * a.E + e);
      else r.zero();
      r.store(so + (int64_t)k * a.E);
    }
  }
  if (t0 >= t1) return;

  float w[W][8], bias[8];
  {
    float q[8 * W];  // w rows of 8 consecutive channels are consecutive
#pragma unroll
    for (int i = 0; i < 2 * W; ++i) {
      const float4 v = *reinterpret_cast<const float4 *>(a.w + (int64_t)e * W + 4 * i);
      q[4 * i] = v.x; q[4 * i + 1] = v.y; q[4 * i + 2] = v.z; q[4 * i + 3] = v.w;
    }
#pragma unroll
    for (int k = 0; k < W; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) w[k][i] = q[i * W + k];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) bias[i] = 0.f;
  if (a.bias) load8(a.bias + e, bias);

  float win[W][8];  // win[k] = row t - W + 1 + k
#pragma unroll
  for (int k = 0; k < W - 1; ++k) {
    const int t = t0 - (W - 1) + k;
    if (t >= 0) load8(x + t * a.ldx, win[k + 1]);
    else state_row8<T, W>(a, b, t, e, win[k + 1]);
  }
  constexpr int kAhead = 8;
  for (int tb = t0; tb < t1; tb += kAhead) {
    raw8<T> nxt[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (tb + j < t1) nxt[j].load(x + (tb + j) * a.ldx);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (tb + j < t1) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) win[k][i] = win[k + 1][i];
        nxt[j].get(win[W - 1]);
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float p = bias[i];
#pragma unroll
          for (int k = 0; k < W; ++k) p = fmaf(w[k][i], win[k][i], p);
          o[i] = a.silu ? p * sigmoid_f32(p) : p;
        }
        store8(y + (int64_t)(tb + j) * a.E, o);
      }
    }
  }
}

template <typename T, int W>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(const __grid_constant__ ConvArgs a) {
  const int cols = a.E / 8;
  const int64_t idx = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (idx >= (int64_t)a.B * cols) return;
  const int e = static_cast<int>(idx % cols) * 8;
  const int64_t b = idx / cols;
  T *st = static_cast<T *>(a.state_out) + b * (W - 1) * a.E + e;
  raw8<T> r[W];
#pragma unroll
  for (int k = 0; k < W - 1; ++k) r[k].load(st + (int64_t)k * a.E);
  r[W - 1].load(static_cast<const T *>(a.x) + b * a.ldx + e);
  float q[8 * W], o[8];
#pragma unroll
  for (int i = 0; i < 2 * W; ++i) {
    const float4 v = *reinterpret_cast<const float4 *>(a.w + (int64_t)e * W + 4 * i);
    q[4 * i] = v.x; q[4 * i + 1] = v.y; q[4 * i + 2] = v.z; q[4 * i + 3] = v.w;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = 0.f;
  if (a.bias) load8(a.bias + e, o);
#pragma unroll
  for (int k = 0; k < W; ++k) {
    float x[8];
    r[k].get(x);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = fmaf(q[i * W + k], x[i], o[i]);
    if (k > 0) r[k].store(st + (int64_t)(k - 1) * a.E);
  }
  if (a.silu)
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] *= sigmoid_f32(o[i]);
  store8(static_cast<T *>(a.y) + b * a.E + e, o);
}

// Backward.  With dpre_t = dy_t silu'(pre_t):
//   dx_s = sum_k w[k] dpre_(s + W - 1 - k)   (s < 0: the gradient of `state`),
//   dw[k] = sum_t dpre_t x_(t - W + 1 + k),   dbias = sum_t dpre_t.
// A thread walks the tokens of its runs with windows of x and of dpre; at
// token t it knows dpre_(t-W+1..t), which is all that dx_(t-W+1) needs.  A run
// of dx rows [s0, s1) reads W - 1 tokens of dpre beyond s1, recomputed by the
// next run too; the sums count a token only in the run that owns it.  A CTA
// is 32 vectors of channels x 8 runs at a time; its sums meet in shared
// memory and leave as one record, and a second kernel adds the records in
// their order, so the result does not depend on scheduling.
constexpr int kBwdCols = 32, kBwdRows = 8, kBwdVec = 4, kBwdRun = 32;

template <typename T, int W>
__global__ void __launch_bounds__(kBwdCols * kBwdRows)
    conv_bwd_kernel(const __grid_constant__ ConvArgs a, const __grid_constant__ ConvGrads g,
                    float *__restrict__ rec, int runs) {
  const int tx = threadIdx.x % kBwdCols, ty = threadIdx.x / kBwdCols;
  const int e = (blockIdx.x * kBwdCols + tx) * kBwdVec;
  const bool in = e < a.E;
  float w[W][4], bias[4], dw[W][4], db[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    bias[i] = in && a.bias ? a.bias[e + i] : 0.f;
    db[i] = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) {
      w[k][i] = in ? a.w[(int64_t)(e + i) * W + k] : 0.f;
      dw[k][i] = 0.f;
    }
  }
  // the first run of a sequence starts W - 1 rows early when the state has a
  // gradient
  const int64_t total = (int64_t)a.B * runs;
  for (int64_t r = (int64_t)blockIdx.y * kBwdRows + ty; in && r < total;
       r += (int64_t)gridDim.y * kBwdRows) {
    const int64_t b = r / runs;
    const int run = static_cast<int>(r - b * runs);
    const int s0 = run * kBwdRun, s1 = min(a.L, s0 + kBwdRun);
    const T *x = static_cast<const T *>(a.x) + b * a.L * a.ldx + e;
    const T *dy = static_cast<const T *>(g.dy) + b * a.L * a.E + e;
    T *dx = static_cast<T *>(g.dx) + b * a.L * a.E + e;
    const T *st = a.state ? static_cast<const T *>(a.state) + b * (W - 1) * a.E + e : nullptr;
    float xw[W][4], dp[W][4];  // xw[k] = row t-W+1+k; dp[k] = dpre of t-W+1+k
#pragma unroll
    for (int k = 0; k < W; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) xw[k][i] = dp[k][i] = 0.f;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
      const int t = s0 - (W - 1) + k;
      float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
      if (t >= 0) q = load4(x + t * a.ldx);
      else if (st) q = load4(st + (int64_t)(t + W - 1) * a.E);
      xw[k + 1][0] = q.x; xw[k + 1][1] = q.y; xw[k + 1][2] = q.z; xw[k + 1][3] = q.w;
    }
    const int last = s1 + W - 1;  // tokens walked: [s0, last)
    constexpr int kAhead = 4;
    for (int tb = s0; tb < last; tb += kAhead) {
      float4 xq[kAhead], gq[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        xq[j] = gq[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (tb + j < min(last, a.L)) {
          xq[j] = load4(x + (tb + j) * a.ldx);
          gq[j] = load4(dy + (int64_t)(tb + j) * a.E);
        }
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int t = tb + j;
        if (t >= last) break;
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            xw[k][i] = xw[k + 1][i];
            dp[k][i] = dp[k + 1][i];
          }
        const float xv[4] = {xq[j].x, xq[j].y, xq[j].z, xq[j].w};
        const float gv[4] = {gq[j].x, gq[j].y, gq[j].z, gq[j].w};
        const bool own = t < s1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          xw[W - 1][i] = xv[i];
          float d = gv[i];  // zero behind the last token
          if (a.silu) {
            float p = bias[i];
#pragma unroll
            for (int k = 0; k < W; ++k) p = fmaf(w[k][i], xw[k][i], p);
            const float s = sigmoid_f32(p);
            d *= s * fmaf(p, 1.f - s, 1.f);
          }
          if (t >= a.L) d = 0.f;
          dp[W - 1][i] = d;
          if (own) {
            db[i] += d;
#pragma unroll
            for (int k = 0; k < W; ++k) dw[k][i] = fmaf(d, xw[k][i], dw[k][i]);
          }
        }
        const int s = t - (W - 1);
        if (s >= s0 || (run == 0 && g.dstate)) {
          float4 q;
          float *o = &q.x;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float v = 0.f;
            // dpre_(s + W - 1 - k) = dp[W - 1 - k]
#pragma unroll
            for (int k = 0; k < W; ++k) v = fmaf(w[k][i], dp[W - 1 - k][i], v);
            o[i] = v;
          }
          if (s >= 0) store4(dx + (int64_t)s * a.E, q);
          else store4(static_cast<T *>(g.dstate) + (b * (W - 1) + s + W - 1) * a.E + e, q);
        }
      }
    }
  }
  // sums of the CTA's runs, in row order; a record is dw [E][W], then dbias [E]
  __shared__ float4 sh[kBwdRows][kBwdCols];
  float *out = rec + (int64_t)blockIdx.y * (W + 1) * a.E;
#pragma unroll
  for (int k = 0; k <= W; ++k) {
    __syncthreads();
    sh[ty][tx] = k < W ? make_float4(dw[k % W][0], dw[k % W][1], dw[k % W][2], dw[k % W][3])
                       : make_float4(db[0], db[1], db[2], db[3]);
    __syncthreads();
    if (ty == 0 && in) {
      float4 q = sh[0][tx];
      for (int j = 1; j < kBwdRows; ++j) {
        q.x += sh[j][tx].x; q.y += sh[j][tx].y; q.z += sh[j][tx].z; q.w += sh[j][tx].w;
      }
      const int stride = k < W ? W : 1;
      float *o = k < W ? out + (int64_t)e * W + k : out + (int64_t)a.E * W + e;
      o[0] = q.x; o[stride] = q.y; o[2 * stride] = q.z; o[3 * stride] = q.w;
    }
  }
}

int conv_bwd_blocks(int B, int L, int E) {
  const int64_t rows = ((int64_t)B * ((L + kBwdRun - 1) / kBwdRun) + kBwdRows - 1) / kBwdRows;
  const int colb = (E / kBwdVec + kBwdCols - 1) / kBwdCols;
  int64_t y = (152 * 4 + colb - 1) / colb;  // about four CTAs per SM
  if (y > rows) y = rows;
  return y < 1 ? 1 : static_cast<int>(y);
}

template <typename T, int W>
cudaError_t conv_fwd_typed(const ConvArgs &a, cudaStream_t s) {
  const int runs = a.L > 0 ? (a.L + kRun - 1) / kRun : 1;
  const int64_t n = (int64_t)a.B * runs * (a.E / 8);
  conv_kernel<T, W><<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, s>>>(a, runs);
  return cudaGetLastError();
}
template <typename T, int W>
cudaError_t conv_step_typed(const ConvArgs &a, cudaStream_t s) {
  const int64_t n = (int64_t)a.B * (a.E / 8);
  conv_step_kernel<T, W><<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}
template <typename T, int W>
cudaError_t conv_bwd_typed(const ConvArgs &a, const ConvGrads &g, void *ws, cudaStream_t s) {
  const int runs = (a.L + kBwdRun - 1) / kBwdRun;
  const int ny = conv_bwd_blocks(a.B, a.L, a.E);
  const int nx = (a.E / kBwdVec + kBwdCols - 1) / kBwdCols;
  float *rec = static_cast<float *>(ws);
  conv_bwd_kernel<T, W><<<dim3(nx, ny), kBwdCols * kBwdRows, 0, s>>>(a, g, rec, runs);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_column_sum(rec, ny, (int64_t)(W + 1) * a.E, g.dw, (int64_t)W * a.E, g.dbias, s);
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
size_t conv_backward_workspace_bytes(int B, int L, int E, int W) {
  return sizeof(float) * (size_t)conv_bwd_blocks(B, L, E) * (W + 1) * E;
}
cudaError_t launch_conv_backward(const ConvArgs &a, const ConvGrads &g, Dtype dt, void *ws,
                                 cudaStream_t s) {
  return dt == kF32 ? conv_widths<float>(a, &g, false, ws, s)
                    : conv_widths<__nv_bfloat16>(a, &g, false, ws, s);
}

}  // namespace linattn
