// Retention: linear attention with one decay per head, signed queries and
// keys as they are and no normaliser,
//
//   S_t = g S_(t-1) + k_t v_t^T,   o_t = scale q_t^T S_t.
//
// One product serves the forward pass and all gradients: rows x of width Dx
// read a state that rows y (width Dx) and w (width Dw) build,
//
//   o_i = scale (sum_(j <= i) g^(i-j) (x_i . y_j) w_j + x_i^T start terms),
//
// forward in time or backward (j >= i):
//
//   o : x = q,  y = k,  w = v                       state S_t
//   dq: x = do, y = v,  w = k                       state S_t^T
//   dk: x = v,  y = do, w = q,  backward in time    state U_t^T
//   dv: x = k,  y = q,  w = do, backward in time    state U_t
//
// where U_t = dL/dS_t / scale = g U_(t+1) + q_t do_t^T, with dL/dS / scale of the
// final state behind the last token.  By chunks of C tokens, the state in front of
// the chunk (in the order of the pass) is carried and the rest is a masked matrix
// of weights.  Over the n tokens of a chunk, forward in time:
//
//   o_i = scale (g^(i+1) x_i S + sum_(j <= i) g^(i-j) (x_i . y_j) w_j)
//   S  <- g^n S + sum_j g^(n-1-j) y_j w_j^T
//
// and backward in time, U being the gradient of the state in front of the tokens
// done so far (so that a gradient of the final state meets the last token
// undecayed):
//
//   o_i = scale (g^(n-1-i) x_i U + sum_(j >= i) g^(j-i) (x_i . y_j) w_j)
//   U  <- g^n U + sum_j g^(j+1) y_j w_j^T
//
// The product is linear in the features of x and y: more than 128 of them are two
// roles whose outputs are added.
#pragma once
#include "kernels.h"

namespace linattn {

// The tokens of sequence b of a call.
__device__ __forceinline__ int ret_tokens(const int *lens, int b, int L) {
  if (!lens) return L;
  const int n = lens[b];
  return n < 0 ? 0 : (n > L ? L : n);
}

// Tokens in front of chunk c of n (in the order in which they are worked: a
// pass backward in time begins with the last chunk, which may be short).
__device__ __forceinline__ int ret_before(int c, int n, int tokens, int C, int reverse) {
  if (c >= n) return tokens;
  if (!reverse || c == 0) return c * C;
  return tokens - (n - 1) * C + (c - 1) * C;
}

// The state in front of a part: what the earlier parts have added (records,
// each relative to its part's end) and the start, weighted by the decay since.
// Row d, column e of a state of Dw columns.
__device__ __forceinline__ float ret_start(const RetRole &r, const float *rec, int64_t bh, int part, int cpp, int n,
                                           int tokens, int C, float lg, int d, int e) {
  const int here = ret_before(part * cpp, n, tokens, C, r.reverse);
  float s = 0.f;
  if (r.start)
    s = exp2f(lg * static_cast<float>(here)) * r.start_scale *
        r.start[bh * r.state + static_cast<int64_t>(d) * r.start_rs + static_cast<int64_t>(e) * r.start_cs];
  for (int j = 0; j < part; ++j) {
    const int end = ret_before((j + 1) * cpp, n, tokens, C, r.reverse);
    s = fmaf(exp2f(lg * static_cast<float>(here - end)), rec[static_cast<int64_t>(j) * r.Dx * r.Dw + d * r.Dw + e], s);
  }
  return s;
}

}  // namespace linattn
