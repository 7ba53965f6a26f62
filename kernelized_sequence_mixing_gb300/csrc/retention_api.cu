// C ABI of retention and of beam search over decode states: argument
// validation, workspace and dispatch.  Every check runs before the first CUDA
// call.
#include "api_common.h"

using namespace linattn;

namespace {

constexpr int64_t kMaxTokens = ((int64_t)1 << 31) - (1 << 16);
constexpr int kMaxBeams = 32, kMaxBest = 64;

struct Dim {
  int64_t size, stride;
};

// Strides of a [B][L][heads][width] tensor with contiguous rows: each a positive
// multiple of 8 elements, and no two rows over one another.  Strides of
// dimensions of one element do not matter and become those of a dense tensor.
bool strides_ok(RetStrides *r, int64_t B, int64_t L, int64_t heads, int64_t width) {
  if (L == 0) return true;
  if (heads <= 1) r->h = width;
  if (L <= 1) r->t = heads * width;
  if (B <= 1) r->b = L * heads * width;
  Dim d[3] = {{B, r->b}, {L, r->t}, {heads, r->h}};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (d[j].stride < d[i].stride) {
        const Dim x = d[i];
        d[i] = d[j];
        d[j] = x;
      }
  int64_t inner = width;
  for (int i = 0; i < 3; ++i) {
    if (d[i].size <= 1) continue;
    if (d[i].stride % 8 != 0 || d[i].stride < inner || d[i].stride >= ((int64_t)1 << 37)) return false;
    inner = d[i].stride * (d[i].size - 1) + inner;
  }
  return true;
}

size_t span_of(const RetStrides &r, int64_t B, int64_t L, int64_t heads, int64_t width, size_t es) {
  return (size_t)((B - 1) * r.b + (L - 1) * r.t + (heads - 1) * r.h + width) * es;
}

RetStrides dense(int64_t L, int64_t heads, int64_t width) { return {L * heads * width, heads * width, width}; }

la_status_t check_sizes(int B, int L, int H, int Hk, int D, int Dv, float scale, la_dtype_t dt) {
  if (!dtype_ok(dt) || B < 0 || L < 0 || H < 0 || D <= 0 || Dv <= 0) return LA_ERR_INVALID_ARG;
  // the backward pass divides by it
  if (!(fabsf(scale) >= 0x1p-64f && fabsf(scale) <= 0x1p64f)) return LA_ERR_INVALID_ARG;
  if (H > 0 && (Hk <= 0 || H % Hk != 0)) return LA_ERR_INVALID_ARG;
  if (H > kMaxHeads || D % 8 != 0 || Dv % 8 != 0 || D > 256 || Dv > 256) return LA_ERR_UNSUPPORTED;
  if ((int64_t)B * (L > 0 ? L : 1) >= kMaxTokens || (int64_t)B * H >= (1 << 26)) return LA_ERR_UNSUPPORTED;
  return LA_OK;
}

// gamma: NULL (all 1) or H values in [0, 1].
bool gammas_ok(const float *gamma, int H, Gammas *g) {
  for (int h = 0; h < kMaxHeads; ++h) g->g[h] = 1.f;
  for (int h = 0; gamma && h < H; ++h) {
    if (!(gamma[h] >= 0.f && gamma[h] <= 1.f)) return false;  // also NaN
    g->g[h] = gamma[h];
  }
  return true;
}

// log2 of each decay.  A decay of zero takes a finite value so low that any
// power but the zeroth vanishes (zero times infinity would not be zero).
Gammas logs(const Gammas &g) {
  Gammas r;
  for (int h = 0; h < kMaxHeads; ++h) r.g[h] = g.g[h] > 0.f ? (float)log2((double)g.g[h]) : -1e30f;
  return r;
}

bool lens_ok(const int *lens, int B, std::initializer_list<Buf> written) {
  if (reinterpret_cast<uintptr_t>(lens) & 3u) return false;
  const Buf l = {lens, sizeof(int) * (size_t)B, false, false};
  for (const Buf &w : written)
    if (overlap(l, w)) return false;
  return true;
}

// A call's roles with their outputs' shares: where query heads share a head of the
// output (group) or there are more than 128 features (the kernels' most: 128 of them
// and then the rest), each share goes to the workspace in fp32 and the sums follow.
struct Plan {
  RetArgs a = {};
  GroupSumArgs sum[3] = {};
  int sums = 0;
  size_t share = 0;  // floats of the workspace in front of the records

  // r: o and os are the output's own; head h of the call writes head h / group.
  void add(RetRole r, int group, size_t es) {
    const int Dx = r.Dx, n = Dx > 128 ? 2 : 1;
    const bool shares = group * n > 1;
    r.state = (int64_t)r.Dx * r.Dw;
    const int H = a.H, Dw = r.Dw;
    if (shares) {
      sum[sums++] = {nullptr, r.o, r.os, a.fill ? nullptr : a.lens, a.B, a.L, H / group, group * n, Dw};
      r.os = {(int64_t)a.L * H * n * Dw, (int64_t)H * n * Dw, (int64_t)n * Dw};
      r.o_f32 = 1;
    }
    for (int i = 0; i < n; ++i) {
      RetRole &to = a.role[a.roles++];
      const int64_t d = 128 * i;
      to = r;
      to.Dx = n == 1 ? Dx : i ? Dx - 128 : 128;
      to.x = static_cast<const char *>(r.x) + d * es;
      to.y = static_cast<const char *>(r.y) + d * es;
      if (r.start) to.start = r.start + d * r.start_rs;
      if (r.end) to.end = r.end + d * Dw;
      // until the workspace is there: where in it
      if (shares) to.o = reinterpret_cast<void *>((share + (size_t)i * Dw) * sizeof(float));
    }
    if (shares) {
      sum[sums - 1].part = reinterpret_cast<const float *>(share * sizeof(float));
      share += (size_t)a.B * a.L * H * n * Dw;
    }
  }

  la_status_t run(Dtype dt, cudaStream_t s) {
    const int parts = ret_parts(a, dt);
    return with_workspace(sizeof(float) * (share + ret_record_floats(a, dt, parts)), s, [&](void *ws) {
      char *base = static_cast<char *>(ws);
      for (int i = 0; i < a.roles; ++i)
        if (a.role[i].o_f32) a.role[i].o = base + reinterpret_cast<size_t>(a.role[i].o);
      ret_layout(&a, dt, parts, static_cast<float *>(ws) + share);
      const cudaError_t e = launch_retention(a, dt, parts, s);
      for (int i = 0; i < sums; ++i)
        sum[i].part = reinterpret_cast<const float *>(base + reinterpret_cast<size_t>(sum[i].part));
      return e == cudaSuccess ? launch_group_sums(sum, sums, dt, s) : e;
    });
  }
};

}  // namespace

extern "C" {

la_status_t la_forward_retention(const void *q, const void *k, const void *v, const float *S0,
                                 const int *lens, void *o, float *S, int B, int L, int H, int Hk,
                                 int D, int Dv, const long long *strides, const float *gamma,
                                 float scale, la_dtype_t dtype, void *stream) {
  const la_status_t st = check_sizes(B, L, H, Hk, D, Dv, scale, dtype);
  if (st != LA_OK) return st;
  Gammas g;
  if (!gammas_ok(gamma, H, &g)) return LA_ERR_INVALID_ARG;
  if (B == 0 || H == 0) return LA_OK;
  RetStrides s[4] = {dense(L, H, D), dense(L, Hk, D), dense(L, Hk, Dv), dense(L, H, Dv)};
  const int heads[4] = {H, Hk, Hk, H}, width[4] = {D, D, Dv, Dv};
  for (int i = 0; i < 4; ++i) {
    if (strides) s[i] = {strides[3 * i], strides[3 * i + 1], strides[3 * i + 2]};
    if (!strides_ok(&s[i], B, L, heads[i], width[i])) return LA_ERR_INVALID_ARG;
  }
  const bool any = L > 0;
  const size_t es = esize(dtype), state = sizeof(float) * (size_t)B * H * D * Dv;
  auto bytes = [&](int i) { return any ? span_of(s[i], B, L, heads[i], width[i], es) : (size_t)0; };
  const Buf ob = {o, bytes(3), any, true}, sb = {S, state, false, true};
  if (!buffers_ok({{q, bytes(0), any, false},
                   {k, bytes(1), any, false},
                   {v, bytes(2), any, false},
                   {S0, state, false, false},
                   ob,
                   sb}) ||
      !lens_ok(lens, B, {ob, sb}))
    return LA_ERR_INVALID_ARG;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (!any) {
    if (!S) return LA_OK;
    if (!S0) return zero(S, state, cs);
    return status(cudaMemcpyAsync(S, S0, state, cudaMemcpyDeviceToDevice, cs));
  }
  Plan p;
  p.a.lens = lens;
  p.a.B = B, p.a.L = L, p.a.H = H;
  p.a.lg = logs(g);
  p.add({q, k, v, o, s[0], s[1], s[2], s[3], 1, H / Hk, H / Hk, D, Dv, S0, S, nullptr, Dv, 1, 0, 1.f, 1.f, scale, 0, 0},
        1, es);
  return p.run(to_dtype(dtype), cs);
}

la_status_t la_backward_retention(const void *q, const void *k, const void *v, const void *dO,
                                  const float *S0, const float *dS, const int *lens, void *dq,
                                  void *dk, void *dv, float *dS0, int B, int L, int H, int Hk, int D,
                                  int Dv, const long long *strides, const float *gamma, float scale,
                                  la_dtype_t dtype, void *stream) {
  const la_status_t st = check_sizes(B, L, H, Hk, D, Dv, scale, dtype);
  if (st != LA_OK) return st;
  Gammas g;
  if (!gammas_ok(gamma, H, &g)) return LA_ERR_INVALID_ARG;
  if (B == 0 || H == 0) return LA_OK;
  RetStrides s[4] = {dense(L, H, D), dense(L, Hk, D), dense(L, Hk, Dv), dense(L, H, Dv)};
  const int heads[4] = {H, Hk, Hk, H}, width[4] = {D, D, Dv, Dv};
  for (int i = 0; i < 4; ++i) {
    if (strides) s[i] = {strides[3 * i], strides[3 * i + 1], strides[3 * i + 2]};
    if (!strides_ok(&s[i], B, L, heads[i], width[i])) return LA_ERR_INVALID_ARG;
  }
  const bool any = L > 0;
  const size_t es = esize(dtype), state = sizeof(float) * (size_t)B * H * D * Dv;
  const int64_t rows = (int64_t)B * L;
  auto bytes = [&](int i) { return any ? span_of(s[i], B, L, heads[i], width[i], es) : (size_t)0; };
  const Buf qb = {dq, (size_t)rows * H * D * es, any, true}, kb = {dk, (size_t)rows * Hk * D * es, any, true},
            vb = {dv, (size_t)rows * Hk * Dv * es, any, true}, sb = {dS0, state, false, true};
  if (!buffers_ok({{q, bytes(0), any, false},
                   {k, bytes(1), any, false},
                   {v, bytes(2), any, false},
                   {dO, bytes(3), any, false},
                   {S0, state, dS0 != nullptr, false},
                   {dS, state, false, false},
                   qb,
                   kb,
                   vb,
                   sb}) ||
      !lens_ok(lens, B, {qb, kb, vb, sb}))
    return LA_ERR_INVALID_ARG;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (!any) {
    if (!dS0) return LA_OK;
    if (!dS) return zero(dS0, state, cs);
    return status(cudaMemcpyAsync(dS0, dS, state, cudaMemcpyDeviceToDevice, cs));
  }
  const int group = H / Hk;
  Plan p;
  p.a.lens = lens;
  p.a.B = B, p.a.L = L, p.a.H = H;
  p.a.fill = lens != nullptr;
  p.a.lg = logs(g);
  // states of dq and dk are the transposes of S and U
  p.add({dO, v, k, dq, s[3], s[2], s[1], dense(L, H, D), 1, group, group, Dv, D, S0, nullptr, nullptr, 1, Dv, 0, 1.f,
         1.f, scale, 0, 0},
        1, es);
  p.add({v, dO, q, dk, s[2], s[3], s[0], dense(L, Hk, D), group, 1, 1, Dv, D, dS, nullptr, nullptr, 1, Dv, 0,
         1.f / scale, 1.f, scale, 1, 0},
        group, es);
  p.add({k, q, dO, dv, s[1], s[0], s[3], dense(L, Hk, Dv), group, 1, 1, D, Dv, dS, dS0, nullptr, Dv, 1, 0, 1.f / scale,
         scale, scale, 1, 0},
        group, es);
  return p.run(to_dtype(dtype), cs);
}

la_status_t la_decode_retention(const void *q, const void *k, const void *v, float *S,
                                const int *slots, void *o, int B, int pool, int H, int Hk, int D,
                                int Dv, long long ldq, long long ldk, long long ldv,
                                const float *gamma, float scale, la_dtype_t dtype, void *stream) {
  const la_status_t st = check_sizes(B, 1, H, Hk, D, Dv, scale, dtype);
  if (st != LA_OK) return st;
  if (pool < 0 || (!slots && pool < B)) return LA_ERR_INVALID_ARG;
  if ((int64_t)pool * H >= ((int64_t)1 << 31)) return LA_ERR_UNSUPPORTED;
  RetStepArgs a = {};
  if (!gammas_ok(gamma, H, &a.g)) return LA_ERR_INVALID_ARG;
  if (B == 0 || H == 0) return LA_OK;
  if (!stride_ok(&ldq, (int64_t)H * D) || !stride_ok(&ldk, (int64_t)Hk * D) || !stride_ok(&ldv, (int64_t)Hk * Dv))
    return LA_ERR_INVALID_ARG;
  const size_t es = esize(dtype);
  const Buf sb = {S, sizeof(float) * (size_t)pool * H * D * Dv, pool > 0, true},
            ob = {o, (size_t)B * H * Dv * es, true, true};
  if (!buffers_ok({{q, span(B, ldq, (int64_t)H * D, es), true, false},
                   {k, span(B, ldk, (int64_t)Hk * D, es), true, false},
                   {v, span(B, ldv, (int64_t)Hk * Dv, es), true, false},
                   sb,
                   ob}) ||
      !lens_ok(slots, B, {sb, ob}))
    return LA_ERR_INVALID_ARG;
  if (pool == 0) return LA_OK;
  a.q = q, a.k = k, a.v = v, a.S = S, a.slots = slots, a.o = o;
  a.B = B, a.H = H, a.Hk = Hk, a.D = D, a.Dv = Dv, a.pool = pool;
  a.ldq = ldq, a.ldk = ldk, a.ldv = ldv;
  a.scale = scale;
  return status(launch_retention_step(a, to_dtype(dtype), static_cast<cudaStream_t>(stream)));
}

la_status_t la_select_beams(const void *logits, const float *scores, const unsigned char *finished,
                            float *out_scores, int *parents, int *tokens, int B, int K, int V, int n,
                            long long ld, int eos, la_dtype_t dtype, void *stream) {
  if (!dtype_ok(dtype) || B < 0 || K <= 0 || V <= 0 || n <= 0) return LA_ERR_INVALID_ARG;
  if (ld == 0) ld = V;
  if (ld < V || (int64_t)n > (int64_t)K * V) return LA_ERR_INVALID_ARG;
  if (finished && (eos < 0 || eos >= V)) return LA_ERR_INVALID_ARG;
  if (K > kMaxBeams || n > kMaxBest || V > (1 << 30) || (int64_t)B * K >= (1 << 26) || ld >= ((int64_t)1 << 40))
    return LA_ERR_UNSUPPORTED;
  if (B == 0) return LA_OK;
  const size_t es = esize(dtype), best = sizeof(float) * (size_t)B * n;
  const int64_t rows = (int64_t)B * K;
  // no vector access needs these on a 16-byte boundary
  const Buf l[] = {{logits, span(rows, ld, V, es), true, false},
                   {scores, sizeof(float) * (size_t)rows, true, false},
                   {finished, (size_t)rows, false, false},
                   {out_scores, best, true, true},
                   {parents, best, true, true},
                   {tokens, best, true, true}};
  const size_t align[] = {es, 4, 1, 4, 4, 4};
  for (int i = 0; i < 6; ++i) {
    if (l[i].required && !l[i].p) return LA_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(l[i].p) % align[i]) return LA_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if ((l[i].written || l[j].written) && overlap(l[i], l[j])) return LA_ERR_INVALID_ARG;
  }
  const BeamArgs a = {logits, scores, finished, out_scores, parents, tokens, B, K, V, n, eos, ld};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return with_workspace(beams_workspace_bytes(B, K, V, n), s,
                        [&](void *ws) { return launch_select_beams(a, to_dtype(dtype), ws, s); });
}

la_status_t la_reorder_states(void *const *states, const long long *bytes, int count,
                              const int *parents, int B, int K, void *stream) {
  if (count < 0 || B < 0 || K <= 0 || (count > 0 && (!states || !bytes))) return LA_ERR_INVALID_ARG;
  if (K > kMaxBeams || (int64_t)B * K >= (1 << 26)) return LA_ERR_UNSUPPORTED;
  if (B == 0 || count == 0) return LA_OK;
  const int64_t rows = (int64_t)B * K;
  const Buf pb = {parents, sizeof(int) * (size_t)rows, true, false};
  if (!parents || (reinterpret_cast<uintptr_t>(parents) & 3u)) return LA_ERR_INVALID_ARG;
  for (int i = 0; i < count; ++i) {
    if (bytes[i] < 0 || (bytes[i] > 0 && !states[i])) return LA_ERR_INVALID_ARG;
    if (bytes[i] > ((int64_t)1 << 46) / rows) return LA_ERR_UNSUPPORTED;
    const Buf s = {states[i], (size_t)(rows * bytes[i]), false, true};
    if (overlap(s, pb)) return LA_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(s, {states[j], (size_t)(rows * bytes[j]), false, true})) return LA_ERR_INVALID_ARG;
  }
  for (int i = 0; i < count; i += kReorderStates) {
    int64_t b[kReorderStates];
    const int m = count - i < kReorderStates ? count - i : kReorderStates;
    for (int j = 0; j < m; ++j) b[j] = bytes[i + j];
    const la_status_t st =
        status(launch_reorder_states(states + i, b, m, parents, B, K, static_cast<cudaStream_t>(stream)));
    if (st != LA_OK) return st;
  }
  return LA_OK;
}

}  // extern "C"
