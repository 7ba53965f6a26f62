// C ABI of the selective scan, its short convolution and the norms around a
// block: argument validation, workspace and dispatch.  Every check runs
// before the first CUDA call.
#include <math.h>
#include <stdint.h>

#include <initializer_list>
#include <mutex>

#include "../../include/linattn.h"
#include "kernels.h"

using namespace linattn;

namespace {

constexpr int kMaxWidth = 65536;
// Tokens of a batch: parts and runs are rounded up in 32 bits, by less than
// 2^16 in all.
constexpr int64_t kMaxTokens = ((int64_t)1 << 31) - (1 << 16);

// A buffer of a call: where it is, how many bytes its elements span, and what
// the call needs of it.
struct Buf {
  const void *p;
  size_t bytes;
  bool required, written;
};

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool overlap(const Buf &a, const Buf &b) {
  if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.bytes && y < x + a.bytes;
}

// Required buffers present, all of them 16-byte aligned, no written buffer
// over any other.
bool buffers_ok(std::initializer_list<Buf> l) {
  for (const Buf *a = l.begin(); a != l.end(); ++a) {
    if (a->required && !a->p) return false;
    if (!aligned16(a->p)) return false;
    for (const Buf *b = a + 1; b != l.end(); ++b)
      if ((a->written || b->written) && overlap(*a, *b)) return false;
  }
  return true;
}

bool dtype_ok(la_dtype_t dt) { return dt == LA_F32 || dt == LA_BF16; }
size_t esize(la_dtype_t dt) { return dt == LA_F32 ? 4 : 2; }
Dtype to_dtype(la_dtype_t dt) { return dt == LA_F32 ? kF32 : kBF16; }

la_status_t status(cudaError_t e) {
  if (e == cudaSuccess) return LA_OK;
  forget_error();
  return e == cudaErrorNotSupported ? LA_ERR_UNSUPPORTED : LA_ERR_CUDA;
}

// Bytes that `rows` rows of `width` elements span, `ld` elements apart.
size_t span(int64_t rows, int64_t ld, int64_t width, size_t es) {
  return rows > 0 ? (size_t)((rows - 1) * ld + width) * es : 0;
}

// Token strides: 0 stands for dense rows; a multiple of 8 elements otherwise.
bool stride_ok(long long *ld, int64_t width) {
  if (*ld == 0) *ld = width;
  return *ld >= width && *ld % 8 == 0 && *ld < ((long long)1 << 40);
}

la_status_t check_width(int B, int L, int E) {
  if (B < 0 || L < 0 || E < 0) return LA_ERR_INVALID_ARG;
  if (E % 8 != 0 || E > kMaxWidth) return LA_ERR_UNSUPPORTED;
  if ((int64_t)B * (L > 0 ? L : 1) >= kMaxTokens || (int64_t)B * E >= ((int64_t)1 << 31))
    return LA_ERR_UNSUPPORTED;
  return LA_OK;
}

// Workspaces come from a pool of the library's own, per device: the default
// pool hands memory back at every synchronisation, and mapping it again costs
// more than a short call.  The pool keeps up to half a gigabyte.
cudaMemPool_t workspace_pool() {
  constexpr int kMaxDev = 64;
  static cudaMemPool_t pools[kMaxDev] = {};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return nullptr;
  std::lock_guard<std::mutex> lock(mu);
  if (!pools[dev]) {
    // the first call may be inside a stream capture, which creating a pool
    // does not touch but a capture's stricter modes would end over
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    if (cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess) return nullptr;
    cudaMemPoolProps props = {};
    props.allocType = cudaMemAllocationTypePinned;
    props.location.type = cudaMemLocationTypeDevice;
    props.location.id = dev;
    cudaMemPool_t pool = nullptr;
    uint64_t keep = (uint64_t)1 << 29;
    bool ok = cudaMemPoolCreate(&pool, &props) == cudaSuccess;
    if (ok && cudaMemPoolSetAttribute(pool, cudaMemPoolAttrReleaseThreshold, &keep) != cudaSuccess) {
      cudaMemPoolDestroy(pool);
      ok = false;
    }
    if (cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess) ok = false;
    if (!ok) return nullptr;
    pools[dev] = pool;
  }
  return pools[dev];
}

// Runs f with a stream-ordered workspace of `bytes` (none for 0).
template <typename F>
la_status_t with_workspace(size_t bytes, cudaStream_t s, F &&f) {
  if (bytes == 0) return status(f(nullptr));
  cudaMemPool_t pool = workspace_pool();
  void *ws = nullptr;
  if (!pool || cudaMallocFromPoolAsync(&ws, bytes, pool, s) != cudaSuccess)
    return status(cudaErrorMemoryAllocation);
  const cudaError_t e = f(ws);
  const cudaError_t ef = cudaFreeAsync(ws, s);
  return status(e != cudaSuccess ? e : ef);
}

la_status_t zero(void *p, size_t bytes, cudaStream_t s) {
  return p && bytes ? status(cudaMemsetAsync(p, 0, bytes, s)) : LA_OK;
}

la_status_t check_scan(int B, int L, int E, int N, int G, la_dtype_t dt) {
  if (!dtype_ok(dt) || N <= 0 || G <= 0) return LA_ERR_INVALID_ARG;
  const la_status_t st = check_width(B, L, E);
  if (st != LA_OK) return st;
  if (!selective_states_supported(N)) return LA_ERR_UNSUPPORTED;
  if (E % G != 0) return LA_ERR_INVALID_ARG;
  if ((E / G) % 8 != 0) return LA_ERR_UNSUPPORTED;
  return LA_OK;
}

}  // namespace

extern "C" {

la_status_t la_forward_selective(const void *x, const void *dt, const float *A, const void *Bm,
                                 const void *Cm, const float *D, const void *z,
                                 const float *dt_bias, const float *h0, const int *lens, void *y,
                                 float *hN, int B, int L, int E, int N, int G, long long ldx,
                                 long long lddt, long long ldz, long long ldb, long long ldc,
                                 int softplus, la_dtype_t dtype, void *stream) {
  const la_status_t st = check_scan(B, L, E, N, G, dtype);
  if (st != LA_OK) return st;
  const int64_t GN = (int64_t)G * N, rows = (int64_t)B * L;
  if (!stride_ok(&ldx, E) || !stride_ok(&lddt, E) || !stride_ok(&ldz, E) || !stride_ok(&ldb, GN) ||
      !stride_ok(&ldc, GN))
    return LA_ERR_INVALID_ARG;
  if (B == 0 || E == 0) return LA_OK;
  const size_t es = esize(dtype), state = sizeof(float) * (size_t)B * E * N;
  const bool any = L > 0;
  if (reinterpret_cast<uintptr_t>(lens) & 3u) return LA_ERR_INVALID_ARG;
  if (!buffers_ok({{x, span(rows, ldx, E, es), any, false},
                   {dt, span(rows, lddt, E, es), any, false},
                   {Bm, span(rows, ldb, GN, es), any, false},
                   {Cm, span(rows, ldc, GN, es), any, false},
                   {z, span(rows, ldz, E, es), false, false},
                   {A, sizeof(float) * (size_t)E * N, true, false},
                   {D, sizeof(float) * (size_t)E, false, false},
                   {dt_bias, sizeof(float) * (size_t)E, false, false},
                   {h0, state, false, false},
                   {y, (size_t)rows * E * es, any, true},
                   {hN, state, false, true}}))
    return LA_ERR_INVALID_ARG;
  const Buf lb = {lens, sizeof(int) * (size_t)B, false, false};
  if (overlap(lb, {y, (size_t)rows * E * es, false, true}) || overlap(lb, {hN, state, false, true}))
    return LA_ERR_INVALID_ARG;
  const ScanArgs a = {x, dt, z, Bm, Cm, A, D, dt_bias, h0, lens, y, hN, B, L, E, N, G,
                      ldx, lddt, ldz, ldb, ldc, softplus != 0};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int S = selective_parts(B, L, E, N, G, to_dtype(dtype), lens != nullptr);
  return with_workspace(selective_workspace_bytes(B, E, N, S, lens != nullptr), s, [&](void *ws) {
    return launch_selective(a, to_dtype(dtype), ws, S, s);
  });
}

la_status_t la_decode_selective(const void *x, const void *dt, const float *A, const void *Bm,
                                const void *Cm, const float *D, const void *z,
                                const float *dt_bias, float *h, void *y, int B, int E, int N,
                                int G, long long ldx, long long lddt, long long ldz,
                                long long ldb, long long ldc, int softplus, la_dtype_t dtype,
                                void *stream) {
  const la_status_t st = check_scan(B, 1, E, N, G, dtype);
  if (st != LA_OK) return st;
  const int64_t GN = (int64_t)G * N;
  if (!stride_ok(&ldx, E) || !stride_ok(&lddt, E) || !stride_ok(&ldz, E) || !stride_ok(&ldb, GN) ||
      !stride_ok(&ldc, GN))
    return LA_ERR_INVALID_ARG;
  if (B == 0 || E == 0) return LA_OK;
  const size_t es = esize(dtype);
  if (!buffers_ok({{x, span(B, ldx, E, es), true, false},
                   {dt, span(B, lddt, E, es), true, false},
                   {Bm, span(B, ldb, GN, es), true, false},
                   {Cm, span(B, ldc, GN, es), true, false},
                   {z, span(B, ldz, E, es), false, false},
                   {A, sizeof(float) * (size_t)E * N, true, false},
                   {D, sizeof(float) * (size_t)E, false, false},
                   {dt_bias, sizeof(float) * (size_t)E, false, false},
                   {h, sizeof(float) * (size_t)B * E * N, true, true},
                   {y, (size_t)B * E * es, true, true}}))
    return LA_ERR_INVALID_ARG;
  const ScanArgs a = {x, dt, z, Bm, Cm, A, D, dt_bias, nullptr, nullptr, y, h, B, 1, E, N, G,
                      ldx, lddt, ldz, ldb, ldc, softplus != 0};
  return status(launch_selective_step(a, to_dtype(dtype), static_cast<cudaStream_t>(stream)));
}

la_status_t la_backward_selective(const void *x, const void *dt, const float *A, const void *Bm,
                                  const void *Cm, const float *D, const void *z,
                                  const float *dt_bias, const float *h0, const void *dy,
                                  const float *dhN, void *dx, void *ddt, float *dA, void *dBm,
                                  void *dCm, float *dD, void *dz, float *ddt_bias, float *dh0,
                                  int B, int L, int E, int N, int G, long long ldx,
                                  long long lddt, long long ldz, long long ldb, long long ldc,
                                  int softplus, la_dtype_t dtype, void *stream) {
  const la_status_t st = check_scan(B, L, E, N, G, dtype);
  if (st != LA_OK) return st;
  const int64_t GN = (int64_t)G * N, rows = (int64_t)B * L;
  if (!stride_ok(&ldx, E) || !stride_ok(&lddt, E) || !stride_ok(&ldz, E) || !stride_ok(&ldb, GN) ||
      !stride_ok(&ldc, GN))
    return LA_ERR_INVALID_ARG;
  if (E == 0) return LA_OK;
  const size_t es = esize(dtype), state = sizeof(float) * (size_t)B * E * N;
  const size_t tok = (size_t)rows * E * es, bc = (size_t)rows * GN * es;
  const size_t nA = sizeof(float) * (size_t)E * N, nE = sizeof(float) * (size_t)E;
  const bool any = rows > 0;
  // a gradient needs its input; dz and z go together
  if ((dD && !D) || (ddt_bias && !dt_bias) || (dh0 && !h0)) return LA_ERR_INVALID_ARG;
  if (any && (dz != nullptr) != (z != nullptr)) return LA_ERR_INVALID_ARG;
  if (!buffers_ok({{x, span(rows, ldx, E, es), any, false},
                   {dt, span(rows, lddt, E, es), any, false},
                   {Bm, span(rows, ldb, GN, es), any, false},
                   {Cm, span(rows, ldc, GN, es), any, false},
                   {z, span(rows, ldz, E, es), false, false},
                   {A, nA, B > 0, false},
                   {D, nE, false, false},
                   {dt_bias, nE, false, false},
                   {h0, state, false, false},
                   {dy, tok, any, false},
                   {dhN, state, false, false},
                   {dx, tok, any, true},
                   {ddt, tok, any, true},
                   {dA, nA, true, true},
                   {dBm, bc, any, true},
                   {dCm, bc, any, true},
                   {dD, nE, false, true},
                   {dz, tok, false, true},
                   {ddt_bias, nE, false, true},
                   {dh0, state, false, true}}))
    return LA_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (B == 0) {  // nothing contributes to the parameters' gradients
    la_status_t r = zero(dA, nA, s);
    if (r == LA_OK) r = zero(dD, nE, s);
    return r == LA_OK ? zero(ddt_bias, nE, s) : r;
  }
  const ScanArgs a = {x, dt, z, Bm, Cm, A, D, dt_bias, h0, nullptr, nullptr, nullptr, B, L, E, N, G,
                      ldx, lddt, ldz, ldb, ldc, softplus != 0};
  const ScanGrads g = {dy, dhN, dx, ddt, dz, dBm, dCm, dA, dD, ddt_bias, dh0};
  return with_workspace(selective_backward_workspace_bytes(B, L, E, N, G), s, [&](void *ws) {
    return launch_selective_backward(a, g, to_dtype(dtype), ws, s);
  });
}

la_status_t la_forward_conv(const void *x, const float *w, const float *bias, const void *state,
                            const int *lens, void *y, void *state_out, int B, int L, int E, int W,
                            long long ldx, int silu, la_dtype_t dtype, void *stream) {
  if (!dtype_ok(dtype) || W <= 0) return LA_ERR_INVALID_ARG;
  const la_status_t st = check_width(B, L, E);
  if (st != LA_OK) return st;
  if (W < 2 || W > 4) return LA_ERR_UNSUPPORTED;
  if (!stride_ok(&ldx, E)) return LA_ERR_INVALID_ARG;
  if (B == 0 || E == 0) return LA_OK;
  const int64_t rows = (int64_t)B * L;
  const size_t es = esize(dtype), nst = (size_t)B * (W - 1) * E * es;
  if (reinterpret_cast<uintptr_t>(lens) & 3u) return LA_ERR_INVALID_ARG;
  if (!buffers_ok({{x, span(rows, ldx, E, es), L > 0, false},
                   {w, sizeof(float) * (size_t)E * W, true, false},
                   {bias, sizeof(float) * (size_t)E, false, false},
                   {state, nst, false, false},
                   {y, (size_t)rows * E * es, L > 0, true},
                   {state_out, nst, false, true}}))
    return LA_ERR_INVALID_ARG;
  const Buf lb = {lens, sizeof(int) * (size_t)B, false, false};
  if (overlap(lb, {y, (size_t)rows * E * es, false, true}) ||
      overlap(lb, {state_out, nst, false, true}))
    return LA_ERR_INVALID_ARG;
  if (L == 0 && !state_out) return LA_OK;
  const ConvArgs a = {x, w, bias, state, lens, y, state_out, B, L, E, W, ldx, silu != 0};
  return status(launch_conv(a, to_dtype(dtype), static_cast<cudaStream_t>(stream)));
}

la_status_t la_decode_conv(const void *x, const float *w, const float *bias, void *state, void *y,
                           int B, int E, int W, long long ldx, int silu, la_dtype_t dtype,
                           void *stream) {
  if (!dtype_ok(dtype) || W <= 0) return LA_ERR_INVALID_ARG;
  const la_status_t st = check_width(B, 1, E);
  if (st != LA_OK) return st;
  if (W < 2 || W > 4) return LA_ERR_UNSUPPORTED;
  if (!stride_ok(&ldx, E)) return LA_ERR_INVALID_ARG;
  if (B == 0 || E == 0) return LA_OK;
  const size_t es = esize(dtype);
  if (!buffers_ok({{x, span(B, ldx, E, es), true, false},
                   {w, sizeof(float) * (size_t)E * W, true, false},
                   {bias, sizeof(float) * (size_t)E, false, false},
                   {state, (size_t)B * (W - 1) * E * es, true, true},
                   {y, (size_t)B * E * es, true, true}}))
    return LA_ERR_INVALID_ARG;
  const ConvArgs a = {x, w, bias, nullptr, nullptr, y, state, B, 1, E, W, ldx, silu != 0};
  return status(launch_conv_step(a, to_dtype(dtype), static_cast<cudaStream_t>(stream)));
}

la_status_t la_backward_conv(const void *x, const float *w, const float *bias, const void *state,
                             const void *dy, void *dx, float *dw, float *dbias, void *dstate,
                             int B, int L, int E, int W, long long ldx, int silu,
                             la_dtype_t dtype, void *stream) {
  if (!dtype_ok(dtype) || W <= 0) return LA_ERR_INVALID_ARG;
  const la_status_t st = check_width(B, L, E);
  if (st != LA_OK) return st;
  if (W < 2 || W > 4) return LA_ERR_UNSUPPORTED;
  if (!stride_ok(&ldx, E)) return LA_ERR_INVALID_ARG;
  if (E == 0) return LA_OK;
  if ((dbias && !bias) || (dstate && !state)) return LA_ERR_INVALID_ARG;
  const int64_t rows = (int64_t)B * L;
  const bool any = rows > 0;
  const size_t es = esize(dtype), nst = (size_t)B * (W - 1) * E * es, tok = (size_t)rows * E * es;
  const size_t nw = sizeof(float) * (size_t)E * W, nb = sizeof(float) * (size_t)E;
  if (!buffers_ok({{x, span(rows, ldx, E, es), any, false},
                   {w, nw, true, false},
                   {bias, nb, false, false},
                   {state, nst, false, false},
                   {dy, tok, any, false},
                   {dx, tok, any, true},
                   {dw, nw, true, true},
                   {dbias, nb, false, true},
                   {dstate, nst, false, true}}))
    return LA_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!any) {
    la_status_t r = zero(dw, nw, s);
    if (r == LA_OK) r = zero(dbias, nb, s);
    return r == LA_OK ? zero(dstate, nst, s) : r;
  }
  const ConvArgs a = {x, w, bias, state, nullptr, nullptr, nullptr, B, L, E, W, ldx, silu != 0};
  const ConvGrads g = {dy, dx, dstate, dw, dbias};
  return with_workspace(conv_backward_workspace_bytes(B, L, E, W, to_dtype(dtype)), s, [&](void *ws) {
    return launch_conv_backward(a, g, to_dtype(dtype), ws, s);
  });
}

static la_status_t check_norm_gate(int B, int H, int L, int D, float eps, la_dtype_t dtype) {
  if (!dtype_ok(dtype) || B < 0 || H < 0 || L < 0 || D <= 0) return LA_ERR_INVALID_ARG;
  if (!isfinite(eps) || eps < 0.f) return LA_ERR_INVALID_ARG;
  if (D % 8 != 0 || D > 8192 || (int64_t)H * D > kMaxWidth) return LA_ERR_UNSUPPORTED;
  if ((int64_t)B * L * H >= ((int64_t)1 << 31)) return LA_ERR_UNSUPPORTED;
  return LA_OK;
}

la_status_t la_forward_norm_gate(const void *y, const void *gate, const float *w, void *out, int B,
                                 int H, int L, int D, int heads_first, int gate_first, float eps,
                                 la_dtype_t dtype, void *stream) {
  const la_status_t st = check_norm_gate(B, H, L, D, eps, dtype);
  if (st != LA_OK) return st;
  const int64_t n = (int64_t)B * H * L * D;
  if (n == 0) return LA_OK;
  const size_t bytes = (size_t)n * esize(dtype);
  if (!buffers_ok({{y, bytes, true, false},
                   {gate, bytes, true, false},
                   {w, sizeof(float) * (size_t)H * D, false, false},
                   {out, bytes, true, true}}))
    return LA_ERR_INVALID_ARG;
  const NormGateArgs a = {y, gate, w, out, B, H, L, D, eps, heads_first != 0, gate_first != 0};
  return status(launch_norm_gate(a, to_dtype(dtype), static_cast<cudaStream_t>(stream)));
}

la_status_t la_backward_norm_gate(const void *y, const void *gate, const float *w, const void *dout,
                                  void *dy, void *dgate, float *dw, int B, int H, int L, int D,
                                  int heads_first, int gate_first, float eps, la_dtype_t dtype,
                                  void *stream) {
  const la_status_t st = check_norm_gate(B, H, L, D, eps, dtype);
  if (st != LA_OK) return st;
  if (dw && !w) return LA_ERR_INVALID_ARG;
  const int64_t n = (int64_t)B * H * L * D;
  const size_t bytes = (size_t)n * esize(dtype), nw = sizeof(float) * (size_t)H * D;
  if (!buffers_ok({{y, bytes, n > 0, false},
                   {gate, bytes, n > 0, false},
                   {w, nw, false, false},
                   {dout, bytes, n > 0, false},
                   {dy, bytes, n > 0, true},
                   {dgate, bytes, n > 0, true},
                   {dw, nw, false, true}}))
    return LA_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (n == 0) return zero(dw, nw, s);
  const NormGateArgs a = {y, gate, w, nullptr, B, H, L, D, eps, heads_first != 0, gate_first != 0};
  const NormGateGrads g = {dout, dy, dgate, dw};
  return with_workspace(dw ? norm_gate_backward_workspace_bytes(B, H, L, D) : 0, s, [&](void *ws) {
    return launch_norm_gate_backward(a, g, to_dtype(dtype), ws, s);
  });
}

static la_status_t check_norm_residual(long long rows, int E, float scale, float eps,
                                       la_dtype_t dtype) {
  if (!dtype_ok(dtype) || rows < 0 || E < 0) return LA_ERR_INVALID_ARG;
  if (!isfinite(eps) || eps < 0.f || !isfinite(scale)) return LA_ERR_INVALID_ARG;
  if (E % 8 != 0 || E > 8192 || rows >= ((long long)1 << 31)) return LA_ERR_UNSUPPORTED;
  return LA_OK;
}

la_status_t la_forward_norm_residual(const void *x, const void *residual, const float *w, void *o,
                                     void *r, long long rows, int E, float scale, float eps,
                                     la_dtype_t dtype, void *stream) {
  const la_status_t st = check_norm_residual(rows, E, scale, eps, dtype);
  if (st != LA_OK) return st;
  if (rows == 0 || E == 0) return LA_OK;
  const size_t bytes = (size_t)rows * E * esize(dtype);
  if (!buffers_ok({{x, bytes, true, false},
                   {residual, bytes, false, false},
                   {w, sizeof(float) * (size_t)E, false, false},
                   {o, bytes, true, true},
                   {r, bytes, true, true}}))
    return LA_ERR_INVALID_ARG;
  const NormResidualArgs a = {x, residual, w, o, r, rows, E, scale, eps};
  return status(launch_norm_residual(a, to_dtype(dtype), static_cast<cudaStream_t>(stream)));
}

la_status_t la_backward_norm_residual(const void *r, const float *w, const void *dout,
                                      const void *dr, void *dresidual, void *dx, float *dw,
                                      long long rows, int E, float scale, float eps,
                                      la_dtype_t dtype, void *stream) {
  const la_status_t st = check_norm_residual(rows, E, scale, eps, dtype);
  if (st != LA_OK) return st;
  if (E == 0) return LA_OK;
  if (dw && !w) return LA_ERR_INVALID_ARG;
  const bool any = rows > 0;
  if (any && !dx && scale != 1.f) return LA_ERR_INVALID_ARG;
  const size_t bytes = (size_t)rows * E * esize(dtype), nw = sizeof(float) * (size_t)E;
  if (!buffers_ok({{r, bytes, any, false},
                   {w, nw, false, false},
                   {dout, bytes, any, false},
                   {dr, bytes, false, false},
                   {dresidual, bytes, any, true},
                   {dx, bytes, false, true},
                   {dw, nw, false, true}}))
    return LA_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!any) return zero(dw, nw, s);
  const NormResidualArgs a = {nullptr, nullptr, w, nullptr, const_cast<void *>(r), rows, E, scale, eps};
  const NormResidualGrads g = {dout, dr, dresidual, dx, dw};
  return with_workspace(dw ? norm_residual_backward_workspace_bytes(rows, E) : 0, s, [&](void *ws) {
    return launch_norm_residual_backward(a, g, to_dtype(dtype), ws, s);
  });
}

}  // extern "C"
