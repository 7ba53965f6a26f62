// What the entry points share: checks of buffers, statuses, workspaces.
#pragma once
#include <math.h>
#include <stdint.h>

#include <initializer_list>

#include "../../include/linattn.h"
#include "kernels.h"

namespace linattn {

// A buffer of a call: where it is, how many bytes its elements span, and what
// the call needs of it.
struct Buf {
  const void *p;
  size_t bytes;
  bool required, written;
};

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool overlap(const Buf &a, const Buf &b) {
  if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.bytes && y < x + a.bytes;
}

// Required buffers present, all of them 16-byte aligned, no written buffer
// over any other.
inline bool buffers_ok(std::initializer_list<Buf> l) {
  for (const Buf *a = l.begin(); a != l.end(); ++a) {
    if (a->required && !a->p) return false;
    if (!aligned16(a->p)) return false;
    for (const Buf *b = a + 1; b != l.end(); ++b)
      if ((a->written || b->written) && overlap(*a, *b)) return false;
  }
  return true;
}

inline bool dtype_ok(la_dtype_t dt) { return dt == LA_F32 || dt == LA_BF16; }
inline size_t esize(la_dtype_t dt) { return dt == LA_F32 ? 4 : 2; }
inline Dtype to_dtype(la_dtype_t dt) { return dt == LA_F32 ? kF32 : kBF16; }

inline la_status_t status(cudaError_t e) {
  if (e == cudaSuccess) return LA_OK;
  forget_error();
  return e == cudaErrorNotSupported ? LA_ERR_UNSUPPORTED : LA_ERR_CUDA;
}

// Bytes that `rows` rows of `width` elements span, `ld` elements apart.
inline size_t span(int64_t rows, int64_t ld, int64_t width, size_t es) {
  return rows > 0 ? (size_t)((rows - 1) * ld + width) * es : 0;
}

// Token strides: 0 stands for dense rows; a multiple of 8 elements otherwise.
inline bool stride_ok(long long *ld, int64_t width) {
  if (*ld == 0) *ld = width;
  return *ld >= width && *ld % 8 == 0 && *ld < ((long long)1 << 40);
}

// Workspaces come from a pool of the library's own, per device: the default
// pool hands memory back at every synchronisation, and mapping it again costs
// more than a short call.  The pool keeps up to half a gigabyte.
cudaMemPool_t workspace_pool();

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

inline la_status_t zero(void *p, size_t bytes, cudaStream_t s) {
  return p && bytes ? status(cudaMemsetAsync(p, 0, bytes, s)) : LA_OK;
}

}  // namespace linattn
