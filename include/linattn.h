/*
 * linattn.h -- C ABI of the GB300 (sm_103a) kernelized linear-attention
 * library.
 *
 * The library computes linear attention with the Linear Transformer feature
 * map phi(x) = elu(x) + 1 (x + 1 for x > 0, exp(x) otherwise):
 *
 *   o_i = phi(q_i)^T S_i / (phi(q_i)^T z_i + eps)
 *
 * in the three forms described on "Linear Attention Mechanisms"
 * (dileepadev.github.io) and "Attention-Free / Sub-Quadratic Architectures"
 * (blog.vguerra.net):
 *   - causal:     S_i = gamma S_{i-1} + phi(k_i) v_i^T, z_i = gamma z_{i-1} +
 *                 phi(k_i) ("Recurrent Reformulation"; "The recurrent form
 *                 (causal)"; fixed decay gamma from "Gating and Selective
 *                 State Updates" / "Evolution: add decay/gating", applied to
 *                 both S and z);
 *   - non-causal: S = sum_j phi(k_j) v_j^T and z = sum_j phi(k_j) over every
 *                 key, shared by every query ("The Kernel Trick for
 *                 Attention"; "Linear Attention (the core trick)");
 *   - decode:     one step of the causal recurrence on a caller-held state;
 *   - gated:      the causal recurrence with a data-dependent gate per key
 *                 feature and token ("Gating and Selective State Updates",
 *                 gated linear attention), forward and decode step;
 *   - Performer:  random exponential features in place of elu + 1
 *                 ("Choosing the Feature Map"), the map alone and the
 *                 attention over it.
 * Beside them stand the selective state space scan with its short causal
 * convolution, the norms before and after a mixing block (see "Selective
 * state space scan" below), retention (the decayed form without feature map and
 * normaliser) and beam search over decode states.
 * eps is added to the denominator after the dot product, as in the NumPy
 * listing on "Linear Attention Mechanisms" (sadullah.online), "The linear
 * attention trick".
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Tensors are dense, row-major, contiguous, in DEVICE memory:
 *     q, k  [B][H][N][D]      v, o  [B][H][N][Dv]     (forward / prefill)
 *     q, k  [B][H][D]         v, o  [B][H][Dv]        (decode step)
 *     S     [B][H][D][Dv] fp32                        (state, caller-owned)
 *     z     [B][H][D]     fp32
 *   q, k, v and o all have the element type `dtype` (LA_F32 or LA_BF16).
 *   Every device pointer must be 16-byte aligned.
 * - gamma is a HOST array of H floats in [0, 1] (one decay per head), or
 *   NULL meaning 1 for every head.  The library copies the values during the
 *   call; the caller keeps ownership.
 * - stream is a cudaStream_t passed as void* (NULL = legacy default stream),
 *   so that this header needs no CUDA header to compile.
 *   Every call is asynchronous on that stream and never synchronises.  The
 *   caller owns all buffers; the library keeps no state between calls
 *   (except la_forward_host's copy streams and memory pool, and the
 *   allocation-free entry point's fixed array, all per device).
 * - Arguments are validated before any CUDA call, so a rejected call has no
 *   side effect.  A launch failure returns LA_ERR_CUDA; an error raised while
 *   a kernel runs surfaces at the caller's next synchronisation.
 * - Supported sizes: D and Dv in {64, 128}; H <= 256; B*H*N < 2^31 tokens per
 *   call.  B, H or N equal to 0 is an empty call that returns LA_OK (for
 *   la_prefill_state with N = 0 the state is set to zero).
 * - Arithmetic: fp32 state and accumulation.  For LA_BF16 the tensor-core
 *   kernels round phi(q), phi(k), the decay-weighted values and the
 *   intra-chunk weights to bf16 as matrix-multiply operands; o is rounded to
 *   bf16 (round to nearest even).
 *
 * Example: a causal pass with one decay per head, then decode steps that
 * continue from its state (all buffers device memory of the documented
 * sizes; error handling shortened):
 *
 *   float gamma[H];                        // host, one decay per head
 *   la_status_t st = la_forward_state(q, k, v, o, S, z, B, H, N, D, Dv,
 *                                     gamma, 1e-6f, LA_BF16, stream);
 *   if (st != LA_OK) fprintf(stderr, "%s\n", la_status_string(st));
 *   for (int t = 0; t < steps; ++t)        // S, z updated in place
 *     st = la_decode_step(q_t, k_t, v_t, S, z, o_t, B, H, D, Dv, gamma,
 *                         1e-6f, LA_BF16, stream);
 *   cudaStreamSynchronize(stream);         // kernel faults surface here
 */
#ifndef LINATTN_H
#define LINATTN_H

#include <stddef.h>

#if defined(__GNUC__)
#define LA_API __attribute__((visibility("default")))
#else
#define LA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  LA_OK = 0,
  LA_ERR_INVALID_ARG = 1, /* null/misaligned pointer, bad size, bad eps or
                             gamma, aliasing output, gamma != 1 when
                             non-causal */
  LA_ERR_UNSUPPORTED = 2, /* valid but not implemented: D or Dv not in
                             {64, 128}, H > 256, too many tokens */
  LA_ERR_CUDA = 3         /* a CUDA call or kernel launch failed */
} la_status_t;

typedef enum { LA_F32 = 0, LA_BF16 = 1 } la_dtype_t;

/*
 * Forward pass over whole sequences.
 *   causal != 0: o_i uses keys/values j <= i (inclusive), decayed by
 *                gamma[h]^(i-j).
 *   causal == 0: o_i uses every key/value of its (b, h); gamma must be NULL
 *                or all 1 (otherwise LA_ERR_INVALID_ARG).  The non-causal
 *                path needs a stream-ordered workspace of about
 *                B*H*(D*Dv + D)*4*(1 + ceil(N/4096)) bytes, taken with
 *                cudaMallocAsync on `stream` and released on it.
 * q, k: [B][H][N][D]; v: [B][H][N][Dv]; o: [B][H][N][Dv] (written).  o must
 * not overlap q, k or v.  eps must be finite and >= 0.
 * Defined on the pages "Linear Attention Mechanisms" (dileepadev.github.io):
 * causal by "Recurrent Reformulation" (S_i, z_i and the read-out o_i), with
 * the per-head decay of "Gating and Selective State Updates" (RetNet, weight
 * gamma^(t-j)) on both S and z; non-causal by "The Kernel Trick for
 * Attention" (S and z once over every key); eps as in the NumPy listing of
 * "Linear Attention Mechanisms" (sadullah.online), "The linear attention
 * trick".
 */
LA_API la_status_t la_forward(const void *q, const void *k, const void *v, void *o,
                       int B, int H, int N, int D, int Dv, int causal,
                       const float *gamma, float eps, la_dtype_t dtype,
                       void *stream);

/*
 * la_forward on HOST buffers: q, k, v are read from host memory and o is
 * written to host memory (same shapes, dtype and arguments as la_forward;
 * no alignment requirement).  The heads are processed in groups (a run of
 * heads of one batch entry each, about eight groups): a group's inputs are
 * copied up on a copy stream the library owns, its forward runs on `stream`
 * once they have landed, and its output is copied down on a second copy
 * stream once the forward is done, so that uploads, kernels and downloads of
 * different groups overlap.  Host buffers should be page-locked
 * (cudaHostAlloc / cudaHostRegister): pageable memory is correct but its
 * copies do not overlap.  Device memory for the whole problem is a
 * stream-ordered allocation on `stream` from a pool the library keeps per
 * device, which holds released memory for the next call until the process
 * exits (the two copy streams are kept likewise).  Asynchronous: o is complete once
 * `stream` has been synchronised; the host buffers must stay valid until
 * then.  The result equals la_forward's up to the order of summation (each
 * group splits its sequences for its own size).  Errors as la_forward.
 * Defined on the same pages as la_forward.
 */
LA_API la_status_t la_forward_host(const void *q, const void *k, const void *v, void *o,
                                   int B, int H, int N, int D, int Dv, int causal,
                                   const float *gamma, float eps, la_dtype_t dtype,
                                   void *stream);

/*
 * State after a causal pass over N tokens (the prefill of the decode loop):
 *   S = sum_j gamma^(N-1-j) phi(k_j) v_j^T,  z = sum_j gamma^(N-1-j) phi(k_j)
 * k: [B][H][N][D]; v: [B][H][N][Dv] (dtype); S: [B][H][D][Dv] fp32 and
 * z: [B][H][D] fp32 are overwritten.  S and z must not overlap k or v, nor
 * each other.
 * Defined on the pages "Linear Attention Mechanisms" (dileepadev.github.io),
 * "Recurrent Reformulation" (S_i and z_i of the causal recurrence at
 * i = N - 1, the state the recurrent form carries into inference) and
 * "Gating and Selective State Updates" (the decay weight gamma^(N-1-j)).
 */
LA_API la_status_t la_prefill_state(const void *k, const void *v, float *S, float *z,
                             int B, int H, int N, int D, int Dv,
                             const float *gamma, la_dtype_t dtype,
                             void *stream);

/*
 * Causal forward that also returns the state after the last token: o as
 * la_forward(..., causal = 1, ...), and S, z as la_prefill_state over the
 * same k, v (the state the decode loop continues from).  On the tensor-core
 * path for D = Dv = 128 the state comes out of the forward's own pass (the
 * CTA of the last part writes it); otherwise the library runs the forward,
 * then the prefill reduction, on `stream`.
 * q, k: [B][H][N][D]; v, o: [B][H][N][Dv] (dtype); S: [B][H][D][Dv] fp32 and
 * z: [B][H][D] fp32 are overwritten (zero for N = 0).  No written buffer (o,
 * S, z) may overlap any other buffer; the read-only inputs may share memory.
 * Errors as la_forward and la_prefill_state.
 * Defined on the pages "Linear Attention Mechanisms" (dileepadev.github.io),
 * "Recurrent Reformulation" (the state S_i, z_i at i = N - 1) and "Gating
 * and Selective State Updates" (the decay on both).
 */
LA_API la_status_t la_forward_state(const void *q, const void *k, const void *v, void *o,
                                    float *S, float *z, int B, int H, int N, int D, int Dv,
                                    const float *gamma, float eps, la_dtype_t dtype,
                                    void *stream);

/*
 * One recurrent decode step, in place: first
 *   S <- gamma S + phi(k) v^T,  z <- gamma z + phi(k),
 * then  o = phi(q)^T S / (phi(q) . z + eps)  with the updated state.
 * q, k: [B][H][D]; v, o: [B][H][Dv] (dtype); S: [B][H][D][Dv] fp32 and
 * z: [B][H][D] fp32 are read and rewritten.  No written buffer (S, z, o) may
 * overlap any other buffer; q, k and v may share memory.
 * Defined on the pages "Linear Attention Mechanisms" (dileepadev.github.io),
 * "Recurrent Reformulation" (one iteration of the recurrence: update with
 * k, v, then read out with q) and "Practical Tradeoffs" (a fixed-size state
 * per step at inference), with the decay of "Gating and Selective State
 * Updates" on both S and z.
 */
LA_API la_status_t la_decode_step(const void *q, const void *k, const void *v,
                           float *S, float *z, void *o, int B, int H, int D,
                           int Dv, const float *gamma, float eps,
                           la_dtype_t dtype, void *stream);

/*
 * Gated causal forward (gated linear attention): per token t
 *   S_t = diag(a_t) S_{t-1} + phi(k_t) v_t^T,  z_t = a_t (.) z_{t-1} + phi(k_t),
 *   o_t = phi(q_t)^T S_t / (phi(q_t) . z_t + eps),   S_{-1} = 0, z_{-1} = 0,
 * i.e. the data-dependent gate G_t of "Linear Attention Mechanisms"
 * (dileepadev.github.io), "Gating and Selective State Updates", taken as one
 * value per key feature and token, G_t = a_t 1^T (row d of S is scaled by
 * a_t[d]), and applied to the normaliser z as well.  a_t = 1 everywhere is
 * la_forward(causal = 1, gamma = NULL); a_t = gamma[h] everywhere is the
 * fixed decay; a_t[d] = 0 clears row d of the state before token t's update.
 * q, k: [B][H][N][D]; v, o: [B][H][N][Dv] (dtype); a: [B][H][N][D] fp32 in
 * DEVICE memory, every value in [0, 1] (the library cannot check device
 * values: outside [0, 1] the result is unspecified, a NaN gate gives NaN
 * outputs).  S: [B][H][D][Dv] fp32 and z: [B][H][D] fp32 are both NULL or
 * both set; when set they receive the state after the last token (zero for
 * N = 0).  fp32 arithmetic on CUDA cores, or for bf16 with D = Dv = 128
 * and B*H >= 8 the tensor-core form described at la_gated_kernel
 * (bf16 operands, fp32 accumulation and state).  A workspace of about
 * B*H*(P-1)*(D*Dv + 2D)*4 bytes (P <= ceil(N/64) parts), plus for the
 * tensor-core form 2*B*H*N*D*2 + B*H*ceil(N/128)*D*4 bytes, is taken with
 * cudaMallocAsync on `stream` and released on it.  No written
 * buffer may overlap another buffer.  Errors as la_forward.
 */
LA_API la_status_t la_forward_gated(const void *q, const void *k, const void *v,
                                    const float *a, void *o, float *S, float *z, int B,
                                    int H, int N, int D, int Dv, float eps,
                                    la_dtype_t dtype, void *stream);

/*
 * Which form la_forward_gated runs for these arguments: 1 = tensor cores
 * (bf16, D = Dv = 128, B*H >= 8, with or without the final state, which
 * want_state no longer changes: q and k scaled per
 * 128-token chunk by gate suffix products, then the 128-token causal kernel
 * with its state rescaled by each chunk's gate products; a call whose gates
 * forget harder than 2^-93 within some chunk and feature falls back at run
 * time to the CUDA-core form, which a device flag selects), 0 = the fp32
 * CUDA-core form, or a negative la_status_t (negated) for invalid sizes.
 * Host-only.
 */
LA_API int la_gated_kernel(int B, int H, int N, int D, int Dv, la_dtype_t dtype, int want_state);

/*
 * One gated decode step, in place: first
 *   S <- diag(a) S + phi(k) v^T,  z <- a (.) z + phi(k),
 * then  o = phi(q)^T S / (phi(q) . z + eps)  with the updated state (the
 * recurrence of la_forward_gated for one token).  q, k: [B][H][D]; v, o:
 * [B][H][Dv] (dtype); a: [B][H][D] fp32 gates in [0, 1] (device); S:
 * [B][H][D][Dv] fp32 and z: [B][H][D] fp32 are read and rewritten.  No
 * written buffer (S, z, o) may overlap any other buffer.  Errors as
 * la_decode_step.
 */
LA_API la_status_t la_decode_gated(const void *q, const void *k, const void *v,
                                   const float *a, float *S, float *z, void *o, int B,
                                   int H, int D, int Dv, float eps, la_dtype_t dtype,
                                   void *stream);

/*
 * Performer random-feature map: for every row x of x [rows][D],
 *   phi(x) = r^(-1/2) [exp(w_1 . x - |x|^2/2), ..., exp(w_r . x - |x|^2/2)]
 * with the directions w_j the rows of W [r][D] (drawn by the caller: iid
 * N(0, 1), or block-orthogonal rows for positive orthogonal random features).
 * "Linear Attention Mechanisms" (dileepadev.github.io), "Choosing the Feature
 * Map": Random Fourier Features (Performer) and FAVOR+.  The -|x|^2/2 term is
 * the reading under which that passage's E[phi(q) . phi(k)] = exp(q . k)
 * holds for w ~ N(0, I).
 * x, W and phi [rows][r] (written) are DEVICE arrays of `dtype`; D and r in
 * {64, 128}.  LA_BF16 runs a tcgen05 GEMM with the exponential in its
 * epilogue (exact bf16 products, fp32 sums, phi rounded to bf16); LA_F32 runs
 * in fp32 on CUDA cores.  exp overflows fp32 where w_j . x - |x|^2/2 > 88.
 * phi may not overlap x or W.
 */
LA_API la_status_t la_favor_features(const void *x, const void *W, void *phi, int rows, int D,
                                     int r, la_dtype_t dtype, void *stream);

/*
 * Performer attention: la_favor_features on q and on k, then linear
 * attention over those r-dimensional features, o_i = phi(q_i)^T S_i /
 * (phi(q_i)^T z_i + eps), causal (S_i, z_i over j <= i, decayed by
 * gamma[h]^(i-j)) or non-causal (every j; gamma must be NULL or all 1).  The
 * attention runs on the same kernels as la_forward with the features in place
 * of phi(q), phi(k) (tensor cores for LA_BF16).  q, k: [B][H][N][D]; v, o:
 * [B][H][N][Dv]; W: [r][D]; all of `dtype`; D, Dv and r in {64, 128}.  The
 * features take a stream-ordered workspace of 2*B*H*N*r elements of `dtype`
 * (cudaMallocAsync on `stream`), plus the attention kernel's own.  o may not
 * overlap q, k, v or W.  Errors as la_forward.
 */
LA_API la_status_t la_forward_favor(const void *q, const void *k, const void *v, const void *W,
                                    void *o, int B, int H, int N, int D, int Dv, int r,
                                    int causal, const float *gamma, float eps,
                                    la_dtype_t dtype, void *stream);

/*
 * Backward pass of the causal form (with the per-head decay): given the
 * upstream gradient dO = dL/do of o = la_forward(q, k, v, causal = 1, gamma,
 * eps), writes dq = dL/dq, dk = dL/dk, dv = dL/dv.  With
 * w_ij = gamma^(i-j) phi(q_i).phi(k_j) (j <= i), d_i = sum_j w_ij + eps,
 * gt_i = dO_i / d_i and c_i = gt_i . o_i, the chain rule through
 * o_i = sum_j w_ij v_j / d_i gives dL/dw_ij = gt_i . v_j - c_i, and
 *   dv_j = sum_(i>=j) w_ij gt_i,
 *   dq_i = phi'(q_i) * sum_(j<=i) gamma^(i-j) (dL/dw_ij) phi(k_j),
 *   dk_j = phi'(k_j) * sum_(i>=j) gamma^(i-j) (dL/dw_ij) phi(q_i),
 * phi'(x) = 1 for x > 0, exp(x) otherwise.  The "parallel training" half
 * of the duality on "Linear Attention Mechanisms" (dileepadev.github.io),
 * "Recurrent Reformulation"; the forward it differentiates is la_forward's.
 * The library recomputes o and d itself (the caller keeps no forward
 * state).  q, k, dq, dk: [B][H][N][D]; v, dO, dv: [B][H][N][Dv]; all of
 * `dtype`.  For LA_BF16 with Dv = 64 and every gamma >= 0.35 the sums run on
 * tcgen05 tensor cores (la_backward_kernel = 1): the forward's undivided
 * numerators and normalisers, then three decayed causal products with bf16
 * operands and fp32 accumulation (dq forward, dk and dv over token-reversed
 * operands), in a stream-ordered workspace of about B*H*N*(8 D + 1412)
 * bytes.  Otherwise fp32 arithmetic on CUDA cores in a stream-ordered
 * workspace of B*H*N*(4D + 6Dv + 16)*4 bytes plus the per-part states of the
 * sequence split.  Workspaces are taken with cudaMallocAsync on `stream`.
 * No gradient may overlap an input or another gradient.  Errors as
 * la_forward.
 */
LA_API la_status_t la_backward(const void *q, const void *k, const void *v, const void *dO,
                               void *dq, void *dk, void *dv, int B, int H, int N, int D,
                               int Dv, const float *gamma, float eps, la_dtype_t dtype,
                               void *stream);

/*
 * Which kernels la_backward runs for these arguments: 1 = tcgen05 tensor
 * cores (bf16, Dv = 64, D in {64, 128}, every gamma >= 0.35), 0 = fp32 CUDA
 * cores, or a negative la_status_t (negated) for invalid arguments.  gamma
 * as in la_backward (host array or NULL).  Host-only apart from reading the
 * current device's SM count.
 */
LA_API int la_backward_kernel(int B, int H, int N, int D, int Dv, const float *gamma,
                              la_dtype_t dtype);

/*
 * Number of kernels one la_backward call with these arguments launches (on
 * CUDA cores it depends on how the sequence is split across the current
 * device's SMs), 0 for an empty call, or a negative la_status_t (negated)
 * for invalid arguments.  Host-only apart from reading the current device's
 * SM count.
 */
LA_API int la_backward_launches(int B, int H, int N, int D, int Dv, const float *gamma,
                                la_dtype_t dtype);

/*
 * Which kernel la_forward would run for a causal call with these arguments:
 * 2 = the tcgen05 tensor-core kernel with 128-token chunks (bf16,
 * D = Dv = 128, every gamma >= 0.61), 1 = the tcgen05 tensor-core kernel with
 * 64-token chunks (bf16, D and Dv in {64, 128}, every gamma >= 0.35),
 * 0 = the fp32 CUDA-core kernel (fp32 inputs, or stronger decays, whose
 * gamma^-63 operand scale would leave the bf16 range), or a negative
 * la_status_t (negated) if the arguments are invalid.
 * Host-only; touches no device.
 */
LA_API int la_causal_kernel(int B, int H, int N, int D, int Dv,
                            const float *gamma, la_dtype_t dtype);

/*
 * Number of bounded device-side waits that gave up on the current device since
 * the library was loaded (or since the last reset).  The tensor-core kernels
 * bound every wait on another warp's progress; a nonzero count means some
 * kernel abandoned its work and the outputs of that call are invalid.  Reads
 * device memory with a blocking copy, so call it after synchronising the
 * streams that ran the kernels.  reset != 0 sets the counter back to zero.
 * Returns -1 if the counter cannot be read.
 */
LA_API int la_device_wait_timeouts(int reset);

/*
 * Diagnostic of the failure path above, without a fault: runs the kernels'
 * own bounded mbarrier wait, with a limit of `cycles` SM clock cycles (1 to
 * 4e9; about 0.5 ms per 1e6 cycles at 2 GHz), on a barrier that nothing
 * arrives on.  The wait gives up, adds one to the counter that
 * la_device_wait_timeouts reads, and *gave_up (host) becomes 1; the context
 * stays usable.  Launches one warp on the legacy default stream of the
 * current device and synchronises the device.  LA_ERR_INVALID_ARG for a
 * null gave_up or cycles out of range.
 */
LA_API la_status_t la_wait_selftest(long long cycles, int *gave_up);

/*
 * Non-causal forward without any device allocation.  No counterpart on the
 * pages: it computes exactly what la_forward(..., causal = 0, gamma = NULL,
 * ...) computes, but keeps its scratch (per-head S, z and the partial sums of
 * the split reduction) in a fixed array inside the library instead of taking
 * a workspace with cudaMallocAsync.  For callers that cannot let a library
 * allocate: applications that reserve device memory up front in their own
 * allocator and forbid third-party allocations, and latency-critical loops
 * where an allocation could stall or fail on a full memory pool.
 *   - The scratch is la_forward_noncausal_static_limit() bytes (32 MiB) on
 *     every GPU that loads the library, held until the process exits.  Calls
 *     whose per-head state alone, B*H*(D*Dv + D)*4 bytes, exceeds it return
 *     LA_ERR_UNSUPPORTED; below that the reduction uses as many sequence
 *     splits as fit.
 *   - The first call on each device queries the device address of the
 *     scratch (one runtime call, with that device current); make that first
 *     call before any stream capture.
 *   - Every call on a device shares the one scratch array.  Calls whose work
 *     overlaps on the GPU (for example on two streams with no ordering
 *     between them) race on it and corrupt each other's results: order them.
 *     Each call writes every scratch word before reading it, so nothing needs
 *     clearing between calls.
 * Arguments, layouts and errors otherwise as la_forward (gamma is implicitly
 * 1; D, Dv in {64, 128}).
 */
LA_API la_status_t la_forward_noncausal_static(const void *q, const void *k, const void *v,
                                               void *o, int B, int H, int N, int D, int Dv,
                                               float eps, la_dtype_t dtype, void *stream);

/* Size in bytes of the per-device scratch used by la_forward_noncausal_static. */
LA_API size_t la_forward_noncausal_static_limit(void);

/*
 * Selective state space scan and the operators around its block.  "Linear
 * Attention Mechanisms" (dileepadev.github.io) sets the state space form
 * h_t = A_t h_(t-1) + B_t x_t beside the gated recurrence of "Gating and
 * Selective State Updates"; here A_t and B_t are chosen per token through a
 * step dt_t.  Conventions of this family, besides those at the top:
 * - Token-major tensors: x, dt, z, y [B][L][E], B_t and C_t [B][L][G][N] (each
 *   group of E / G consecutive channels shares one), of `dtype`; for a single
 *   token [B][E] and [B][G][N].  Parameters (A [E][N], D, dt_bias, w, bias) and
 *   scan states [B][E][N] are fp32.
 * - ldx, lddt, ldz, ldb, ldc: elements between consecutive tokens of that
 *   input (the batch stride is L times it), so that slices of a projection's
 *   output are read in place; 0 means dense rows.  A stride is a multiple of 8
 *   and at least the row's width; outputs are dense.
 * - Sizes: E a multiple of 8 up to 65536, E / G a multiple of 8, N in {8, 16,
 *   32, 64}, B L < 2^31 - 2^16 tokens and B E < 2^31.
 * - lens (optional, int32 [B] in DEVICE memory, 4-byte aligned): sequence b
 *   has lens[b] tokens (clamped to [0, L]).  Rows behind it have no
 *   effect and are left alone in the outputs, and the final state is the one after the last token.
 * - fp32 arithmetic; each output is rounded once to `dtype`.  Results do not
 *   depend on scheduling (no atomics).  Workspaces are stream-ordered
 *   allocations from a pool the library keeps per device (up to 512 MiB held
 *   between calls).
 * - No written buffer may overlap any other buffer of the call (strided inputs
 *   count from their first to their last element).
 */

/*
 * Selective scan of whole sequences: per channel e and state n
 *   dt_t = softplus(dt_t + dt_bias)   (softplus = 0: the plain sum)
 *   h_t  = exp(dt_t A) h_(t-1) + dt_t x_t B_t,      h_(-1) = h0 (NULL: zeros)
 *   y_t  = (sum_n C_t h_t + D x_t) silu(z_t)
 * D, z and dt_bias may be NULL (no such term).  States are meant to decay
 * (dt_t A <= 0; any rate down to -inf): the tokens are worked in parts, and
 * where exp(A sum dt) over a part leaves the fp32 range a result may be inf or
 * NaN although its own token-by-token terms are finite.  hN (optional) receives the
 * state after the last token (h0 for no tokens), the state
 * la_decode_selective continues from; it may not be h0 itself.  Few channels
 * split the tokens into up to 128 parts of 32 tokens or more, with a workspace of
 * B*E*(N + 1)*4 bytes for each part but one (each part of a ragged batch, whose
 * parts are laid out over its sequences by their lengths).
 */
LA_API la_status_t la_forward_selective(const void *x, const void *dt, const float *A,
                                        const void *Bm, const void *Cm, const float *D,
                                        const void *z, const float *dt_bias, const float *h0,
                                        const int *lens, void *y, float *hN, int B, int L, int E,
                                        int N, int G, long long ldx, long long lddt, long long ldz,
                                        long long ldb, long long ldc, int softplus,
                                        la_dtype_t dtype, void *stream);

/*
 * One token of the scan, in place on the state h [B][E][N] fp32: x, dt, z, y
 * [B][E], Bm, Cm [B][G][N].  y must not be any input.
 */
LA_API la_status_t la_decode_selective(const void *x, const void *dt, const float *A,
                                       const void *Bm, const void *Cm, const float *D,
                                       const void *z, const float *dt_bias, float *h, void *y,
                                       int B, int E, int N, int G, long long ldx, long long lddt,
                                       long long ldz, long long ldb, long long ldc, int softplus,
                                       la_dtype_t dtype, void *stream);

/*
 * Gradients of la_forward_selective (every sequence of L tokens) for the
 * upstream gradients dy of y and, optionally, dhN of the final state.  With
 * gy_t = dy_t silu(z_t) and the adjoint state g_t = C_t gy_t + exp(dt_(t+1) A)
 * g_(t+1) (dhN behind the last token):
 *   dC_t = sum_e h_t gy_t,  dB_t = sum_e g_t dt_t x_t    (over a group)
 *   du_t = sum_n g_t B_t,   w_t = g_t exp(dt_t A) h_(t-1)
 *   dx_t = du_t dt_t + D gy_t
 *   ddt_t = (sum_n w_t A + du_t x_t) softplus'(.),  ddt_bias = sum_t ddt_t
 *   dA = sum_t w_t dt_t,  dD = sum_t gy_t x_t,  dz_t = dy_t (y_t before the gate) silu'(z_t)
 *   dh0 = exp(dt_0 A) g_0.
 * States are recomputed (the caller keeps no forward state).  dx, ddt, dz
 * [B][L][E] and dBm, dCm [B][L][G][N] are dense, of `dtype`; dA, dD, ddt_bias
 * and dh0 fp32.  dD, ddt_bias and dh0 may be NULL and need their input; dz is
 * given exactly when z is.  A batch padded at the end is given zero rows of dy
 * and finite values in the padding of the other inputs (a later token does not
 * reach an earlier one, but zero times NaN is NaN); with dhN also steps of zero
 * there (raw dt -inf under softplus), which carry the state to the end.  The
 * workspace is about B*L*E*(9N/64 + N*N/512) floats (11 bytes per token and
 * channel for N = 16): per part of 64 tokens (32 or 48 for N = 8) seven states
 * within it, one in front and one adjoint behind, and the channel tiles' sums
 * of dB and dC.
 */
LA_API la_status_t la_backward_selective(
    const void *x, const void *dt, const float *A, const void *Bm, const void *Cm, const float *D,
    const void *z, const float *dt_bias, const float *h0, const void *dy, const float *dhN,
    void *dx, void *ddt, float *dA, void *dBm, void *dCm, float *dD, void *dz, float *ddt_bias,
    float *dh0, int B, int L, int E, int N, int G, long long ldx, long long lddt, long long ldz,
    long long ldb, long long ldc, int softplus, la_dtype_t dtype, void *stream);

/*
 * Short causal depthwise convolution (ahead of the scan):
 *   y_t[e] = act(bias[e] + sum_(k < W) w[e][k] x_(t - W + 1 + k)[e]),
 * act = SiLU when silu is nonzero, W in 2..4.  The W - 1 rows before the first
 * token come from state [B][W-1][E] (`dtype`, oldest first; NULL: zeros).
 * state_out (optional, not `state` itself) receives the last W - 1 rows, the
 * state la_decode_conv continues from.  w [E][W], bias [E] (optional) fp32.
 */
LA_API la_status_t la_forward_conv(const void *x, const float *w, const float *bias,
                                   const void *state, const int *lens, void *y, void *state_out,
                                   int B, int L, int E, int W, long long ldx, int silu,
                                   la_dtype_t dtype, void *stream);

/* One token of the convolution, in place on state [B][W-1][E]: x, y [B][E]. */
LA_API la_status_t la_decode_conv(const void *x, const float *w, const float *bias, void *state,
                                  void *y, int B, int E, int W, long long ldx, int silu,
                                  la_dtype_t dtype, void *stream);

/*
 * Gradients of la_forward_conv (every sequence of L tokens) for the upstream
 * gradient dy: dx [B][L][E] and dstate [B][W-1][E] (optional, needs state) of
 * `dtype`, dw [E][W] and dbias [E] (optional, needs bias) fp32.  A gradient of
 * state_out is one of x's last rows (or of state's): the caller adds it there.
 * A batch padded at the end is given zero rows of dy and finite rows of x there.
 */
LA_API la_status_t la_backward_conv(const void *x, const float *w, const float *bias,
                                    const void *state, const void *dy, void *dx, float *dw,
                                    float *dbias, void *dstate, int B, int L, int E, int W,
                                    long long ldx, int silu, la_dtype_t dtype, void *stream);

/*
 * RMS norm of a mixing form's output per head, with its gate:
 *   gate_first = 0:  o = y rsqrt(mean y^2 + eps) w silu(gate)
 *   gate_first = 1:  o = p rsqrt(mean p^2 + eps) w,   p = y silu(gate)
 * over rows of D values, one per (b, h, token).  y is [B][H][L][D]
 * (heads_first, as la_forward and la_forward_gated write o) or [B][L][H][D];
 * gate and out are token-major [B][L][H*D], as the projections before and
 * behind it hold them; all of `dtype`.  w [H][D] fp32 (NULL: ones).  D a
 * multiple of 8 up to 8192, H*D up to 65536, fewer than 2^31 rows; eps finite
 * and >= 0.  All tensors are dense; out may not overlap an input.  The sum of
 * squares is fp32: a row for which it overflows (values beyond 2^64 / sqrt(D))
 * gives zeros.
 */
LA_API la_status_t la_forward_norm_gate(const void *y, const void *gate, const float *w, void *out,
                                        int B, int H, int L, int D, int heads_first,
                                        int gate_first, float eps, la_dtype_t dtype, void *stream);

/*
 * Gradients of la_forward_norm_gate for the upstream gradient dout [B][L][H*D]:
 * dy (laid out as y), dgate [B][L][H*D] of `dtype` and dw [H][D] fp32
 * (optional, needs w).
 */
LA_API la_status_t la_backward_norm_gate(const void *y, const void *gate, const float *w,
                                         const void *dout, void *dy, void *dgate, float *dw, int B,
                                         int H, int L, int D, int heads_first, int gate_first,
                                         float eps, la_dtype_t dtype, void *stream);

/*
 * Scaled residual sum and the RMS norm ahead of the next block, over rows of E
 * values of `dtype`:
 *   r = residual + scale x  (residual NULL: scale x),  o = r rsqrt(mean r^2 + eps) w.
 * The norm takes the fp32 sum r (and an fp32 sum of squares, as above); r is
 * also written, rounded.  w [E] fp32 (NULL: ones).  E a multiple of 8 up to
 * 8192, fewer than 2^31 rows.  o and r may not overlap an input or each other.
 */
LA_API la_status_t la_forward_norm_residual(const void *x, const void *residual, const float *w,
                                            void *o, void *r, long long rows, int E, float scale,
                                            float eps, la_dtype_t dtype, void *stream);

/*
 * Gradients of la_forward_norm_residual at the written r, for the upstream
 * gradients dout of o and dr of r (NULL: none): dresidual = dr + the norm's
 * gradient, dx = scale dresidual (NULL when scale is 1, where the two are
 * equal), dw [E] fp32 (optional, needs w).
 */
LA_API la_status_t la_backward_norm_residual(const void *r, const float *w, const void *dout,
                                             const void *dr, void *dresidual, void *dx, float *dw,
                                             long long rows, int E, float scale, float eps,
                                             la_dtype_t dtype, void *stream);

/*
 * Retention: linear attention with one decay per head, q and k as they are (no
 * feature map) and no normaliser (the retention of "Gating and Selective State
 * Updates" and "Evolution: add decay/gating": RetNet, gamma^(t-j)):
 *
 *   S_t = gamma S_(t-1) + k_t v_t^T,   o_t = scale q_t^T S_t,   S_(-1) = S0.
 *
 * Conventions of this family, besides those at the top:
 * - q [B][L][H][D], k [B][L][Hk][D], v [B][L][Hk][Dv], o [B][L][H][Dv] of
 *   `dtype`; Hk divides H, and H / Hk consecutive heads of q share one of k and
 *   v.  Each (b, h) has its own state [D][Dv], fp32, caller-owned.
 * - strides (HOST array of 12, or NULL for dense tensors as above): elements
 *   between batches, tokens and heads of q, k, v and o (la_backward_retention:
 *   dO), so that slices of a projection's output and tensors laid out heads
 *   first are read in place.  Multiples of 8, rows contiguous and apart from
 *   one another; the stride of a dimension of size 1 is not looked at.
 * - Sizes: D and Dv multiples of 8 up to 256, H <= 256, B L < 2^31 - 2^16
 *   tokens, B H < 2^26.  |scale| between 2^-64 and 2^64.
 * - lens (optional, int32 [B] in DEVICE memory, 4-byte aligned): sequence b has
 *   lens[b] tokens (clamped to [0, L]).  Rows behind it have no effect; outputs there are left alone, gradients there are zero; the final
 *   state is the one after the last token.
 * - Arithmetic: fp32 states and sums, each output rounded once.  For LA_BF16
 *   with Dv a multiple of 32 and D at most 64, 128, at most 192 or 256 (gradients:
 *   with D and Dv in each other's place too) the products run on tcgen05 tensor
 *   cores: there the weights of a chunk and the decayed rows that build the states
 *   for outputs are rounded to bf16 once, and states enter as sums of two bf16
 *   values.  Returned states (S, dS0) are summed from decayed
 *   rows as three bf16 values, to fp32 accuracy.  Results do not depend on
 *   scheduling (no atomics).
 * - Within a chunk of up to 128 tokens a weight of zero times an infinity or NaN
 *   of a later token is NaN: inputs are finite.
 * - Few (batch, head) pairs split long sequences into parts that run side by
 *   side, with a workspace of B*H*D*Dv*4 bytes for each part but the last
 *   (gradients: three times that); where a state is returned from the tensor cores,
 *   once more for the last part.  More than 128 features are worked as 128 and
 *   the rest, with a workspace of 2*B*L*H*Dv*4 bytes for the two shares of o.
 *   Workspaces as in the selective scan's family; no written buffer may overlap
 *   any other buffer of the call.
 */

/*
 * Whole sequences: o and, unless S is NULL, the state after the last token,
 * which la_decode_retention continues from.  S0 [B][H][D][Dv] fp32 (NULL:
 * zeros) may not be S itself.
 */
LA_API la_status_t la_forward_retention(const void *q, const void *k, const void *v, const float *S0,
                                        const int *lens, void *o, float *S, int B, int L, int H,
                                        int Hk, int D, int Dv, const long long *strides,
                                        const float *gamma, float scale, la_dtype_t dtype,
                                        void *stream);

/*
 * One token of each of B sequences, in place on states S [pool][H][D][Dv]:
 * sequence b has state slots[b] (int32 [B] in DEVICE memory; NULL: state b,
 * pool >= B).  A slot outside [0, pool) marks an idle row of a padded batch:
 * nothing of it is read or written, its row of o is left alone.  No slot may
 * occur twice.  q, o [B][H][*], k, v [B][Hk][*]; ldq, ldk, ldv: elements between
 * consecutive sequences' rows, 0 for dense (as in the selective scan's family).
 */
LA_API la_status_t la_decode_retention(const void *q, const void *k, const void *v, float *S,
                                       const int *slots, void *o, int B, int pool, int H, int Hk,
                                       int D, int Dv, long long ldq, long long ldk, long long ldv,
                                       const float *gamma, float scale, la_dtype_t dtype,
                                       void *stream);

/*
 * Gradients of la_forward_retention for the upstream gradients dO of o and,
 * unless NULL, dS [B][H][D][Dv] fp32 of the final state.  With
 * U_t = dL/dS_t = gamma U_(t+1) + scale q_t dO_t^T (gamma U behind the last
 * token: dS):
 *   dq_t = scale S_t dO_t,  dk_t = U_t v_t,  dv_t = U_t^T k_t,  dS0 = gamma U_0,
 * dk and dv summed over the heads that share them.  dq, dk, dv are dense, of
 * `dtype`; dS0 fp32 (NULL: not wanted; needs S0).  Nothing of the forward pass
 * is kept: the states are computed again.  Shared heads take a workspace of
 * B*L*H*(D + Dv)*4 bytes for dk and dv before they are added; Dv above 128 takes
 * room for two shares of dq and dk, D above 128 of dv.
 */
LA_API la_status_t la_backward_retention(const void *q, const void *k, const void *v,
                                         const void *dO, const float *S0, const float *dS,
                                         const int *lens, void *dq, void *dk, void *dv, float *dS0,
                                         int B, int L, int H, int Hk, int D, int Dv,
                                         const long long *strides, const float *gamma, float scale,
                                         la_dtype_t dtype, void *stream);

/*
 * Beam search between two decode steps.  For each of B requests the n best of
 * its K beams' continuations: beam k with token v scores
 *   scores[b][k] + logits[b][k][v] - log sum_u exp(logits[b][k][u]).
 * out_scores fp32, parents and tokens int32, all [B][n], best first; equal
 * scores (as computed: rows of the same logits have the same sums wherever they
 * lie; rows that hold them in another order, or all moved by a constant, may differ
 * by the roundings of their sums) in the order of k, then v.  finished (optional, bytes [B][K]): a beam
 * that has ended, whose one continuation is `eos` at its own score.  A beam
 * whose score or log-sum is not finite (a start's unused beams at -inf, a row
 * with a NaN or +inf) offers nothing, nor does a logit of -inf (a forbidden
 * token); places beyond the last continuation get score -inf, parent and token
 * -1.  logits of `dtype` with ld elements between rows (0: V), scores fp32;
 * no alignment beyond the elements' own.  K <= 32, n <= 64, V <= 2^30.  Scores
 * are compared in 64 bits, sums of exponentials are fp32 within pieces of at
 * most 8192 logits and 64-bit over them.  Workspace: 8 n + 8 bytes a piece.
 */
LA_API la_status_t la_select_beams(const void *logits, const float *scores,
                                   const unsigned char *finished, float *out_scores, int *parents,
                                   int *tokens, int B, int K, int V, int n, long long ld, int eos,
                                   la_dtype_t dtype, void *stream);

/*
 * The beams' states after a selection: for each of `count` buffers, states[i]
 * [B][K] records of bytes[i] bytes (HOST arrays of device pointers and sizes;
 * the states of la_decode_retention, la_decode_step, la_decode_selective and
 * la_decode_conv, tokens so far), record k of request b is replaced in place by
 * record parents[b][k].  A parent outside [0, K) keeps the beam's own.  No two
 * buffers may overlap.  K <= 32.  Buffers of 16-byte records on 16-byte
 * boundaries move fastest.
 */
LA_API la_status_t la_reorder_states(void *const *states, const long long *bytes, int count,
                                     const int *parents, int B, int K, void *stream);

/* Static, NUL-terminated description of a status code. */
LA_API const char *la_status_string(la_status_t s);

#ifdef __cplusplus
}
#endif
#endif /* LINATTN_H */
