// Host-side launchers of the library's kernels (internal to the library).
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace linattn {

constexpr int kMaxHeads = 256;
constexpr int kSMs = 152;  // of a GB300, for the rules that size grids

// A runtime call that fails stays the thread's last error, where the check
// behind a later launch would find it: whatever turns an error into a status
// takes it away.
inline void forget_error() { (void)cudaGetLastError(); }

// Per-head decay values, passed to kernels by value.
struct Gammas {
  float g[kMaxHeads];
};

enum Dtype { kF32 = 0, kBF16 = 1 };

struct Problem {
  const void *q, *k, *v;
  void *o;
  int B, H, N, D, Dv;
  bool decay;  // any gamma != 1
  float eps;
  Dtype dtype;
  // q, k already are features (the Performer path computes them first): the
  // kernels use them as they are instead of applying phi = elu + 1
  bool ident = false;
};

// First chunk of part p when nch chunks split into P equal parts (the
// 128-token kernel's split; the gated form's gate tables follow it).
__host__ __device__ inline int chunk_part_begin(int p, int P, int nch) {
  if (p <= 0) return 0;
  if (p >= P) return nch;
  const int base = nch / P, rem = nch % P;
  return p * base + (p < rem ? p : rem);
}

// Causal forward on CUDA cores (fp32 FFMA): any dtype.
cudaError_t launch_causal_simt(const Problem &p, const Gammas &g,
                               cudaStream_t s);

// Sequence-parallel chunked kernels on tcgen05 tensor cores (bf16 operands,
// fp32 state).  chunk_tc_supported() gives the envelope (bf16, D and Dv in
// {64, 128}, every decay >= 0.35); chunk_parts() the number of parts per
// (batch, head); chunk_workspace_bytes() the fp32 per-part records for that
// many parts (prefill, non-causal) and chunk_causal_workspace_bytes() the
// causal launcher's workspace (flags and inclusive states; 0 for one part).
bool chunk_tc_supported(const Problem &p, const Gammas &g);
int chunk_parts(int BH, int N);        // causal
int chunk_state_parts(int BH, int N, int D, int Dv);  // prefill, non-causal
size_t chunk_workspace_bytes(int BH, int P, int D, int Dv);
size_t chunk_causal_workspace_bytes(int BH, int P, int D, int Dv);
Gammas log2_gammas(const Gammas &g, int H, bool decay);
cudaError_t launch_causal_chunk(const Problem &p, const Gammas &g, void *ws, int P,
                                cudaStream_t s);
// The causal chunk kernel with another epilogue in place of o = numerators /
// (normaliser + eps) (p.o unused): out_raw [B*H][N][Dv] and den_raw [B*H][N]
// fp32, the undivided numerators and normalisers; or grad_out [B*H][N][Dv]
// bf16, the numerators times phi'(grad_in) elementwise (factor 1 when
// grad_in is null), at row N - 1 - t for rev (a product over token-reversed
// operands stored back in token order).
struct ChunkEpilogue {
  float *out_raw, *den_raw;
  __nv_bfloat16 *grad_out;
  const __nv_bfloat16 *grad_in;
  int rev;
};
// Non-causal forward on tensor cores with persistent streaming kernels
// (noncausal_tc.cu): bf16, D and Dv in {64, 128}, no decay.  A reduce pass
// writes per-part [S | z] records (noncausal_tc_workspace_bytes()), a scan
// sums them, an apply pass writes o.
bool noncausal_tc_supported(const Problem &p);
size_t noncausal_tc_workspace_bytes(const Problem &p);
cudaError_t launch_noncausal_tc(const Problem &p, void *ws, cudaStream_t s);
cudaError_t launch_causal_chunk_epilogue(const Problem &p, const Gammas &g, void *ws, int P,
                                         cudaStream_t s, const ChunkEpilogue &ep);
// The causal kernel with 128-token chunks for D = Dv = 128 (chunk128.cu):
// bf16, every decay >= 0.61; workspace (flags and inclusive states) for P
// parts, 0 for one part.
bool chunk128_supported(const Problem &p, const Gammas &g);
int chunk128_parts(int BH, int N);
size_t chunk128_workspace_bytes(int BH, int P);
// S_out, z_out (optional, both or neither): the state after the last token,
// [B*H][D][Dv] and [B*H][D] fp32.
cudaError_t launch_causal_chunk128(const Problem &p, const Gammas &g, void *ws, int P,
                                   cudaStream_t s, float *S_out = nullptr,
                                   float *z_out = nullptr);
// Final state S [BH][D][Dv], z [BH][D] of the causal recurrence over N tokens.
cudaError_t launch_prefill_chunk(const void *k, const void *v, float *S, float *z, int B, int H,
                                 int N, int D, int Dv, bool decay, const Gammas &g, void *ws,
                                 int P, cudaStream_t s);

// Scan over per-part records [BH][P][D*Dv + D] (part_scan.cu): kScanStarts
// turns A_p into the state before part p in place; kScanFinal writes the
// state after all parts to S_out, z_out; kScanSum writes sum_p A_p to slot 0.
enum ScanMode { kScanStarts = 0, kScanFinal = 1, kScanSum = 2 };
cudaError_t launch_part_scan(float *rec, int BH, int H, int P, int N, int D, int Dv,
                             const Gammas &lg, int mode, float *S_out, float *z_out,
                             cudaStream_t s);

// Split-N reduction of S = sum_j w_j phi(k_j) v_j^T and z = sum_j w_j
// phi(k_j) with w_j = gamma^(N-1-j): partials [nsplit][BH][D*Dv + D] in
// `partials` (fp32) unless nsplit == 1, in which case S, z are written
// directly.  Then a fixed-order reduction into S [BH][D][Dv], z [BH][D].
int kv_state_num_splits(int BH, int N);
size_t kv_state_workspace_bytes(int BH, int N, int D, int Dv);
// ident: k already holds features (no phi).
cudaError_t launch_kv_state(const void *k, const void *v, float *S, float *z,
                            float *partials, int B, int H, int N, int D,
                            int Dv, bool decay, const Gammas &g, Dtype dt,
                            cudaStream_t s, bool ident = false);

// The same reduction (no decay) with a caller-chosen number of splits
// (partials [nsplit][BH][D*Dv + D] in `partials` when nsplit > 1).
cudaError_t launch_kv_state_splits(const void *k, const void *v, float *S, float *z,
                                   float *partials, int B, int H, int N, int D, int Dv,
                                   int nsplit, const Gammas &g, Dtype dt, cudaStream_t s);

// o = phi(q) S / (phi(q) . z + eps) for every row, S and z per (b, h).
cudaError_t launch_noncausal_apply(const void *q, const float *S,
                                   const float *z, void *o, int BH, int N,
                                   int D, int Dv, float eps, Dtype dt,
                                   cudaStream_t s, bool ident = false);

// One decode step in place on S, z.
cudaError_t launch_decode_step(const void *q, const void *k, const void *v,
                               float *S, float *z, void *o, int B, int H,
                               int D, int Dv, bool decay, const Gammas &g,
                               float eps, Dtype dt, cudaStream_t s);

// One gated decode step in place on S, z: row d of S and z[d] scaled by
// a[(b, h)][d] (fp32 gates in [0, 1]) before the update.
cudaError_t launch_decode_gated(const void *q, const void *k, const void *v, const float *a,
                                float *S, float *z, void *o, int B, int H, int D, int Dv,
                                float eps, Dtype dt, cudaStream_t s);

// Gated causal forward on CUDA cores (gla_simt.cu): gates a [B*H][N][D] fp32
// in [0, 1], one per key feature and token.  gla_parts() gives the number of
// sequence parts, gla_workspace_bytes() the per-part records (0 for one
// part).  S_out, z_out (optional, both or neither): the state after the last
// token, [B*H][D][Dv] and [B*H][D] fp32.
int gla_parts(int BH, int N, int Dv);
size_t gla_workspace_bytes(int BH, int P, int D, int Dv);
// only_if (optional): the kernels do nothing unless *only_if is nonzero
cudaError_t launch_gla_simt(const Problem &p, const float *a, void *ws, int P, float *S_out,
                            float *z_out, cudaStream_t s, const int *only_if = nullptr);
// The gated tensor-core form (bf16, D = Dv = 128, B*H >= 8; S_out, z_out
// optional, the state after the last token):
// a prep kernel scales q, k per 128-token chunk by gate suffix products,
// then the 128-token causal kernel runs with one part per (batch, head) and
// rescales its state by each chunk's gate products.  *hard_out receives a
// device flag that is nonzero when some chunk forgets too hard for this form
// (the causal kernel then does nothing and the caller runs the CUDA-core
// form with only_if = the flag).
bool gla_tc_supported(const Problem &p);
size_t gla_tc_workspace_bytes(int BH, int N);
cudaError_t launch_gla_tc(const Problem &p, const float *a, void *ws, cudaStream_t s,
                          const int **hard_out, float *S_out = nullptr, float *z_out = nullptr);
// gate_suf / gate_part: see gla_tc (P > 1); ws: chunk128_workspace_bytes(BH, P)
cudaError_t launch_gated_chunk128(const Problem &p, const float *gate_prod, const float *gate_suf,
                                  const float *gate_part, const int *skip, void *ws, int P,
                                  cudaStream_t s, float *S_out = nullptr, float *z_out = nullptr);

// Performer random-feature map (favor.cu): fq = phi(q), fk = phi(k) for
// `rows` rows of q and k [rows][D], directions W [R][D], outputs [rows][R],
// all of dtype dt; phi(x) = R^(-1/2) exp(W x - |x|^2 / 2).  D, R in {64, 128}.
// k = nullptr: q only (fk unused).
cudaError_t launch_favor_features(const void *q, const void *k, const void *W, void *fq,
                                  void *fk, long long rows, int D, int R, Dtype dt,
                                  cudaStream_t s);

// Backward of the causal form (backward_simt.cu): dq, dk, dv (dtype of p)
// from q, k, v of p and the upstream gradient dO [B*H][N][Dv]; fp32 on CUDA
// cores in a workspace of backward_workspace_bytes().
size_t backward_workspace_bytes(int BH, int N, int D, int Dv);
int backward_launches(int BH, int N, int D, int Dv);  // kernels one call launches
cudaError_t launch_backward(const Problem &p, const void *dO, void *dq, void *dk, void *dv,
                            const Gammas &g, void *ws, cudaStream_t s);
// The same on tensor cores (backward_tc.cu) for bf16, Dv = 64, D in {64,
// 128} and the 64-token chunk kernel's decay envelope: the forward's
// undivided n and d, a prep kernel, three gradient products.
bool backward_tc_supported(const Problem &p, const Gammas &g);
size_t backward_tc_workspace_bytes(int BH, int N, int D);
int backward_tc_launches();
cudaError_t launch_backward_tc(const Problem &p, const void *dO, void *dq, void *dk, void *dv,
                               const Gammas &g, void *ws, cudaStream_t s);

// out0[c] (c < C0) and out1[c - C0] (the rest; may be null) = sum of rec[r][c]
// over the n records of C columns, in a fixed order (column_sum.cu).  To be
// launched right behind the kernel that writes the records.
cudaError_t launch_column_sum(const float *rec, int n, int64_t C, float *out0, int64_t C0,
                              float *out1, cudaStream_t s);

// Selective state space scan (selective.cu, selective_bwd.cu).  x, dt, z, y
// and the gradients: [B][L][E] (one step: [B][E]); Bm, Cm [B][L][G][N]; x,
// dt, z, Bm, Cm with ld elements between tokens; parameters and states fp32:
// A [E][N], D, dt_bias [E], h0, hN [B][E][N].  z, D, dt_bias, lens (int32
// [B]), h0, hN may be null.  For a step hN is updated in place.
struct ScanArgs {
  const void *x, *dt, *z, *Bm, *Cm;
  const float *A, *D, *dt_bias, *h0;
  const int *lens;
  void *y;
  float *hN;
  int B, L, E, N, G;
  int64_t ldx, lddt, ldz, ldb, ldc;
  bool softplus;
};
bool selective_states_supported(int N);
// Sequence parts of the scan (of a ragged batch: on average over its
// sequences), tokens per part where they are not, and the workspace of the
// parts' records (0 for one part).
int selective_parts(int B, int L, int E, int N, int G, Dtype dt, bool ragged);
int selective_part_len(int L, int S);
size_t selective_workspace_bytes(int B, int E, int N, int S, bool ragged);
cudaError_t launch_selective(const ScanArgs &a, Dtype dt, void *ws, int S, cudaStream_t s);
cudaError_t launch_selective_step(const ScanArgs &a, Dtype dt, cudaStream_t s);
// Records of the scan's parts (S of them; the forward pass keeps S - 1), fp32:
// end states from zero h [B][S][E][N] and sums of dt [B][S][E]; for the
// backward pass also each part's adjoint contribution to the state before it
// g [B][S][E][N], and every kScanCheckpoint tokens (not at the part's start)
// the state ck [B][S][K][E][N] and the sum of dt so far ckdt [B][S][K][E],
// K = part_len / kScanCheckpoint - 1.
constexpr int kScanCheckpoint = 8;
struct ScanRecords {
  float *h, *dt, *g, *ck, *ckdt;
};
cudaError_t launch_selective_local(const ScanArgs &a, const void *dy, const ScanRecords &rec, int S,
                                   int part_len, Dtype dt, cudaStream_t s);
// Backward of the scan from h0 (null: zeros): gradients of every input from
// dy and, when dhN is set, the upstream gradient of the final state.  dD,
// dz, ddt_bias, dh0 are null where their input is.
struct ScanGrads {
  const void *dy;
  const float *dhN;
  void *dx, *ddt, *dz, *dBm, *dCm;
  float *dA, *dD, *ddt_bias, *dh0;
};
size_t selective_backward_workspace_bytes(int B, int L, int E, int N, int G);
cudaError_t launch_selective_backward(const ScanArgs &a, const ScanGrads &g, Dtype dt, void *ws,
                                      cudaStream_t s);

// Short causal depthwise convolution (short_conv.cu): x, y [B][L][E] (x with
// ldx elements between tokens), w [E][W] and bias [E] fp32, W in 2..4, state
// [B][W-1][E] (the rows before the first token; null: zeros).
struct ConvArgs {
  const void *x;
  const float *w, *bias;
  const void *state;
  const int *lens;
  void *y, *state_out;
  int B, L, E, W;
  int64_t ldx;
  bool silu;
};
cudaError_t launch_conv(const ConvArgs &a, Dtype dt, cudaStream_t s);
// One token, in place on state_out (a.state and a.lens unused).
cudaError_t launch_conv_step(const ConvArgs &a, Dtype dt, cudaStream_t s);
// dx [B][L][E], dw [E][W], dbias [E] (optional), dstate [B][W-1][E] (optional).
struct ConvGrads {
  const void *dy;
  void *dx, *dstate;
  float *dw, *dbias;
};
size_t conv_backward_workspace_bytes(int B, int L, int E, int W, Dtype dt);
cudaError_t launch_conv_backward(const ConvArgs &a, const ConvGrads &g, Dtype dt, void *ws,
                                 cudaStream_t s);

// RMS norms around a block (norms.cu).  Gated: rows of D values, one per
// (b, t, h); y [B][H][L][D] (heads_first) or [B][L][H][D], gate and out
// [B][L][H*D], w [H][D] fp32 or null.
struct NormGateArgs {
  const void *y, *gate;
  const float *w;
  void *out;
  int B, H, L, D;
  float eps;
  bool heads_first, gate_first;
};
struct NormGateGrads {
  const void *dout;
  void *dy, *dgate;
  float *dw;  // null when w is
};
cudaError_t launch_norm_gate(const NormGateArgs &a, Dtype dt, cudaStream_t s);
size_t norm_gate_backward_workspace_bytes(int B, int H, int L, int D);
cudaError_t launch_norm_gate_backward(const NormGateArgs &a, const NormGateGrads &g, Dtype dt,
                                      void *ws, cudaStream_t s);
// Residual: r = residual + scale x, o = norm(r) w; rows of E values.
struct NormResidualArgs {
  const void *x, *residual;  // residual null: r = scale x
  const float *w;            // [E] or null
  void *o, *r;               // backward: r is an input, o unused
  int64_t rows;
  int E;
  float scale, eps;
};
struct NormResidualGrads {
  const void *dout, *dr;     // dr null: no other gradient of r
  void *dresidual, *dx;      // dx null when scale is 1
  float *dw;                 // null when w is
};
cudaError_t launch_norm_residual(const NormResidualArgs &a, Dtype dt, cudaStream_t s);
size_t norm_residual_backward_workspace_bytes(int64_t rows, int E);
cudaError_t launch_norm_residual_backward(const NormResidualArgs &a, const NormResidualGrads &g,
                                          Dtype dt, void *ws, cudaStream_t s);

// Retention (retention.cuh): one product of rows x over the state that rows y
// and w build, forward or backward in time.  Strides in elements between
// batches, tokens and heads; head h of the call reads head h / xg of x (and so
// on).  start, end: states [B][H][Dx][Dw] fp32 (start with its own row and
// column strides, so that it may be stored transposed), each with a factor.
// o_f32: o is fp32 whatever the inputs' type.
struct RetStrides {
  int64_t b, t, h;
};
struct RetRole {
  const void *x, *y, *w;
  void *o;
  RetStrides xs, ys, ws, os;
  int xg, yg, wg, Dx, Dw;
  const float *start;
  float *end, *rec;  // rec: [B][H][records][Dx][Dw]
  int start_rs, start_cs;
  int64_t state;  // elements between the states of start and end (Dx Dw, or more for a role of some features)
  float start_scale, end_scale, out_scale;
  int reverse, o_f32;
  int records;  // one for each part but the last; on tensor cores one more where there is an end
};
constexpr int kRetRoles = 6;
struct RetArgs {
  RetRole role[kRetRoles];
  int roles;
  const int *lens;
  int B, L, H;
  bool fill;  // rows behind a sequence's end become zero (otherwise they are left)
  Gammas lg;  // log2 of each head's decay
};
// Parts of the tokens that run side by side; the size in floats of the records of all
// roles; the kernels take a.role[].rec and records as laid out by ret_layout.
int ret_parts(const RetArgs &a, Dtype dt);
size_t ret_record_floats(const RetArgs &a, Dtype dt, int parts);
void ret_layout(RetArgs *a, Dtype dt, int parts, float *ws);
cudaError_t launch_retention(const RetArgs &a, Dtype dt, int parts, cudaStream_t s);
bool ret_tc_supported(const RetArgs &a, Dtype dt);
cudaError_t launch_retention_simt(const RetArgs &a, Dtype dt, int parts, cudaStream_t s);
cudaError_t launch_retention_tc(const RetArgs &a, int parts, cudaStream_t s);
int ret_parts_simt(const RetArgs &a);
int ret_parts_tc(const RetArgs &a);
// out[b][t][h][e] = sum over the g shares of part[b][t][h g + i][e]; out with
// strides of its own, rows behind lens left alone (lens null: none).
struct GroupSumArgs {
  const float *part;
  void *out;
  RetStrides os;
  const int *lens;
  int B, L, heads, g, width;
};
cudaError_t launch_group_sums(const GroupSumArgs *a, int n, Dtype dt, cudaStream_t s);  // n <= 3, one launch

// One token of retention in place on states [slots][H][D][Dv] fp32: sequence b
// has the state slots[b] (null: b); one outside [0, pool) is passed over.
struct RetStepArgs {
  const void *q, *k, *v;
  float *S;
  const int *slots;
  void *o;
  int B, H, Hk, D, Dv, pool;
  int64_t ldq, ldk, ldv;
  float scale;
  Gammas g;
};
cudaError_t launch_retention_step(const RetStepArgs &a, Dtype dt, cudaStream_t s);

// Beam search (beams.cu): the n best of score[b][k] + log softmax(logits[b][k]).
struct BeamArgs {
  const void *logits;
  const float *scores;
  const uint8_t *finished;  // or null
  float *out_scores;
  int *parents, *tokens;
  int B, K, V, n, eos;
  int64_t ld;  // elements between rows of logits
};
size_t beams_workspace_bytes(int B, int K, int V, int n);
cudaError_t launch_select_beams(const BeamArgs &a, Dtype dt, void *ws, cudaStream_t s);
// states[i]: [B][K][bytes[i]], each beam's bytes replaced in place by its parent's.
constexpr int kReorderStates = 64;  // of one launch
cudaError_t launch_reorder_states(void *const *states, const int64_t *bytes, int count, const int *parents, int B,
                                  int K, cudaStream_t s);

}  // namespace linattn
