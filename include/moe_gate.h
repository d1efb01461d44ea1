/*
 * moe_gate.h -- C ABI of the single-GPU top-k Mixture-of-Experts layer hot path
 * (gate -> capacity/locations -> encode -> expert FFN -> decode, plus the
 * backward of encode and decode), built for NVIDIA GB300 (sm_103a).
 *
 * Sources restated (web pages, cited by title and section):
 *   [Tutel]  "Tutel" project profile: key-configuration table (MOELayer
 *            gate_type {'type': 'top', 'k', 'capacity_factor'}, experts
 *            {'type': 'ffn', hidden_size_per_expert, has_fc1_bias,
 *            has_fc2_bias}) and the FAQ on capacity_factor.
 *   [Blog]   "MoE training systems: DeepSpeed-MoE vs Tutel", section 1.4
 *            (dense token-to-expert mapping table; fused top-k + cumsum +
 *            scatter; data-layout transform instead of einsum) and section 3.5
 *            (fast encode/decode kernels K0, K1, K2; dynamic capacity factor).
 *   [PR8195] DeepSpeed PR #8195 (follow-up to #8174): change 1 (per-route
 *            int32 index/location/gate, capacity resolved once without a
 *            device-to-host sync), change 2 (the [e, c, m] vs flat [e*c, m]
 *            buffer hazard), change 3 (index dispatch, fp32 combine).
 *
 * Conventions shared by every call:
 *   - Every pointer argument is caller-owned memory.  Device pointers must be
 *     16-byte aligned.  Tensors are dense row-major with the shapes given.
 *     Outputs overlap neither the inputs nor each other.
 *   - No call allocates, frees or synchronises.  Work is enqueued on `stream`
 *     (a cudaStream_t passed as void*; NULL = the legacy default stream).
 *   - Routing tables are route-major [k, s]: entry (r, t) is at r*s + t.
 *     Route r of token t is its r-th best expert.
 *   - Expert buffers are physically [e, c_max, m] (row stride c_max*m per
 *     expert).  The logical [e, c, m] view is rows 0..c-1 of each expert.
 *     c_max is fixed by the caller; the data-dependent c lives in device
 *     memory (`c_dev`) and is never read back by the library.
 *   - A route is kept iff loc < c.  Dropped routes keep their un-clipped loc.
 *   - dev_status: caller-owned device int32, zeroed by the caller.  A kernel
 *     that detects a data-dependent error (c > c_max, an index out of range,
 *     a bounded wait that gave up) stores the first error code there.  Every
 *     kernel reads it on entry and does nothing if it is non-zero.  The caller
 *     reads it after its own synchronisation.
 *   - Host-side validation is synchronous: a bad shape, NULL or misaligned
 *     pointer returns MOE_ERR_INVALID_ARG and nothing is launched.  A launch
 *     failure returns MOE_ERR_CUDA.
 *   - Shapes: s >= 1, 1 <= k <= min(e, 32), 1 <= e <= 1024, m, h >= 1.
 *     Rows must be 16-byte multiples: m and h multiples of 8 (bf16) or 4 (fp32).
 */
#ifndef MOE_GATE_H
#define MOE_GATE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = 1,  /* bad shape / pointer (host) or bad index (device) */
    MOE_ERR_UNSUPPORTED = 2,  /* valid but not implemented combination */
    MOE_ERR_CUDA = 3,         /* a CUDA runtime/driver call failed */
    MOE_ERR_CAPACITY = 4,     /* device: capacity c exceeds c_max */
    MOE_ERR_TIMEOUT = 5       /* device: a bounded wait gave up */
} moe_status;

typedef enum { MOE_F32 = 0, MOE_BF16 = 1 } moe_dtype;

typedef enum {
    MOE_ACT_RELU = 0,   /* y = relu(x W1^T + b1) W2^T + b2 */
    MOE_ACT_GELU = 1,   /* y = gelu_erf(x W1^T + b1) W2^T + b2 */
    MOE_ACT_SWIGLU = 2  /* y = (silu(x W1^T) * (x W3^T)) W2^T, no biases */
} moe_act;

typedef enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 } moe_score;

/* Microscaled 4-bit formats: e2m1 codes (0, .5, 1, 1.5, 2, 3, 4, 6, signed). */
typedef enum {
    MOE_FP4_MX = 0,  /* blocks of 32 along the row, one e8m0 (power of two) scale each */
    MOE_FP4_NV = 1   /* blocks of 16, one e4m3 scale each, one fp32 factor per batch */
} moe_fp4;

#define MOE_FLAG_NORMALIZE_GATES 1u /* divide the k selected gates by their sum */
#define MOE_FLAG_ZERO_FILL 2u       /* zero the unoccupied rows 0..c-1 of each expert */

/*
 * Gate ([Tutel] gate_type 'top'; [Blog] 1.4 fused top-k).
 *   logits[t, j] = fp32 dot(x[t, :], wg[:, j]) + bias[j], fused multiply-adds
 *   (one rounding each) in a fixed order, then one fp32 add of the bias:
 *     e <= 32: the features are cut into chunks of one 16-byte load (8 bf16 or
 *       4 fp32 elements); chunk c goes to lane c mod 32; each of the 32 lanes
 *       accumulates its features from +0 in ascending index; the lane sums are
 *       combined by an xor butterfly (o = 16, 8, 4, 2, 1: v[l] + v[l xor o]),
 *       and the logit is lane 0's value.
 *     e > 32: one accumulator from +0 in ascending feature index.
 *   This fixed order makes idx reproducible bit for bit.
 *   idx[r, t]: expert at position r when experts are ordered by (logit
 *   descending, index ascending).  gates[r, t]: softmax probability of that
 *   expert over all e logits; with MOE_FLAG_NORMALIZE_GATES divided by the sum
 *   of the k selected probabilities.
 * x [s, m] in `xdt`; wg [m, e] fp32; bias [e] fp32 or NULL.
 * idx [k, s] int32 and gates [k, s] fp32 are written.  e <= 256 here.
 */
moe_status moe_gate_topk(const void *x, moe_dtype xdt, const float *wg, const float *bias,
                         int64_t s, int m, int e, int k, unsigned flags,
                         int32_t *idx, float *gates, int32_t *dev_status, void *stream);

/*
 * Capacity bound on the host ([Tutel] FAQ capacity_factor; [Blog] 3.5).
 *   f > 0: exactly c = ceil(f*k*s/e)  (evaluated exactly on the float value f);
 *   f = 0: s  (the largest c the no-drop rule can produce);
 *   f < 0: min(ceil(-f*k*s/e), s).
 * A c_max at least this large never triggers MOE_ERR_CAPACITY.
 */
int64_t moe_capacity_bound(float capacity_factor, int64_t s, int e, int k);

/* Bytes of device workspace moe_capacity_locations needs. */
size_t moe_capacity_workspace_size(int64_t s, int e, int k);

/*
 * Capacity and slot locations ([Blog] 1.4 cumsum; [Blog] 3.5 dynamic capacity).
 *   counts[j] = number of routes that chose expert j (before any drop).
 *   c = ceil(f*k*s/e) for f > 0; max_j counts[j] for f = 0;
 *       min(ceil(-f*k*s/e), max_j counts[j]) for f < 0.   Written to c_dev[0].
 *   loc[r, t] = number of routes ahead of (r, t) in route-priority order
 *   (all tokens' route 0 in token order, then route 1, ...) that chose the
 *   same expert.  Kept iff loc < c.
 *   c > c_max stores MOE_ERR_CAPACITY in dev_status (loc/counts still valid).
 * idx [k, s] int32 in; loc [k, s] int32, counts [e] int32, c_dev [1] int32 out.
 * workspace: device memory of moe_capacity_workspace_size() bytes, contents
 * ignored on entry (scratch).
 */
moe_status moe_capacity_locations(const int32_t *idx, int64_t s, int e, int k,
                                  float capacity_factor, int64_t c_max,
                                  void *workspace, size_t workspace_bytes,
                                  int32_t *loc, int32_t *counts, int32_t *c_dev,
                                  int32_t *dev_status, void *stream);

/*
 * moe_capacity_locations without a workspace argument: the same results from
 * the same kernels, with their scratch in a fixed array inside the library.
 * The pages have no counterpart; this entry point exists for callers that
 * cannot allocate device memory themselves -- for example a plugin running
 * inside an inference engine that owns the device's whole memory pool, or a
 * latency-critical path where cudaMalloc's implicit device synchronisation is
 * not acceptable.  It calls no cudaMalloc, cudaFree or other allocating routine.
 *   - Scratch limit: MOE_CAPACITY_NOALLOC_SCRATCH_BYTES (1 MiB), held
 *     on every GPU that loads the library until the process exits.  Shapes
 *     whose moe_capacity_workspace_size() exceeds it return
 *     MOE_ERR_UNSUPPORTED with nothing launched.
 *   - The first call on a device looks up the array's device address (with
 *     that device current) and keeps it for that device's CUDA context; after
 *     cudaDeviceReset the next call looks it up again.  Make the first call on
 *     each device (and the first after a reset) before any stream capture.
 *   - All calls share the one array: calls that overlap on the GPU (different
 *     streams without ordering between them) race and give wrong locations.
 *     Calls ordered on one stream are safe; nothing needs clearing in between.
 */
moe_status moe_capacity_locations_noalloc(const int32_t *idx, int64_t s, int e, int k,
                                          float capacity_factor, int64_t c_max, int32_t *loc,
                                          int32_t *counts, int32_t *c_dev, int32_t *dev_status,
                                          void *stream);

/* Bytes of the fixed scratch array moe_capacity_locations_noalloc uses. */
#define MOE_CAPACITY_NOALLOC_SCRATCH_BYTES (1u << 20)

/*
 * Fast encode ([Blog] 3.5, kernel K1 forward; [PR8195] change 3).
 *   buf[idx[r,t], loc[r,t], :] = x[t, :] for every kept route (unweighted copy).
 *   With MOE_FLAG_ZERO_FILL, rows min(counts[j], c)..c-1 of every expert j are
 *   set to zero as well (counts required then, else it may be NULL).  Other
 *   rows of buf are left untouched.
 * x [s, m]; buf [e, c_max, m], both in `dt`.
 */
moe_status moe_encode(const void *x, moe_dtype dt, const int32_t *idx, const int32_t *loc,
                      const int32_t *counts, const int32_t *c_dev, int64_t s, int m, int e,
                      int k, int64_t c_max, unsigned flags, void *buf, int32_t *dev_status,
                      void *stream);

/* Bytes of device workspace moe_expert_ffn needs (the hidden activations). */
size_t moe_expert_ffn_workspace_size(moe_dtype dt, moe_act act, int e, int64_t c_max, int m,
                                     int h);

/*
 * Per-expert FFN ([Tutel] experts 'ffn'; [Blog] 3.5 batched expert matmul over
 * (E, C, D)).  For every expert j and row i < min(counts[j], c):
 *   hid = act(buf[j,i,:] W1[j]^T + b1[j])        (ReLU / GELU, exact erf form)
 *   hid = silu(buf[j,i,:] W1[j]^T) * (buf[j,i,:] W3[j]^T)      (SwiGLU)
 *   out[j,i,:] = hid W2[j]^T + b2[j]
 * Accumulation in fp32; the hidden activation is rounded to `dt` before the
 * second product; each output is rounded once to `dt`.  Rows >= the kept
 * count are not written.
 * buf, out [e, c_max, m]; w1, w3 [e, h, m]; w2 [e, m, h]; b1 [e, h]; b2 [e, m];
 * all in `dt`.  b1/b2 may be NULL (no bias); w3 only for SwiGLU, which takes
 * no biases.  workspace: moe_expert_ffn_workspace_size() bytes, scratch.
 * bf16 runs on the tensor cores (tcgen05, fp32 accumulation in TMEM); fp32
 * runs on the SIMT cores with fp32 fused multiply-add.
 */
moe_status moe_expert_ffn(const void *buf, moe_dtype dt, const int32_t *counts,
                          const int32_t *c_dev, const void *w1, const void *b1, const void *w3,
                          const void *w2, const void *b2, moe_act act, int e, int64_t c_max,
                          int m, int h, void *workspace, size_t workspace_bytes, void *out,
                          int32_t *dev_status, void *stream);

/*
 * moe_expert_ffn for training (bf16): the same outputs, and fc1 also stores
 * what moe_expert_ffn_bwd_saved needs instead of recomputing it, for the kept
 * rows (other rows not written), rounded once to bf16 from the fp32 sums:
 *   ReLU / GELU: the pre-activation buf W1^T + b1, pre [e, c_max, h];
 *   SwiGLU:      a = buf W1^T and b = buf W3^T, pre [e, c_max, 2h] (a, then b).
 * Errors: as moe_expert_ffn; MOE_ERR_INVALID_ARG for a NULL or misaligned
 * pre; MOE_ERR_UNSUPPORTED for fp32.
 */
moe_status moe_expert_ffn_train(const void *buf, moe_dtype dt, const int32_t *counts,
                                const int32_t *c_dev, const void *w1, const void *b1,
                                const void *w3, const void *w2, const void *b2, moe_act act, int e,
                                int64_t c_max, int m, int h, void *workspace,
                                size_t workspace_bytes, void *out, void *pre, int32_t *dev_status,
                                void *stream);

/*
 * Fast decode ([Blog] 3.5, K0 forward; [PR8195] change 3, fp32 combine).
 *   y[t, :] = sum over kept routes r of gates[r,t] * out[idx[r,t], loc[r,t], :],
 *   accumulated in fp32 with fused multiply-add in ascending r from +0 and
 *   rounded once to `dt`.  Tokens with every route dropped get 0.
 * out [e, c_max, m], y [s, m] in `dt`; gates [k, s] fp32.
 */
moe_status moe_decode(const void *out, moe_dtype dt, const int32_t *idx, const int32_t *loc,
                      const float *gates, const int32_t *c_dev, int64_t s, int m, int e, int k,
                      int64_t c_max, void *y, int32_t *dev_status, void *stream);

/*
 * Backward of decode ([Blog] 3.5: K1 is combine's backward, K2 the cross term).
 *   d_out[idx, loc, :] = gates[r,t] * dy[t, :]  (exact product rounded once)
 *   d_gates[r, t] = sum_i dy[t,i] * out[idx, loc, i]  (fp32), 0 if dropped.
 *   With MOE_FLAG_ZERO_FILL (counts required) unoccupied rows < c of d_out
 *   are zeroed; otherwise they are left untouched.
 * dy [s, m], out and d_out [e, c_max, m] in `dt`; gates, d_gates [k, s] fp32.
 */
moe_status moe_decode_bwd(const void *dy, const void *out, moe_dtype dt, const int32_t *idx,
                          const int32_t *loc, const float *gates, const int32_t *counts,
                          const int32_t *c_dev, int64_t s, int m, int e, int k, int64_t c_max,
                          unsigned flags, void *d_out, float *d_gates, int32_t *dev_status,
                          void *stream);

/*
 * Backward of encode ([Blog] 3.5: K0 with unit weights).
 *   dx[t, :] = sum over kept routes of d_buf[idx, loc, :], fp32 accumulation
 *   in ascending r from +0, rounded once to `dt`.  All-dropped tokens get 0.
 * d_buf [e, c_max, m], dx [s, m] in `dt`.
 */
moe_status moe_encode_bwd(const void *d_buf, moe_dtype dt, const int32_t *idx,
                          const int32_t *loc, const int32_t *c_dev, int64_t s, int m, int e,
                          int k, int64_t c_max, void *dx, int32_t *dev_status, void *stream);

/* Bytes of device workspace moe_expert_ffn_bwd needs (0 if unsupported). */
size_t moe_expert_ffn_bwd_workspace_size(moe_dtype dt, moe_act act, int e, int64_t c_max, int m,
                                         int h);

/*
 * Per-expert FFN backward (the gradient of moe_expert_ffn; the pages give
 * only the forward experts 'ffn' of [Tutel]).  For L = sum over kept rows of
 * <d_out, out>, with every kept row i < min(counts[j], c) of expert j:
 *   pre = buf W1^T + b1 (recomputed), d_hid = d_out W2,
 *   d_pre = d_hid * act'(pre)   (SwiGLU: d_a = d_hid * b * silu'(a),
 *                                d_b = d_hid * silu(a), a = buf W1^T, b = buf W3^T),
 *   d_buf = d_pre W1 (+ d_b W3), d_w2 = d_out^T hid, d_b2 = sum d_out,
 *   d_w1 = d_pre^T buf (d_a for SwiGLU), d_w3 = d_b^T buf, d_b1 = sum d_pre.
 * Inputs: buf [e, c_max, m] and hid [e, c_max, h] as moe_expert_ffn read and
 * wrote them (hid is its workspace after the call); w1, w3 [e, h, m];
 * w2 [e, m, h]; b1 [e, h] or NULL; d_out [e, c_max, m]; counts, c_dev as for
 * the forward.  Outputs in `dt`: d_buf [e, c_max, m] (rows past the kept
 * count not written), d_w1, d_w3 [e, h, m], d_w2 [e, m, h], d_b1 [e, h],
 * d_b2 [e, m].  d_w3 is SwiGLU's only, which takes no biases; d_b1 / d_b2 may
 * be NULL.  workspace: moe_expert_ffn_bwd_workspace_size() bytes, scratch.
 * bf16 only (MOE_ERR_UNSUPPORTED for fp32): every product is the forward's
 * tensor-core grouped GEMM (fp32 accumulation in TMEM); d_hid and d_pre (and
 * SwiGLU's recomputed a and b) are rounded to bf16 between the products, the
 * ReLU / GELU pre-activation is recomputed in fp32 inside the product that
 * forms d_pre.
 */
moe_status moe_expert_ffn_bwd(const void *buf, const void *hid, moe_dtype dt,
                              const int32_t *counts, const int32_t *c_dev, const void *w1,
                              const void *b1, const void *w3, const void *w2, moe_act act, int e,
                              int64_t c_max, int m, int h, const void *d_out, void *workspace,
                              size_t workspace_bytes, void *d_buf, void *d_w1, void *d_w3,
                              void *d_w2, void *d_b1, void *d_b2, int32_t *dev_status,
                              void *stream);

/*
 * moe_expert_ffn_bwd with what moe_expert_ffn_train kept (pre): d_pre is
 * formed in the epilogue of the product d_out W2, so d_hid is neither rounded
 * nor stored and nothing is recomputed:
 *   ReLU / GELU: d_pre = (d_out W2) * act'(pre), pre [e, c_max, h];
 *   SwiGLU:      [d_a | d_b] = (d_out W2) * [b silu'(a) | silu(a)],
 *                pre = [a | b] [e, c_max, 2h].
 * The other outputs as moe_expert_ffn_bwd (w3 and d_w3 for SwiGLU only, NULL
 * otherwise; d_b1 / d_b2 for ReLU / GELU only, or NULL).  d_w1, d_w3, d_w2,
 * d_b1, d_b2 in `wgrad_dt`: MOE_BF16, or MOE_F32 for gradients kept in fp32
 * (the products' fp32 sums stored unrounded, as an optimiser with fp32 master
 * weights wants them); d_buf in `dt`.  workspace:
 * moe_expert_ffn_bwd_workspace_size() bytes.  Errors: as moe_expert_ffn_bwd;
 * MOE_ERR_INVALID_ARG for a NULL or misaligned pre or another wgrad_dt.
 */
moe_status moe_expert_ffn_bwd_saved(const void *buf, const void *hid, const void *pre,
                                    moe_dtype dt, const int32_t *counts, const int32_t *c_dev,
                                    const void *w1, const void *w3, const void *w2, moe_act act,
                                    int e, int64_t c_max, int m, int h, const void *d_out,
                                    void *workspace, size_t workspace_bytes, void *d_buf,
                                    moe_dtype wgrad_dt, void *d_w1, void *d_w3, void *d_w2,
                                    void *d_b1, void *d_b2, int32_t *dev_status, void *stream);

/*
 * Gate backward ([Tutel] gate_type 'top': the gates are softmax probabilities
 * of the k selected experts, renormalised over them with
 * MOE_FLAG_NORMALIZE_GATES).  Top-k selection is piecewise constant, so the
 * gradient flows through the softmax only.  With A = sum_r dg[r,t] g[r,t]:
 *   renormalised:  d_logits[t, idx[r,t]] = g (dg - A), other experts 0;
 *   raw softmax:   d_logits[t, j] = -p_j A + sum over routes r to j of dg g,
 *                  p = softmax of the logits (recomputed here from x, wg, bias);
 *   d_wg = x^T d_logits [m, e],  d_bias = sum over t of d_logits [e],
 *   d_x = d_logits wg^T [s, m].
 * Inputs: x [s, m] in `xdt`; wg [m, e] fp32; bias [e] fp32 or NULL (used only
 * to recompute the logits of the raw softmax); idx, gates [k, s] as the gate
 * wrote them; d_gates [k, s] fp32 (e.g. moe_decode_bwd's).  Outputs, all fp32
 * and deterministic: d_logits [s, e] (required), d_wg [m, e], d_bias [e],
 * d_x [s, m] (each may be NULL).  Fixed summation orders: A sums the routes in
 * route order; d_wg and d_bias sum each of 64 contiguous token slices in token
 * order, then the slices in order; d_x sums, per token, the experts in order
 * (raw softmax) or its k routes in route order (renormalised gates, where the
 * other experts' d_logits are zero).  e <= 256 here.
 * This entry point extends the pages' forward gate to its backward.
 */
moe_status moe_gate_bwd(const void *x, moe_dtype xdt, const float *wg, const float *bias,
                        int64_t s, int m, int e, int k, unsigned flags, const int32_t *idx,
                        const float *gates, const float *d_gates, float *d_logits, float *d_wg,
                        float *d_bias, float *d_x, int32_t *dev_status, void *stream);

/*
 * Low-precision experts ([Tutel] profile, notes and highlights: FP8 among its
 * inference formats, "blockwise FP8" without a block size).  Here an operand
 * is e4m3 (OCP FP8 E4M3: 4 exponent bits, bias 7, 3 mantissa bits, largest
 * finite 448) with one fp32 scale per row, so the scales apply once, after
 * the contraction:
 *   q[r, i] = e4m3(x[r, i] / scale[r]),  scale[r] = amax_i |x[r, i]| / 448
 * (fp32 divisions, nearest-even, saturating at +-448; scale 1 for a zero row).
 *
 * moe_quantize_rows_fp8: src [batches, rows_per_batch, cols] bf16 -> q (same
 * shape, one byte per code) and scale [batches, rows_per_batch] fp32.  With
 * counts [batches] and c_dev (both or neither), only the rows r <
 * min(counts[b], *c_dev, rows_per_batch) of batch b are written (the kept
 * rows of an expert buffer); else every row (e.g. weights [e, rows, cols]).
 * cols a multiple of 16.  Deterministic; the codes match an exact-arithmetic
 * reference bit for bit.  This entry point extends the pages' expert FFN to
 * the FP8 format.
 */
moe_status moe_quantize_rows_fp8(const void *src, int64_t batches, int64_t rows_per_batch,
                                 int cols, const int32_t *counts, const int32_t *c_dev, void *q,
                                 float *scale, int32_t *dev_status, void *stream);

/* Bytes of device workspace moe_expert_ffn_fp8 needs (0: bad shape). */
size_t moe_expert_ffn_fp8_workspace_size(int e, int64_t c_max, int m, int h);

/*
 * The expert FFN (ReLU / GELU) on e4m3 operands: buf_q [e, c_max, m] with
 * buf_scale [e, c_max] (moe_quantize_rows_fp8 of the encoded buffer's kept
 * rows), w1_q [e, h, m] with w1_scale [e, h], w2_q [e, m, h] with w2_scale
 * [e, m] (weights quantised per output channel), b1 [e, h], b2 [e, m] bf16 or
 * NULL.  For the kept rows of every expert:
 *   hid = bf16(act(s_x s_w1 (x_q . w1_q^T) + b1));  hid quantised per row;
 *   out = bf16(s_h s_w2 (hid_q . w2_q^T) + b2)
 * with fp32 accumulation (tcgen05 kind::f8f6f4 on CTA pairs).  out [e, c_max,
 * m] bf16.  m and h multiples of 16.  Workspace (moe_expert_ffn_fp8_workspace
 * _size() bytes): the bf16 hidden [e, c_max, h] at offset 0, its codes [e,
 * c_max, h] and its scales [e, c_max] fp32 after it, each starting on a
 * 256-byte boundary; a caller may read them after the call.  SwiGLU returns
 * MOE_ERR_UNSUPPORTED.  This entry point extends the pages' expert FFN to the
 * FP8 format.
 */
moe_status moe_expert_ffn_fp8(const void *buf_q, const float *buf_scale, const int32_t *counts,
                              const int32_t *c_dev, const void *w1_q, const float *w1_scale,
                              const void *b1, const void *w2_q, const float *w2_scale,
                              const void *b2, moe_act act, int e, int64_t c_max, int m, int h,
                              void *workspace, size_t workspace_bytes, void *out,
                              int32_t *dev_status, void *stream);

/*
 * Routing from router logits, for gates that moe_gate_topk does not form:
 * sigmoid scores, a balance bias, group-limited selection, scaled gates.
 * Per token, with l its e logits:
 *   score_j = 1 / (1 + exp(-l_j))                       (MOE_SCORE_SIGMOID)
 *           = exp(l_j - max l) / sum_i exp(l_i - max l)  (MOE_SCORE_SOFTMAX),
 *     the sum taken by adjacent pairs (v[2j] + v[2j+1], level by level) over e
 *     padded with zeros to a power of two, divisions rounded correctly;
 *   choice_j = score_j + bias_j (bias NULL: score_j);
 *   the experts are cut into `groups` equal runs of consecutive experts; a
 *     group's value is the sum of its group_top (1 or 2) best choices, and the
 *     topk_groups groups of the largest value (ties to the lower index) stay;
 *   idx[r, t]: the r-th expert of the groups that stay by (choice descending,
 *     index ascending);
 *   gates[r, t] = score[idx[r, t]], with MOE_FLAG_NORMALIZE_GATES divided by
 *     the sum of the k of them in route order (0 where that is 0), then times
 *     `scale`.
 * The bias steers the choice and is not part of the gates, so that a balance
 * update of it changes which experts run and not what they weigh.
 * A logit of -inf masks its expert: score 0, chosen only where fewer than k
 * others stay, after them, with gate 0; it does not count in its group's value
 * (a group with none left ranks last).  A row of -inf alone gets the gates 0.
 * A NaN choice ranks like a masked expert; a NaN score passes into its gate
 * (softmax: a NaN or +inf logit makes every score of the row NaN).
 * A route to a masked expert is a route like any other: moe_capacity_locations
 * gives it a slot (a row of -inf alone: of experts 0 .. k-1), so that with a
 * capacity it can push out a token that weighs something.
 * logits [s, e] in `ldt` (16-byte aligned as a whole; its rows need not be: e may
 * be odd);
 * bias [e] fp32 or NULL; idx [k, s] int32 and gates [k, s] fp32 are written.
 * e <= 1024; e a multiple of groups, groups <= 32, 1 <= topk_groups <= groups,
 * k <= topk_groups * (e / groups).
 */
moe_status moe_route_topk(const void *logits, moe_dtype ldt, const float *bias, int64_t s, int e,
                          int k, moe_score score, int groups, int topk_groups, int group_top,
                          float scale, unsigned flags, int32_t *idx, float *gates,
                          int32_t *dev_status, void *stream);

/*
 * Gradient of moe_route_topk's gates with respect to the logits, the selection
 * taken as constant (the bias has no gradient).  With g the selected scores,
 * G = g / sum g, A = sum_r d_gates[r] G[r]:
 *   softmax, normalised: scale G (d_gates - A) at the selection, else 0;
 *   softmax, raw:  scale p_j (d_gates_j [selected] - sum_r d_gates[r] p_idx[r]);
 *   sigmoid, normalised: scale G (d_gates - A) (1 - g) at the selection, else 0;
 *   sigmoid, raw:  scale d_gates g (1 - g) at the selection, else 0.
 * The gradient goes with the gates: it is 0 where they are the constant 0 (rows
 * without a live expert; renormalised gates whose chosen scores all round to 0),
 * and NaN at the selection where a NaN or +inf in the row makes softmax gates
 * NaN.  (Elsewhere a renormalised softmax's G is formed from the chosen logits
 * and their largest, with less rounding than a quotient of scores.)
 * logits [s, e] in `ldt` as given to the
 * forward; idx, d_gates [k, s], a token's k experts distinct (as the forward
 * chooses them; of a repeated one some single route's gradient is stored);
 * d_logits [s, e] in `ddt`, every element written, sums in fp32, one rounding.
 * An idx outside [0, e) stores MOE_ERR_INVALID_ARG in dev_status.
 */
moe_status moe_route_bwd(const void *logits, moe_dtype ldt, const int32_t *idx,
                         const float *d_gates, int64_t s, int e, int k, moe_score score,
                         float scale, unsigned flags, void *d_logits, moe_dtype ddt,
                         int32_t *dev_status, void *stream);

/*
 * Microscaled 4-bit operands.  A row of `cols` values (a multiple of 32) is cut
 * into blocks of B = 32 (MOE_FP4_MX) or 16 (MOE_FP4_NV); value = code * scale:
 *   MX: scale = 2^(floor(log2 amax) - 2), at least 2^-127, stored as e8m0
 *       (exponent + 127); 1 for a block of zeros;
 *   NV: scale = s8 * g with g the batch's factor (`global_scale`, NULL: 1) and
 *       s8 = e4m3(min(amax / (6 g), 448)), nearest-even; where s8 is 0, or s8 * g
 *       so small that its reciprocal overflows (2^-128), the codes are 0;
 *   code = e2m1(x * (1 / scale)), nearest-even, saturating at +-6, 1 / scale
 *       rounded to fp32 (exact for MX).
 * A block that holds an infinity or a NaN gets the NaN scale (0xFF / 0x7F).
 * Codes: two a byte, the even column in the low half; [batches, rows, cols/2].
 * Scales: tiles of 128 rows x 4 blocks, 512 bytes each: row r, block b of a
 * tile at (r % 32) * 16 + (r / 32) * 4 + b; a batch's tiles ordered by row
 * tile, then by block tile; moe_fp4_scale_bytes() bytes per batch.  The bytes
 * of blocks past the row's last must hold a number (the library writes 0);
 * those of rows past the last are ignored.
 */
size_t moe_fp4_scale_bytes(moe_fp4 fmt, int64_t rows, int cols);

/*
 * src [batches, rows_per_batch, cols] in `sdt` -> q [batches, rows_per_batch,
 * cols/2], scale [batches, moe_fp4_scale_bytes()].  global_scale [batches]
 * fp32 > 0, NV only.  With counts [batches] and c_dev (both or neither) only
 * the rows r < min(counts[b], *c_dev, rows_per_batch) of batch b are written.
 * The codes and scales match an exact-arithmetic reference bit for bit.
 */
moe_status moe_quantize_fp4(const void *src, moe_dtype sdt, int64_t batches,
                            int64_t rows_per_batch, int cols, moe_fp4 fmt,
                            const float *global_scale, const int32_t *counts,
                            const int32_t *c_dev, void *q, void *scale, int32_t *dev_status,
                            void *stream);

/*
 * The values that 4-bit rows stand for: dst [batches, rows_per_batch, cols] in
 * `ddt` = code * scale (NV: s8 * g rounded to fp32 first), one rounding.  Rows
 * past the kept ones (counts, c_dev as above) are not written.
 */
moe_status moe_dequantize_fp4(const void *q, const void *scale, int64_t batches,
                              int64_t rows_per_batch, int cols, moe_fp4 fmt,
                              const float *global_scale, const int32_t *counts,
                              const int32_t *c_dev, void *dst, moe_dtype ddt, int32_t *dev_status,
                              void *stream);

/*
 * Grouped product of 4-bit operands: for the kept rows i < min(counts[j],
 * *c_dev, c_max) of every expert j
 *   out[j,i,:] = bf16(a_global[j] b_global[j] sum_k a[j,i,k] b[j,:,k] + bias[j])
 * with exact products and fp32 accumulation (tcgen05 block-scaled MMA).
 * a_q [e, c_max, k/2] with a_scale; b_q [e, n, k/2] with b_scale; a_global,
 * b_global [e] fp32 (NV; NULL: 1; must be NULL for MX); bias [e, n] bf16 or
 * NULL; out [e, c_max, n] bf16, other rows not written.  e = 1 is a plain
 * dense product.  k a multiple of 32, n a multiple of 8.
 */
moe_status moe_product_fp4(const void *a_q, const void *a_scale, const float *a_global,
                           const int32_t *counts, const int32_t *c_dev, const void *b_q,
                           const void *b_scale, const float *b_global, const void *bias,
                           moe_fp4 fmt, int e, int64_t c_max, int k, int n, void *out,
                           int32_t *dev_status, void *stream);

/* Bytes of device workspace moe_expert_ffn_fp4 needs (0: bad shape). */
size_t moe_expert_ffn_fp4_workspace_size(moe_fp4 fmt, moe_act act, int e, int64_t c_max, int m,
                                         int h);

/*
 * The expert FFN on 4-bit operands.  For the kept rows of every expert:
 *   hid = act(s (x . w1^T) + b1), or silu(s x . w1^T) * (s x . w3^T) (SwiGLU,
 *         no biases), in fp32 and quantised from there, block by block, as
 *         moe_quantize_fp4 does with the factor hid_global[j];
 *   out = bf16(s (hid . w2^T) + b2),
 * s the operands' factors.  (GELU is within 1e-5 of its own value down to -6,
 * 2e-4 down to -8: a block that lies in the tail is scaled by the tail.)
 * buf_q, buf_scale, buf_global: moe_quantize_fp4 of
 * the buffer's kept rows; w1, w3 [e, h, m/2], w2 [e, m, h/2] with their scales
 * and factors ([e] fp32, NV only; NULL: 1).  hid_global [e]: a fixed
 * (calibrated) factor, because a block's scale has to be known before the
 * row's other blocks are.  m, h multiples of 32.  b1 [e, h], b2 [e, m] bf16 or
 * NULL.  Workspace: the hidden's codes [e, c_max, h/2], then, from the next
 * 256-byte boundary, its scales; a caller may read them after the call.
 */
moe_status moe_expert_ffn_fp4(const void *buf_q, const void *buf_scale, const float *buf_global,
                              const float *hid_global, const int32_t *counts,
                              const int32_t *c_dev, const void *w1_q, const void *w1_scale,
                              const float *w1_global, const void *b1, const void *w3_q,
                              const void *w3_scale, const float *w3_global, const void *w2_q,
                              const void *w2_scale, const float *w2_global, const void *b2,
                              moe_fp4 fmt, moe_act act, int e, int64_t c_max, int m, int h,
                              void *workspace, size_t workspace_bytes, void *out,
                              int32_t *dev_status, void *stream);

/*
 * Rows sorted by expert ("dropless"): instead of an [e, c_max, m] buffer with a
 * capacity, one [n, m] buffer in which expert j has the rows offsets[j] ..
 * offsets[j+1]-1.  No route is dropped and no row is padding.  n is the caller's
 * (s*k always suffices) and at most 2^31 - 1024; rows from offsets[e] on belong
 * to no expert: no call reads them as data or writes them.
 *
 * moe_sort_routes: the order of the routes of idx [k, s], which is stable: the
 * rows of an expert are its routes in route-priority order (as
 * moe_capacity_locations ranks them).
 *   offsets [e+1]: offsets[0] = 0, offsets[j+1] - offsets[j] = routes of expert j;
 *   rows [k, s]: rows[r, t] = the row of route r of token t;
 *   source [k*s] or NULL: the route r*s + t of each row, -1 behind the last row.
 * An idx of -1 is a route without an expert (a padded token, an expert that is
 * not held here): it gets no row, rows = -1.  Any other idx outside [0, e)
 * stores MOE_ERR_INVALID_ARG in dev_status.  Deterministic.  k may exceed e here
 * (an expert may be named twice by a token: two rows).  workspace:
 * moe_sort_workspace_size() bytes, scratch.
 */
size_t moe_sort_workspace_size(int64_t s, int e, int k);
moe_status moe_sort_routes(const int32_t *idx, int64_t s, int e, int k, int32_t *rows,
                           int32_t *offsets, int32_t *source, void *workspace,
                           size_t workspace_bytes, int32_t *dev_status, void *stream);

/*
 * The tokens' rows on their way in: out[rows[r,t], :] = x[t, :], or, with gates
 * (NULL: none), gates[r,t] * x[t, :] (the exact product rounded once).
 * x [s, m], out [n, m] in `dt`; rows [k, s] as moe_sort_routes writes them (each
 * row at most once; -1: no row); gates [k, s] fp32.  In this call and the next
 * three a rows entry outside [-1, n) stores MOE_ERR_INVALID_ARG in dev_status, the
 * gate of a route without a row is not used, and 1 <= k <= 32.
 */
moe_status moe_encode_sorted(const void *x, moe_dtype dt, const int32_t *rows, const float *gates,
                             int64_t s, int m, int k, int64_t n, void *out, int32_t *dev_status,
                             void *stream);

/*
 * Gradient of moe_encode_sorted: d_x[t, :] = sum over the token's rows of
 * gates[r,t] * d_out[rows[r,t], :] (gates NULL: the plain sum), in fp32 in
 * ascending r from +0 with fused multiply-adds, rounded once; and, with d_gates
 * (needs gates and x, else NULL), d_gates[r,t] = <x[t, :], d_out[rows[r,t], :]> in
 * fp32 in an order fixed by the shape, 0 for a route without a row.
 */
moe_status moe_encode_sorted_bwd(const void *d_out, const void *x, moe_dtype dt,
                                 const int32_t *rows, const float *gates, int64_t s, int m, int k,
                                 int64_t n, void *d_x, float *d_gates, int32_t *dev_status,
                                 void *stream);

/*
 * The way back: y[t, :] = sum over the token's rows of gates[r,t] *
 * xs[rows[r,t], :] (gates NULL: the plain sum), in fp32 in ascending r from +0 with
 * fused multiply-adds, rounded once; 0 for a token without rows.
 */
moe_status moe_decode_sorted(const void *xs, moe_dtype dt, const int32_t *rows, const float *gates,
                             int64_t s, int m, int k, int64_t n, void *y, int32_t *dev_status,
                             void *stream);

/*
 * Gradient of moe_decode_sorted with gates: d_xs[rows[r,t], :] = gates[r,t] *
 * dy[t, :] (one rounding; rows of no route are not written), d_gates[r,t] =
 * <dy[t, :], xs[rows[r,t], :]> in fp32, 0 for a route without a row.  (Without
 * gates, d_xs is moe_encode_sorted of dy.)
 */
moe_status moe_decode_sorted_bwd(const void *dy, const void *xs, moe_dtype dt, const int32_t *rows,
                                 const float *gates, int64_t s, int m, int k, int64_t n,
                                 void *d_xs, float *d_gates, int32_t *dev_status, void *stream);

/*
 * The expert FFN (moe_expert_ffn, _train) on sorted rows: for every expert j and
 * its rows i,
 *   hid[i,:] = act(x[i,:] W1[j]^T + b1[j]), or silu(x W1^T) * (x W3^T) (SwiGLU);
 *   out[i,:] = hid[i,:] W2[j]^T + b2[j],
 * fp32 accumulation; hid [n, h] is an output, rounded to bf16, and what the second
 * product reads.  pre (NULL: not kept): the pre-activation [n, h], SwiGLU's a and b
 * [n, 2h], rounded to bf16, for moe_expert_ffn_sorted_bwd.  x, out [n, m]; offsets
 * [e+1] int32 on the device, ascending from 0 to at most n (else, in every call on
 * sorted rows, MOE_ERR_INVALID_ARG in dev_status and unspecified rows inside the
 * buffers); weights and biases as moe_expert_ffn.  A NaN in a row makes that row of
 * hid and out NaN, under ReLU too, and no other.  bf16 only.
 */
moe_status moe_expert_ffn_sorted(const void *x, moe_dtype dt, const int32_t *offsets,
                                 const void *w1, const void *b1, const void *w3, const void *w2,
                                 const void *b2, moe_act act, int e, int64_t n, int m, int h,
                                 void *hid, void *pre, void *out, int32_t *dev_status,
                                 void *stream);

/* Bytes of device workspace moe_expert_ffn_sorted_bwd needs (0: bad shape). */
size_t moe_expert_ffn_sorted_bwd_workspace_size(moe_act act, int e, int64_t n, int m, int h);

/*
 * Gradient of moe_expert_ffn_sorted from what it kept (hid, pre), as
 * moe_expert_ffn_bwd_saved: d_x [n, m] (other rows not written) and the weights' and
 * biases' gradients in wgrad_dt (MOE_BF16 or MOE_F32), zeros for an expert without
 * rows.  d_pre = (d_out W2) * act'(pre) is rounded to bf16 as the operand of the
 * products after it; sums in fp32.  d_b1, d_b2 may be NULL.
 */
moe_status moe_expert_ffn_sorted_bwd(const void *x, const void *hid, const void *pre, moe_dtype dt,
                                     const int32_t *offsets, const void *w1, const void *w3,
                                     const void *w2, moe_act act, int e, int64_t n, int m, int h,
                                     const void *d_out, void *workspace, size_t workspace_bytes,
                                     void *d_x, moe_dtype wgrad_dt, void *d_w1, void *d_w3,
                                     void *d_w2, void *d_b1, void *d_b2, int32_t *dev_status,
                                     void *stream);

/*
 * 8-bit integer rows, one fp32 scale each: value = code * scale,
 *   scale = amax / 127,  code = round(x * (127 / amax)) to nearest even,
 * in fp32 (both quotients and the product rounded); codes 0 and scale 1 for a row
 * whose largest magnitude amax is below 2^-100, codes 0 and a NaN scale for a row
 * that holds an infinity or a NaN.
 *
 * moe_quantize_rows_int8: src [s, cols] in `sdt`, cols a multiple of 16.
 *   rows NULL: q [s, cols] int8, scale [s]; k = 0 and n = s then;
 *   rows [k, s] (moe_sort_routes): the codes and scale of token t go to the rows
 *   rows[r, t] of q [n, cols], scale [n], as moe_encode_sorted moves rows (the
 *   tokens are read once); other rows are not written.
 * Weights [e, rows, cols] are quantised per output channel as e * rows rows.
 */
moe_status moe_quantize_rows_int8(const void *src, moe_dtype sdt, const int32_t *rows, int64_t s,
                                  int cols, int k, int64_t n, void *q, float *scale,
                                  int32_t *dev_status, void *stream);

/* Bytes of device workspace moe_product_int8 needs (0: bad shape). */
size_t moe_product_int8_workspace_size(int e, int64_t n, int k, int n_out);

/*
 * Grouped product of 8-bit integers on sorted rows: for every expert j and its
 * rows i (offsets as moe_expert_ffn_sorted; NULL with e = 1: all n rows)
 *   out[i,:] = a_scale[i] b_scale[j,:] (sum_k a_q[i,k] b_q[j,:,k]) + bias[j,:],
 * rounded once to `odt`.  a_q [n, k] int8 with a_scale [n]; b_q [e, n_out, k] int8
 * with b_scale [e, n_out] (one per output channel); bias [e, n_out] bf16 or NULL;
 * out [n, n_out].  Codes may take all of -128 .. 127, scales any value (their product
 * may leave fp32's range).  The sum is exact while its partial sums stay below 2^24
 * (for k <= 1024 always); beyond it is an fp32 sum (of few rows it is exact all the
 * same).  k a multiple of 16 below 2^17, n_out a multiple of 8.
 */
moe_status moe_product_int8(const void *a_q, const float *a_scale, const int32_t *offsets,
                            const void *b_q, const float *b_scale, const void *bias, int e,
                            int64_t n, int k, int n_out, void *workspace, size_t workspace_bytes,
                            void *out, moe_dtype odt, int32_t *dev_status, void *stream);

/* Bytes of device workspace moe_expert_ffn_int8 needs (0: bad shape). */
size_t moe_expert_ffn_int8_workspace_size(moe_act act, int e, int64_t n, int m, int h);

/*
 * The expert FFN on 8-bit integer operands and sorted rows: for every expert's rows
 *   hid = bf16(act(x . w1^T + b1)), or bf16(silu(x . w1^T) * (x . w3^T)) (SwiGLU, no
 *         biases), quantised by rows as moe_quantize_rows_int8 does;
 *   out = bf16(hid . w2^T + b2),
 * the products as moe_product_int8 forms them.  GELU within 1e-3 of its value down to
 * a pre-activation of -8 (a row is scaled by its maximum, which may lie there).
 * x_q [n, m], x_scale [n]; w1, w3 [e, h, m], w2 [e, m, h] int8 with scales [e, h],
 * [e, h], [e, m]; b1 [e, h], b2 [e, m] bf16 or NULL; out [n, m] bf16.  m and h
 * multiples of 16 below 2^17.  Workspace: the hidden [n, h] bf16, then, from the next
 * 256-byte boundary, its scales [n]; a caller may read them after the call.
 */
moe_status moe_expert_ffn_int8(const void *x_q, const float *x_scale, const int32_t *offsets,
                               const void *w1_q, const float *w1_scale, const void *b1,
                               const void *w3_q, const float *w3_scale, const void *w2_q,
                               const float *w2_scale, const void *b2, moe_act act, int e, int64_t n,
                               int m, int h, void *workspace, size_t workspace_bytes, void *out,
                               int32_t *dev_status, void *stream);

/* Bytes of device workspace moe_layer_forward needs. */
size_t moe_layer_workspace_size(moe_dtype dt, moe_act act, int64_t s, int m, int e, int k,
                                int64_t c_max, int h);

/*
 * The whole forward layer in one call: moe_gate_topk, moe_capacity_locations,
 * moe_encode, moe_expert_ffn and moe_decode enqueued back to back on `stream`
 * with no host synchronisation.  Intermediate tensors the caller may inspect
 * (idx, gates, loc, counts, c_dev, buf, out) are caller-owned outputs; the
 * rest lives in `workspace` (moe_layer_workspace_size() bytes).
 */
moe_status moe_layer_forward(const void *x, moe_dtype dt, const float *wg, const float *gate_bias,
                             const void *w1, const void *b1, const void *w3, const void *w2,
                             const void *b2, moe_act act, int64_t s, int m, int e, int k, int h,
                             float capacity_factor, int64_t c_max, unsigned flags,
                             int32_t *idx, float *gates, int32_t *loc, int32_t *counts,
                             int32_t *c_dev, void *buf, void *out, void *y,
                             void *workspace, size_t workspace_bytes,
                             int32_t *dev_status, void *stream);

/*
 * moe_layer_forward with the layer's input taken from host memory and its
 * output returned to host memory, for a caller whose tokens live on the host:
 * x_host [s, m] is copied into the device buffer x, the layer runs as in
 * moe_layer_forward, and y is copied to y_host [s, m], all three enqueued on
 * `stream` (cudaMemcpyAsync: with pinned host memory the copies are
 * asynchronous; with pageable memory the runtime may block the calling thread
 * until they are done).  Arguments after x are those of moe_layer_forward.
 * The caller synchronises the stream before reading y_host.
 */
moe_status moe_layer_forward_host(const void *x_host, void *y_host, const void *x, moe_dtype dt,
                                  const float *wg, const float *gate_bias, const void *w1,
                                  const void *b1, const void *w3, const void *w2, const void *b2,
                                  moe_act act, int64_t s, int m, int e, int k, int h,
                                  float capacity_factor, int64_t c_max, unsigned flags,
                                  int32_t *idx, float *gates, int32_t *loc, int32_t *counts,
                                  int32_t *c_dev, void *buf, void *out, void *y, void *workspace,
                                  size_t workspace_bytes, int32_t *dev_status, void *stream);

/*
 * moe_layer_forward with the capacity dimension cut into `chunks` pieces so
 * that encoding one piece overlaps the expert FFN of the previous one (the
 * one-GPU form of the adaptive pipelining in [Blog] 3.4, which overlaps
 * all-to-all with expert computation by splitting the capacity dimension):
 * gate and capacity run on `stream`; slot rows [i*q, (i+1)*q) of every expert
 * (q = c_max / chunks rounded up to 256 rows) are encoded on `aux_stream` and
 * run through the FFN on `stream` once their encode is done; decode follows
 * on `stream` (a token's routes may fall in different pieces).  Results are
 * bit-identical to moe_layer_forward.  events: 1 + chunks cudaEvent_t handles
 * (passed as void*) created by the caller, used for the cross-stream order;
 * aux_stream may equal stream (no overlap).  bf16 only (fp32, or chunks = 1:
 * the single pass).  1 <= chunks <= 64.  The caller synchronises `stream`.
 */
moe_status moe_layer_forward_pipelined(const void *x, moe_dtype dt, const float *wg,
                                       const float *gate_bias, const void *w1, const void *b1,
                                       const void *w3, const void *w2, const void *b2, moe_act act,
                                       int64_t s, int m, int e, int k, int h, float capacity_factor,
                                       int64_t c_max, unsigned flags, int32_t *idx, float *gates,
                                       int32_t *loc, int32_t *counts, int32_t *c_dev, void *buf,
                                       void *out, void *y, void *workspace, size_t workspace_bytes,
                                       int32_t *dev_status, int chunks, void *stream,
                                       void *aux_stream, void *const *events);

/*
 * Measurement helper, not part of the layer: launches `blocks` CTAs of 256
 * threads, each thread running 8 independent two-wide chains of `iters` fp32
 * fused multiply-adds (packed fp32x2 FMA when `packed`, else scalar pairs),
 * i.e. blocks * 256 * iters * 32 flop.  Timed by the caller with events, it
 * gives this GPU's fp32 FMA throughput, the roofline of a gate whose logits
 * (2*m*e flop per token) outweigh its HBM bytes.  out: one device float the
 * kernel may write (never for these values).
 */
moe_status moe_probe_fp32_fma(int packed, int blocks, int iters, float *out, void *stream);

/* Human-readable name of a status code (static string). */
const char *moe_status_str(moe_status st);

/* Number of kernels this library has launched in this process (monotonic). */
uint64_t moe_launch_count(void);

/*
 * Error-path test hook, not for production use.  The next n launches of the
 * tensor-core grouped GEMMs in this process (moe_expert_ffn, _fp8, _fp4, _bwd,
 * moe_product_fp4 and the layer calls use them; fc1 and fc2 are one launch each) issue no operand
 * copies, so the MMA issuer's bounded wait on its first stage runs out after
 * about one second: the launch sets MOE_ERR_TIMEOUT in the call's status
 * word, drains, releases its tensor memory and returns, and every later
 * kernel that reads that status word writes nothing.  The context stays
 * usable.  n = 0 cancels pending stalls.  The count is process-wide: calls
 * made meanwhile from other threads may take the stalls.
 * Errors: MOE_ERR_INVALID_ARG for n < 0.
 */
moe_status moe_debug_stall_gemms(int32_t n);

/*
 * Test hook, not for production use.  In the next n launches of the 4-bit
 * grouped products in this process (moe_product_fp4, and two per
 * moe_expert_ffn_fp4) the copies of the second half of every row tile lag by
 * 20 us a stage: slower, with the same results.  n = 0 cancels what is pending.
 * Errors: MOE_ERR_INVALID_ARG for n < 0.
 */
moe_status moe_debug_lag_gemms(int32_t n);

#ifdef __cplusplus
}
#endif
#endif /* MOE_GATE_H */
