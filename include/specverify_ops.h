/*
 * libspecverify_ops: operators around the verification step, a companion of
 * libspecverify with the same conventions (specverify.h): device pointers
 * owned by the caller, nothing allocated, no pointer kept, asynchronous on
 * `stream`, host-checkable errors returned with nothing enqueued, no random
 * numbers drawn.  It is a library of its own so that libspecverify's set of
 * symbols and its version stay as they are.
 *
 *  specv_hidden_norm         the norms around the target's last block with its
 *                            gate and residual scale: the hidden states that
 *                            an LM head takes, in bfloat16, float32 or 8 bits
 *  specv_fp8_*               an LM head on 8-bit floats with one scale for
 *                            each run of 128 along the hidden size
 *  specv_verify_fp8_lm_head  the verification step on that LM head's logits
 *  specv_verify_probs        the verification step from probabilities instead
 *                            of logits, with or without a draft distribution
 */
#ifndef SPECVERIFY_OPS_H
#define SPECVERIFY_OPS_H

#include "specverify.h"

#if defined(__GNUC__)
#define SPECV_OPS_API __attribute__((visibility("default")))
#else
#define SPECV_OPS_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Sizes whose launch would take 2^32 or more threads are SPECV_EUNSUPPORTED. */

/* Values that share one scale in the 8-bit formats below. */
#define SPECV_FP8_BLOCK 128

/* Element type of an output that may be 8-bit. */
typedef enum {
  SPECV_OUT_F32 = 0,
  SPECV_OUT_BF16 = 1,
  SPECV_OUT_E4M3 = 2      /* e4m3 bytes (largest value 448) with e8m0 scales */
} specv_out_t;

/*
 * The norms around the last block of the target model, fused with the
 * block's gate and residual scale.  With N(v; w) = w * v / sqrt(mean(v^2) +
 * eps), for every row m of M:
 *
 *   r'[m] = residual[m] + scale * gate[m / (M / gate_rows)] * N(x[m]; post_weight)
 *   y[m]  = N(r'[m]; weight)
 *
 *  x            [M][D] of x_dtype: the block's output.
 *  residual     [M][D] of residual_dtype: the residual stream before the block.
 *  post_weight  [D] of weight_dtype, or NULL: x is then taken as it is.
 *  gate         [gate_rows][D] of weight_dtype, or NULL (a factor of one):
 *               1 row for all, one for each request (M / gate_rows consecutive
 *               rows share it) or one for each row.  gate_rows divides M; it is
 *               not read when gate is NULL.
 *  weight       [D] of weight_dtype.
 *  scale, eps   finite; eps > 0.
 *  residual_out [M][D] of residual_dtype, output: r' rounded to nearest even.
 *               It may be the residual array itself.
 *  out          [M][D] output: y as out_dtype, rounded to nearest even (y is
 *               formed from r' before its rounding).  With SPECV_OUT_E4M3, D is
 *               a multiple of SPECV_FP8_BLOCK and out holds e4m3 bytes as
 *               specv_fp8_quantize writes them.  It may be the x array itself
 *               where both have the same element type.
 *  out_scale    [M][D/128] e8m0 bytes, output; read only with SPECV_OUT_E4M3.
 *
 * M >= 1, 1 <= D <= SPECV_MAX_D.  Arrays element-aligned; with 16-byte aligned
 * arrays and D a multiple of 8 all loads are 16 bytes wide; e4m3 output needs
 * out 8-byte aligned.  Outputs may not overlap inputs or each other but for
 * the two cases above.  Sums in float32: a row of x or r' whose sum of squares
 * passes the largest float is scaled by 0.  A NaN or an infinity in a row
 * makes NaN of that row's y at least where it stands (a whole run of 128 with
 * SPECV_OUT_E4M3); other rows are not affected.
 */
SPECV_OPS_API specv_status_t specv_hidden_norm(
    const void *x, specv_dtype_t x_dtype, const void *residual, specv_dtype_t residual_dtype,
    const void *post_weight, const void *gate, int gate_rows, const void *weight,
    specv_dtype_t weight_dtype, int M, int D, float scale, float eps, void *residual_out,
    void *out, specv_out_t out_dtype, uint8_t *out_scale, hipStream_t stream);

/*
 * Values in 8 bits with a power-of-two scale for each run of 128 along the
 * last axis: x[r][d] ~ q[r][d] * 2^(scale[r][d / 128] - 127).  The scale is
 * the smallest power of two (at least 2^-126) that brings the run's largest
 * magnitude to at most 448, 1 for a run of zeros; q is x / scale rounded to
 * the nearest e4m3 value, ties to even.  With elements that are floating
 * point themselves a power-of-two scale costs no relative precision, and the
 * matrix cores apply it.  A run that holds a NaN or an infinity becomes NaN
 * bytes (0x7f) with scale byte 255, the NaN of the e8m0 format.
 *
 *  x      [rows][D] of dtype (bfloat16 or float32), 16-byte aligned.
 *  q      [rows][D] output, 8-byte aligned.
 *  scale  [rows][D/128] output.
 * rows >= 1; D a positive multiple of 128, at most SPECV_MAX_D.  Outputs do
 * not overlap x or each other.
 */
SPECV_OPS_API specv_status_t specv_fp8_quantize(const void *x, specv_dtype_t dtype, int rows, int D,
                                                uint8_t *q, uint8_t *scale, hipStream_t stream);

/*
 * An LM-head weight in 8 bits (q [V][D] e4m3, scale [V][D/128] e8m0, as
 * specv_fp8_quantize writes them) in the order the products below read it.
 * Pack it once, when the model is loaded.
 *
 * The packed weight is [ceil(V/32)][D/128][4][64] 16-byte pieces: piece
 * (g, kb, s, l) holds q[32 g + l % 32][128 kb + 64 (s / 2) + 32 (l / 32) +
 * 16 (s % 2) .. + 15],
 * zeros past V; then [ceil(V/32)][ceil(D/512)][32] 4-byte words of scale
 * bytes: byte i of word (g, j, r) is scale[32 g + r][4 j + i], 127 past the
 * end.
 *
 * specv_fp8_lm_head_packed_weight_bytes: the packed size, or 0 for invalid
 * sizes (V outside [1, SPECV_MAX_V], D not a positive multiple of 128 or
 * above SPECV_MAX_D).
 * specv_fp8_lm_head_pack_weight: q 16-byte aligned; packed_weight 16-byte
 * aligned and not overlapping q or scale.
 */
SPECV_OPS_API size_t specv_fp8_lm_head_packed_weight_bytes(int V, int D);
SPECV_OPS_API specv_status_t specv_fp8_lm_head_pack_weight(const uint8_t *q, const uint8_t *scale,
                                                           void *packed_weight, int V, int D,
                                                           hipStream_t stream);

/*
 * The LM head on 8-bit floats, on the matrix cores:
 *   logits[m][v] = sum_b hs[m][b] ws[v][b] sum_{d in run b} hq[m][d] wq[v][d]
 * rounded to out_dtype to nearest even.  Float32 logits accumulate in float32.
 * bfloat16 logits take the matrix cores' 8-bit product, which holds less: of
 * each 8 products that it adds at once it drops of each what lies below 2^-13
 * of the largest, before it adds them to a float32 sum.  Besides the rounding a
 * bfloat16 logit may so be off by up to 2^-10 of sum |h w| (on random operands
 * some 1e-5 to 6e-5 of a typical logit, 0.3 to 1.5 % of 2^-8: one logit in 60
 * rounds the other way), which tells where large products cancel.
 *
 *  hidden         [M][D] e4m3 bytes, 16-byte aligned.
 *  hidden_scale   [M][D/128] e8m0 bytes.
 *  packed_weight  as specv_fp8_lm_head_pack_weight writes it for V and D.
 *  logits         [M][V] of out_dtype, output; not overlapping the inputs.
 * M >= 1, 1 <= V <= SPECV_MAX_V, D a positive multiple of 128 up to
 * SPECV_MAX_D.  A NaN byte (element or scale) in a hidden row makes that row
 * of logits NaN, one in a weight row that vocabulary id.  Float32 logits take
 * each value, element times scale, as a bfloat16 number: one below 2^-126 in
 * size may count as 0, one past the largest float as infinite (scale bytes
 * below 10 or above 246 alone can make such values).
 */
SPECV_OPS_API specv_status_t specv_fp8_lm_head(const uint8_t *hidden, const uint8_t *hidden_scale,
                                               const void *packed_weight, int M, int D, int V,
                                               void *logits, specv_dtype_t out_dtype,
                                               hipStream_t stream);

/*
 * The verification step on that LM head's logits: specv_fp8_lm_head writes
 * target_logits [B][K+1][V] bfloat16 from hidden [B][K+1][D], and
 * specv_verify_debug runs on them, with the same arguments, status codes,
 * per-request errors and nullable diagnostics.  The workspace is at least
 * specv_verify_fp8_lm_head_workspace_bytes(...) bytes, 16-byte aligned.
 * Outputs and workspace do not overlap the inputs or each other.  In a
 * captured graph that takes path 3 (specv_path_kind) the workspace either
 * belongs to that graph alone, untouched between replays, or is cleared by a
 * fill kernel in the graph before this call.
 */
SPECV_OPS_API size_t specv_verify_fp8_lm_head_workspace_bytes(int B, int K, int V, int D, int top_k,
                                                              float top_p);
SPECV_OPS_API specv_status_t specv_verify_fp8_lm_head(
    const uint8_t *hidden, const uint8_t *hidden_scale, const void *packed_weight,
    const void *draft_logits, const int32_t *draft_tokens, const int32_t *draft_len,
    const float *u, const float *u_final, int B, int K, int V, int D, float temperature, int top_k,
    float top_p, int eos_id, void *target_logits, int32_t *out_tokens, int32_t *n_emitted,
    void *workspace, size_t workspace_bytes, hipStream_t stream, float *accept_prob,
    double *residual_mass, int32_t *stop_pos, int32_t *path);

/*
 * The verification step from probabilities: for engines whose target and
 * draft distributions are already processed (whatever their filters), and for
 * drafts that come without a distribution (a lookup or an n-gram table).
 * The rule is specv_verify's: draft x_k is accepted when u[b][k] < p_k(x_k) /
 * q_k(x_k); the first rejection j is replaced by a draw from
 * max(p_j - q_j, 0), and after n accepted drafts a bonus token is drawn from
 * p_n, both by inverse CDF at u_final[b] over ascending token ids, the draw
 * scaled by the weights' own sum.  The accept test is exact: u q < p is
 * decided on the products themselves.  The draws sum in float64.  A rejection
 * whose residual is zero everywhere (p <= q at every token, which only
 * rounding of the caller's probabilities allows) is replaced by a draw from
 * p_j.
 *
 *  target_probs  row k of request b starts at element b * target_stride_b +
 *                k * target_stride_k, k = 0..K, V consecutive values of dtype.
 *  draft_probs   the same with draft_stride_b, draft_stride_k, k = 0..K-1; or
 *                NULL: q_k is then one at the drafted token, zero elsewhere
 *                (and so x_k is accepted when u < p_k(x_k), and the correction
 *                drawn from p_j without x_j).  Strides are at least 0, in
 *                elements.
 *  draft_tokens, draft_len, u, u_final, eos_id, out_tokens, n_emitted: as for
 *                specv_verify.
 *  workspace     at least specv_verify_probs_workspace_bytes(B, K, V) bytes,
 *                16-byte aligned; needs no initialisation.  A small V needs
 *                none: the size is then 0 (as for sizes the call refuses).
 *  accept_prob, residual_mass, stop_pos, path: nullable diagnostics, as for
 *                specv_verify_debug.
 *
 * Outputs and workspace do not overlap the inputs or each other; between rows
 * whose strides leave room they may lie.
 *
 * 1 <= B, 0 <= K <= SPECV_MAX_K, 1 <= V <= SPECV_MAX_V.  Per-request errors
 * as specv_verify (draft_len, a token or a uniform out of range, q(x) not
 * positive); also a probability that is negative, NaN or infinite among those
 * the request reads (its drafted tokens' entries and the rows its draw uses),
 * or a target row to draw from that sums to zero.  Rows need not sum to one:
 * the accept test takes the values as they are.
 */
SPECV_OPS_API size_t specv_verify_probs_workspace_bytes(int B, int K, int V);
SPECV_OPS_API specv_status_t specv_verify_probs(
    const void *target_probs, int64_t target_stride_b, int64_t target_stride_k,
    const void *draft_probs, int64_t draft_stride_b, int64_t draft_stride_k, specv_dtype_t dtype,
    const int32_t *draft_tokens, const int32_t *draft_len, const float *u, const float *u_final,
    int B, int K, int V, int eos_id, int32_t *out_tokens, int32_t *n_emitted, void *workspace,
    size_t workspace_bytes, hipStream_t stream, float *accept_prob, double *residual_mass,
    int32_t *stop_pos, int32_t *path);

/* Version of this library, 100 * major + minor. */
SPECV_OPS_API int specv_ops_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SPECVERIFY_OPS_H */
