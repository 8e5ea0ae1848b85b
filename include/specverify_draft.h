/*
 * libspecverify_draft: operators of a draft step, a companion of libspecverify
 * with the same conventions (specverify.h): device pointers owned by the
 * caller, nothing allocated, no pointer kept, asynchronous on `stream`,
 * host-checkable errors returned with nothing enqueued, no random numbers
 * drawn.  It is a library of its own so that the others' sets of symbols and
 * their versions stay as they are.
 *
 *  specv_fp4_*      an LM head on 4-bit floats with one scale for each block of
 *                   32 along the hidden size (microscaled), for hidden states
 *                   in 4 or in 8 bits
 *  specv_filter_*   each row's distribution after temperature, top-k, top-p and
 *                   min-p, with parameters of each request's own, and one token
 *                   drawn from it: what a draft step emits, and what
 *                   specv_verify_probs takes
 */
#ifndef SPECVERIFY_DRAFT_H
#define SPECVERIFY_DRAFT_H

#include "specverify.h"

#if defined(__GNUC__)
#define SPECV_DRAFT_API __attribute__((visibility("default")))
#else
#define SPECV_DRAFT_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Sizes whose launch would take 2^32 or more threads are SPECV_EUNSUPPORTED. */

/* Values that share one scale in the 4-bit format. */
#define SPECV_FP4_BLOCK 32

/*
 * Values in 4 bits with a power-of-two scale for each block of 32 along the
 * last axis: x[r][d] ~ q[r][d] * 2^(scale[r][d / 32] - 127), q an e2m1 code (0,
 * 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives).  The scale is the smallest power
 * of two (at least 2^-126) that brings the block's largest magnitude to at most
 * 6, 1 for a block of zeros; q is x / scale rounded to the nearest code, ties to
 * the even one, so that no value is clipped.  A block that holds a NaN or an
 * infinity gets scale byte 255, the NaN of the e8m0 format, and zero codes.
 *
 *  x      [rows][D] of dtype (bfloat16 or float32), 16-byte aligned.
 *  q      [rows][D/2] output, 4-byte aligned: element 2 i in the low half of
 *         byte i, element 2 i + 1 in the high half.
 *  scale  [rows][D/32] output.
 * rows >= 1; D a positive multiple of 32, at most SPECV_MAX_D.  Outputs do not
 * overlap x or each other.
 */
SPECV_DRAFT_API specv_status_t specv_fp4_quantize(const void *x, specv_dtype_t dtype, int rows,
                                                  int D, uint8_t *q, uint8_t *scale,
                                                  hipStream_t stream);

/*
 * An LM-head weight in 4 bits (q [V][D/2], scale [V][D/32], as
 * specv_fp4_quantize writes them) in the order the product below reads it.
 * Pack it once, when the model is loaded.
 *
 * The packed weight is [ceil(V/32)][D/64][64] 16-byte pieces: piece (g, s, l)
 * holds the 32 codes of row 32 g + l % 32 from column 64 s + 32 (l / 32) on,
 * zeros past V; then [ceil(V/32)][ceil(D/256)][64] 4-byte words of scale
 * bytes: byte i of word (g, j, l) is scale[32 g + l % 32][8 j + 2 i + l / 32],
 * 127 past the end.
 *
 * specv_fp4_lm_head_packed_weight_bytes: the packed size, or 0 for invalid
 * sizes (V outside [1, SPECV_MAX_V], D not a positive multiple of 128 or
 * above SPECV_MAX_D).
 * specv_fp4_lm_head_pack_weight: q 16-byte aligned; packed_weight 16-byte
 * aligned and not overlapping q or scale.
 */
SPECV_DRAFT_API size_t specv_fp4_lm_head_packed_weight_bytes(int V, int D);
SPECV_DRAFT_API specv_status_t specv_fp4_lm_head_pack_weight(const uint8_t *q, const uint8_t *scale,
                                                             void *packed_weight, int V, int D,
                                                             hipStream_t stream);

/* How the hidden states of the product below are held. */
typedef enum {
  SPECV_HIDDEN_E4M3 = 0,  /* e4m3 bytes [M][D], a scale byte for each 128 (specv_hidden_norm) */
  SPECV_HIDDEN_E2M1 = 1   /* e2m1 codes [M][D/2], a scale byte for each 32 (specv_fp4_quantize) */
} specv_hidden_t;

/*
 * The LM head on 4-bit floats, on the matrix cores:
 *   logits[m][v] = sum_d h[m][d] w[v][d]
 * of the values that codes and scales stand for, rounded to out_dtype to
 * nearest even.  4-bit hidden states and float32 logits accumulate in float32.
 * bfloat16 logits of 8-bit hidden states take the matrix cores' mixed product,
 * which drops of each 8 products that it adds at once what lies below 2^-13 of
 * the largest: besides the rounding such a logit may be off by up to 2^-10 of
 * sum |h w|, which tells where large products cancel.
 *
 *  hidden         [M][D] or [M][D/2] bytes of hidden_type, 16-byte aligned.
 *  hidden_scale   [M][D/128] or [M][D/32] e8m0 bytes.
 *  packed_weight  as specv_fp4_lm_head_pack_weight writes it for V and D.
 *  logits         [M][V] of out_dtype, output; not overlapping the inputs.
 * M >= 1, 1 <= V <= SPECV_MAX_V, D a positive multiple of 128 up to
 * SPECV_MAX_D.  A NaN (an e4m3 byte or a scale byte) in a hidden row makes that
 * row of logits NaN, one in a weight row that vocabulary id.  Float32 logits of
 * 8-bit hidden states take each value, element times scale, as a bfloat16
 * number: one below 2^-126 in size may count as 0, one past the largest float
 * as infinite (scale bytes below 10 or above 246 alone can make such values).
 */
SPECV_DRAFT_API specv_status_t specv_fp4_lm_head(const uint8_t *hidden, specv_hidden_t hidden_type,
                                                 const uint8_t *hidden_scale,
                                                 const void *packed_weight, int M, int D, int V,
                                                 void *logits, specv_dtype_t out_dtype,
                                                 hipStream_t stream);

/*
 * The filters of a call's rows.  Each is an array with one value a request, on
 * the device, or, where the array is NULL, the one value beside it for all.
 *  temperature  >= 0 and finite.  0 is greedy: the distribution is one at the
 *               lowest id among the largest logits, whatever the other filters.
 *  top_k        0 = off; otherwise keep logits >= the top_k-th largest (ties
 *               kept).  top_k >= V is the same as off.
 *  top_p        1 = off; otherwise in (0, 1): keep the shortest prefix of the
 *               top-k renormalised distribution, by logit descending, whose
 *               mass reaches top_p (crossing token and its ties kept).
 *  min_p        0 = off; otherwise in [0, 1]: keep tokens at least min_p times
 *               as probable as the most probable one.
 * A token is kept where all three keep it.
 */
typedef struct {
  const float *temperature_array;
  const int32_t *top_k_array;
  const float *top_p_array;
  const float *min_p_array;
  float temperature;
  int32_t top_k;
  float top_p;
  float min_p;
} specv_filters_t;

/*
 * Filtered distributions and draws.  Row l of request b is
 *   p(v) = exp((z(v) - max z) / T) / S over the kept tokens, 0 elsewhere,
 * S their sum, and its token the first id whose running sum of the kept
 * weights exceeds u S (ids ascending, strict comparison, as specv_sample
 * draws; a weight of at most 1e-290 of the largest counts as nothing).  Weights
 * are float64, good to 1e-13 of their size down to 100 T below the largest logit.
 * Min-p is decided on a weight, top-p on sums of weights in whole multiples of
 * 2^-s of the largest one, s = 62 - ceil(log2 V) but at most 51; the draw sums in
 * float64.  Results do not change from run to run.
 *
 *  logits      row l of request b starts at element b * stride_b + l *
 *              stride_l, V consecutive values of dtype, any alignment of an
 *              element; finite or -inf (-inf masks a token out).  Strides here and
 *              below are in elements and at least 0.
 *  filters     see above; read on the host, its arrays on the device.
 *  u           [B][L] float32 in [0, 1) with its strides; NULL where out_tokens is.
 *  out_tokens  [B][L] int32 output with its strides, or NULL: distributions only.
 *  probs       output, rows as of logits with its own strides, of probs_dtype
 *              (rounded to nearest even through float32), or NULL: tokens only.
 *  workspace   at least specv_filter_workspace_bytes(B, L, V, dtype) bytes,
 *              16-byte aligned; needs no initialisation.  A small V needs none:
 *              the size is then 0 (as for sizes the call refuses).
 *
 * B, L >= 1, 1 <= V <= SPECV_MAX_V.  Outputs and workspace do not overlap the
 * inputs or each other (between rows whose strides leave room they may lie),
 * nor an output's rows each other.  A row with a parameter outside its range,
 * with u outside [0, 1) where a token is asked for, with no finite logit, or
 * with a NaN or +inf logit has token -1 and probabilities 0; other rows are not
 * affected.
 */
SPECV_DRAFT_API size_t specv_filter_workspace_bytes(int B, int L, int V, specv_dtype_t dtype);
SPECV_DRAFT_API specv_status_t specv_filter(const void *logits, int64_t stride_b, int64_t stride_l,
                                            specv_dtype_t dtype, int B, int L, int V,
                                            const specv_filters_t *filters, const float *u,
                                            int64_t u_stride_b, int64_t u_stride_l,
                                            int32_t *out_tokens, int64_t token_stride_b,
                                            int64_t token_stride_l, void *probs,
                                            int64_t probs_stride_b, int64_t probs_stride_l,
                                            specv_dtype_t probs_dtype, void *workspace,
                                            size_t workspace_bytes, hipStream_t stream);

/* Version of this library, 100 * major + minor. */
SPECV_DRAFT_API int specv_draft_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SPECVERIFY_DRAFT_H */
