// C ABI of libspecverify_draft: argument checks and launches on the caller's
// stream.  The declarations and their contract live in
// include/specverify_draft.h.
#include "specverify_draft.h"

#include <cmath>
#include <cstdint>

#include "abi_checks.h"
#include "strided.h"

namespace specv {
bool fp4_quantize_fits(int rows, int D);
hipError_t launch_fp4_quantize(const void* x, bool bf16, int rows, int D, uint8_t* q,
                               uint8_t* scale, hipStream_t stream);
size_t fp4_packed_bytes(int V, int D);
bool fp4_pack_fits(int V, int D);
hipError_t launch_fp4_pack(const uint8_t* q, const uint8_t* scale, void* packed, int V, int D,
                           hipStream_t stream);
bool fp4_head_fits(int M, int V);
hipError_t launch_fp4_head(const uint8_t* hidden, bool h8, const uint8_t* hscale, const void* packed,
                           int M, int D, int V, void* logits, bool bf16, hipStream_t stream);
bool filter_fits(int B, int L, int V, bool bf16);
size_t filter_workspace_bytes(int B, int L, int V, bool bf16);
hipError_t launch_filter(const void* logits, long long zsb, long long zsl, bool bf16, int B, int L,
                         int V, const specv_filters_t& f, const float* u, long long usb,
                         long long usl, int* tokens, long long tsb, long long tsl, void* probs,
                         long long psb, long long psl, bool probs_bf16, void* workspace,
                         hipStream_t stream);

namespace {

constexpr int kRun = 128;                        // columns of a product's run

specv_status_t check_head_sizes(int M, int D, int V) {
  if (M < 1 || V < 1 || D < 1 || D % kRun != 0) return SPECV_EINVAL;
  if (V > SPECV_MAX_V || D > SPECV_MAX_D) return SPECV_EUNSUPPORTED;
  if (!fp4_head_fits(M, V) || !fp4_pack_fits(V, D)) return SPECV_EUNSUPPORTED;
  return SPECV_OK;
}

specv_status_t check_filter_sizes(int B, int L, int V, specv_dtype_t dtype) {
  if (B < 1 || L < 1 || V < 1 || !known(dtype)) return SPECV_EINVAL;
  if (V > SPECV_MAX_V || (long long)B * L > 0x7fffffff) return SPECV_EUNSUPPORTED;
  if (!filter_fits(B, L, V, dtype == SPECV_BF16)) return SPECV_EUNSUPPORTED;
  return SPECV_OK;
}

// Whether rows of n elements, size bytes each, have a stride below 0 or reach further
// than any memory: byte offsets within 2^60 are what the kernels and checks hold.
bool far(int B, int64_t sb, int L, int64_t sl, int64_t n, size_t size) {
  return sb < 0 || sl < 0 ||
         ((double)(B - 1) * sb + (double)(L - 1) * sl + n) * size > (double)((int64_t)1 << 60);
}

}  // namespace
}  // namespace specv

extern "C" {

specv_status_t specv_fp4_quantize(const void* x, specv_dtype_t dtype, int rows, int D, uint8_t* q,
                                  uint8_t* scale, hipStream_t stream) {
  using namespace specv;
  if (rows < 1 || D < 1 || D % SPECV_FP4_BLOCK != 0 || !known(dtype)) return SPECV_EINVAL;
  if (D > SPECV_MAX_D || !fp4_quantize_fits(rows, D)) return SPECV_EUNSUPPORTED;
  if (!x || !q || !scale || misaligned(x, 16) || misaligned(q, 4)) return SPECV_EINVAL;
  const size_t n = (size_t)rows * D;
  const Span in[1] = {{x, n * size_of(dtype)}}, o[2] = {{q, n / 2}, {scale, n / SPECV_FP4_BLOCK}};
  if (clash(o, in)) return SPECV_EINVAL;
  return status(launch_fp4_quantize(x, dtype == SPECV_BF16, rows, D, q, scale, stream));
}

size_t specv_fp4_lm_head_packed_weight_bytes(int V, int D) {
  if (specv::check_head_sizes(1, D, V) != SPECV_OK) return 0;
  return specv::fp4_packed_bytes(V, D);
}

specv_status_t specv_fp4_lm_head_pack_weight(const uint8_t* q, const uint8_t* scale,
                                             void* packed_weight, int V, int D,
                                             hipStream_t stream) {
  using namespace specv;
  const specv_status_t st = check_head_sizes(1, D, V);
  if (st != SPECV_OK) return st;
  if (!q || !scale || !packed_weight || misaligned(q, 16) || misaligned(packed_weight, 16))
    return SPECV_EINVAL;
  const size_t n = (size_t)V * D;
  const Span in[2] = {{q, n / 2}, {scale, n / SPECV_FP4_BLOCK}};
  const Span o[1] = {{packed_weight, fp4_packed_bytes(V, D)}};
  if (clash(o, in)) return SPECV_EINVAL;
  return status(launch_fp4_pack(q, scale, packed_weight, V, D, stream));
}

specv_status_t specv_fp4_lm_head(const uint8_t* hidden, specv_hidden_t hidden_type,
                                 const uint8_t* hidden_scale, const void* packed_weight, int M,
                                 int D, int V, void* logits, specv_dtype_t out_dtype,
                                 hipStream_t stream) {
  using namespace specv;
  const specv_status_t st = check_head_sizes(M, D, V);
  if (st != SPECV_OK) return st;
  if (!known(out_dtype) || (hidden_type != SPECV_HIDDEN_E4M3 && hidden_type != SPECV_HIDDEN_E2M1))
    return SPECV_EINVAL;
  if (!hidden || !hidden_scale || !packed_weight || !logits) return SPECV_EINVAL;
  if (misaligned(hidden, 16) || misaligned(packed_weight, 16) ||
      misaligned(logits, size_of(out_dtype)))
    return SPECV_EINVAL;
  const bool h8 = hidden_type == SPECV_HIDDEN_E4M3;
  const size_t n = (size_t)M * D;
  const Span in[3] = {{hidden, h8 ? n : n / 2}, {hidden_scale, h8 ? n / kRun : n / SPECV_FP4_BLOCK},
                      {packed_weight, fp4_packed_bytes(V, D)}};
  const Span o[1] = {{logits, (size_t)M * V * size_of(out_dtype)}};
  if (clash(o, in)) return SPECV_EINVAL;
  return status(launch_fp4_head(hidden, h8, hidden_scale, packed_weight, M, D, V, logits,
                                out_dtype == SPECV_BF16, stream));
}

size_t specv_filter_workspace_bytes(int B, int L, int V, specv_dtype_t dtype) {
  if (specv::check_filter_sizes(B, L, V, dtype) != SPECV_OK) return 0;
  return specv::filter_workspace_bytes(B, L, V, dtype == SPECV_BF16);
}

specv_status_t specv_filter(const void* logits, int64_t stride_b, int64_t stride_l,
                            specv_dtype_t dtype, int B, int L, int V,
                            const specv_filters_t* filters, const float* u, int64_t u_stride_b,
                            int64_t u_stride_l, int32_t* out_tokens, int64_t token_stride_b,
                            int64_t token_stride_l, void* probs, int64_t probs_stride_b,
                            int64_t probs_stride_l, specv_dtype_t probs_dtype, void* workspace,
                            size_t workspace_bytes, hipStream_t stream) {
  using namespace specv;
  const specv_status_t st = check_filter_sizes(B, L, V, dtype);
  if (st != SPECV_OK) return st;
  if (!logits || !filters || (!out_tokens && !probs) || (out_tokens && !u)) return SPECV_EINVAL;
  if (probs && !known(probs_dtype)) return SPECV_EINVAL;
  const specv_filters_t& f = *filters;
  if (!f.temperature_array && !(f.temperature >= 0.0f && std::isfinite(f.temperature)))
    return SPECV_EINVAL;
  if (!f.top_k_array && f.top_k < 0) return SPECV_EINVAL;
  if (!f.top_p_array && !(f.top_p > 0.0f && f.top_p <= 1.0f)) return SPECV_EINVAL;
  if (!f.min_p_array && !(f.min_p >= 0.0f && f.min_p <= 1.0f)) return SPECV_EINVAL;
  const size_t zs = size_of(dtype), ps = probs ? size_of(probs_dtype) : 4;
  if (misaligned(logits, zs) || misaligned(u, 4) || misaligned(out_tokens, 4) ||
      misaligned(probs, ps) || misaligned(f.temperature_array, 4) || misaligned(f.top_k_array, 4) ||
      misaligned(f.top_p_array, 4) || misaligned(f.min_p_array, 4))
    return SPECV_EINVAL;
  if (far(B, stride_b, L, stride_l, V, zs) ||
      (out_tokens && (far(B, u_stride_b, L, u_stride_l, 1, 4) ||
                      far(B, token_stride_b, L, token_stride_l, 1, 4))) ||
      (probs && far(B, probs_stride_b, L, probs_stride_l, V, ps)))
    return SPECV_EINVAL;
  const Rows z = {logits, stride_b * zs, stride_l * zs, B, L, V * zs};
  const Rows ur = {out_tokens ? u : nullptr, (size_t)u_stride_b * 4, (size_t)u_stride_l * 4, B, L, 4};
  const Rows t = {out_tokens, (size_t)token_stride_b * 4, (size_t)token_stride_l * 4, B, L, 4};
  const Rows p = {probs, probs_stride_b * ps, probs_stride_l * ps, B, L, V * ps};
  auto array = [](const void* at, size_t n) { return Rows{at, 0, 0, 1, 1, n}; };
  const Rows params[4] = {array(f.temperature_array, (size_t)B * 4), array(f.top_k_array, (size_t)B * 4),
                          array(f.top_p_array, (size_t)B * 4), array(f.min_p_array, (size_t)B * 4)};
  if (self_overlap(t) || self_overlap(p) || rows_overlap(t, p)) return SPECV_EINVAL;
  for (const Rows* o : {&t, &p}) {
    if (rows_overlap(*o, z) || rows_overlap(*o, ur)) return SPECV_EINVAL;
    for (const Rows& r : params)
      if (rows_overlap(*o, r)) return SPECV_EINVAL;
  }
  const size_t need = filter_workspace_bytes(B, L, V, dtype == SPECV_BF16);
  if (need > 0 && (!workspace || misaligned(workspace, 16) || workspace_bytes < need))
    return SPECV_EWORKSPACE;
  const Rows ws = array(workspace, need);
  for (const Rows* r : {&z, &ur, &t, &p, &params[0], &params[1], &params[2], &params[3]})
    if (rows_overlap(ws, *r)) return SPECV_EINVAL;
  return status(launch_filter(logits, stride_b, stride_l, dtype == SPECV_BF16, B, L, V, f, u,
                              u_stride_b, u_stride_l, out_tokens, token_stride_b, token_stride_l,
                              probs, probs_stride_b, probs_stride_l, probs && probs_dtype == SPECV_BF16,
                              workspace, stream));
}

int specv_draft_version(void) { return 100; }

}  // extern "C"
