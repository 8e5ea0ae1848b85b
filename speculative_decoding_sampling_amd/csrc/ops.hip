// C ABI of libspecverify_ops: argument checks and launches on the caller's
// stream.  The declarations and their contract live in
// include/specverify_ops.h.
#include "specverify_ops.h"

#include "abi_checks.h"

#include <cmath>
#include <cstdint>

namespace specv {
bool probs_fits(int B, int V);
size_t probs_workspace_bytes(int B, int V);
hipError_t launch_verify_probs(bool bf16, const void* tgt, long long tsb, long long tsk,
                               const void* dft, long long dsb, long long dsk, const int* tokens,
                               const int* draft_len, const float* u, const float* u_final, int B,
                               int K, int V, int eos_id, int* out_tokens, int* n_emitted,
                               void* workspace, float* alpha_out, double* rmass_out, int* stop_out,
                               int* path_out, hipStream_t stream);
bool hidden_norm_fits(int M, int D);
hipError_t launch_hidden_norm(const void* x, bool xb, const void* r, bool rb, const void* w1,
                              const void* gate, int gate_rows, const void* w2, bool wb, int M,
                              int D, float scale, float eps, void* r_out, void* out, int out_dtype,
                              uint8_t* out_scale, hipStream_t stream);
bool fp8_quantize_fits(int rows, int D);
hipError_t launch_fp8_quantize(const void* x, bool bf16, int rows, int D, uint8_t* q,
                               uint8_t* scale, hipStream_t stream);
size_t fp8_packed_bytes(int V, int D);
hipError_t launch_fp8_pack(const uint8_t* q, const uint8_t* scale, void* packed, int V, int D,
                           hipStream_t stream);
bool fp8_head_fits(int M, int V);
bool fp8_pack_fits(int V, int D);
hipError_t launch_fp8_head(const uint8_t* hidden, const uint8_t* hscale, const void* packed, int M,
                           int D, int V, void* logits, bool bf16, hipStream_t stream);

namespace {

specv_status_t check_head_sizes(int M, int D, int V) {
  if (M < 1 || V < 1 || D < 1 || D % SPECV_FP8_BLOCK != 0) return SPECV_EINVAL;
  if (V > SPECV_MAX_V || D > SPECV_MAX_D) return SPECV_EUNSUPPORTED;
  if (!fp8_head_fits(M, V) || !fp8_pack_fits(V, D)) return SPECV_EUNSUPPORTED;
  return SPECV_OK;
}

specv_status_t check_probs_sizes(int B, int K, int V) {
  if (B < 1 || K < 0 || K > SPECV_MAX_K || V < 1) return SPECV_EINVAL;
  if (V > SPECV_MAX_V) return SPECV_EUNSUPPORTED;
  if (!probs_fits(B, V)) return SPECV_EUNSUPPORTED;
  return SPECV_OK;
}

}  // namespace
}  // namespace specv

extern "C" {

specv_status_t specv_hidden_norm(const void* x, specv_dtype_t x_dtype, const void* residual,
                                 specv_dtype_t residual_dtype, const void* post_weight,
                                 const void* gate, int gate_rows, const void* weight,
                                 specv_dtype_t weight_dtype, int M, int D, float scale, float eps,
                                 void* residual_out, void* out, specv_out_t out_dtype,
                                 uint8_t* out_scale, hipStream_t stream) {
  using namespace specv;
  if (M < 1 || D < 1) return SPECV_EINVAL;
  if (D > SPECV_MAX_D || !hidden_norm_fits(M, D)) return SPECV_EUNSUPPORTED;
  if (!known(x_dtype) || !known(residual_dtype) || !known(weight_dtype)) return SPECV_EINVAL;
  const bool fp8 = out_dtype == SPECV_OUT_E4M3;
  if (!fp8 && out_dtype != SPECV_OUT_F32 && out_dtype != SPECV_OUT_BF16) return SPECV_EINVAL;
  if (fp8 && (D % SPECV_FP8_BLOCK != 0 || !out_scale)) return SPECV_EINVAL;
  if (!std::isfinite(scale) || !std::isfinite(eps) || !(eps > 0.0f)) return SPECV_EINVAL;
  if (!x || !residual || !weight || !residual_out || !out) return SPECV_EINVAL;
  if (gate && (gate_rows < 1 || M % gate_rows != 0)) return SPECV_EINVAL;
  const size_t xs = size_of(x_dtype), rs = size_of(residual_dtype), ws = size_of(weight_dtype);
  const size_t os = fp8 ? 1 : out_dtype == SPECV_OUT_BF16 ? 2 : 4;
  if (misaligned(x, xs) || misaligned(residual, rs) || misaligned(residual_out, rs) ||
      misaligned(weight, ws) || misaligned(post_weight, ws) || misaligned(gate, ws) ||
      misaligned(out, fp8 ? 8 : os))
    return SPECV_EINVAL;
  // every row is read whole before any of it is written, so an output may be
  // the very array it replaces; anything else that overlaps is an error
  const size_t n = (size_t)M * D;
  const Span in[5] = {{x, n * xs}, {residual, n * rs}, {weight, D * ws}, {post_weight, D * ws},
                      {gate, gate ? (size_t)gate_rows * D * ws : 0}};
  const Span o[3] = {{residual_out, n * rs}, {out, n * os}, {fp8 ? out_scale : nullptr, n / SPECV_FP8_BLOCK}};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < 5; ++j) {
      const bool same = (i == 0 && j == 1 && residual_out == residual) ||
                        (i == 1 && j == 0 && out == x && os == xs);
      if (!same && overlap(o[i], in[j])) return SPECV_EINVAL;
    }
    for (int j = 0; j < i; ++j)
      if (overlap(o[i], o[j])) return SPECV_EINVAL;
  }
  return status(launch_hidden_norm(x, x_dtype == SPECV_BF16, residual, residual_dtype == SPECV_BF16,
                                   post_weight, gate, gate_rows, weight,
                                   weight_dtype == SPECV_BF16, M, D, scale, eps, residual_out, out,
                                   (int)out_dtype, out_scale, stream));
}

specv_status_t specv_fp8_quantize(const void* x, specv_dtype_t dtype, int rows, int D, uint8_t* q,
                                  uint8_t* scale, hipStream_t stream) {
  using namespace specv;
  if (rows < 1 || D < 1 || D % SPECV_FP8_BLOCK != 0 || !known(dtype)) return SPECV_EINVAL;
  if (D > SPECV_MAX_D || !fp8_quantize_fits(rows, D)) return SPECV_EUNSUPPORTED;
  if (!x || !q || !scale || misaligned(x, 16) || misaligned(q, 8)) return SPECV_EINVAL;
  const size_t n = (size_t)rows * D;
  const Span in = {x, n * size_of(dtype)}, o = {q, n}, s = {scale, n / SPECV_FP8_BLOCK};
  if (overlap(in, o) || overlap(in, s) || overlap(o, s)) return SPECV_EINVAL;
  return status(launch_fp8_quantize(x, dtype == SPECV_BF16, rows, D, q, scale, stream));
}

size_t specv_fp8_lm_head_packed_weight_bytes(int V, int D) {
  if (specv::check_head_sizes(1, D, V) != SPECV_OK) return 0;
  return specv::fp8_packed_bytes(V, D);
}

specv_status_t specv_fp8_lm_head_pack_weight(const uint8_t* q, const uint8_t* scale,
                                             void* packed_weight, int V, int D,
                                             hipStream_t stream) {
  using namespace specv;
  const specv_status_t st = check_head_sizes(1, D, V);
  if (st != SPECV_OK) return st;
  if (!q || !scale || !packed_weight || misaligned(q, 16) || misaligned(packed_weight, 16))
    return SPECV_EINVAL;
  const size_t n = (size_t)V * D;
  const Span o = {packed_weight, fp8_packed_bytes(V, D)};
  if (overlap(o, {q, n}) || overlap(o, {scale, n / SPECV_FP8_BLOCK})) return SPECV_EINVAL;
  return status(launch_fp8_pack(q, scale, packed_weight, V, D, stream));
}

specv_status_t specv_fp8_lm_head(const uint8_t* hidden, const uint8_t* hidden_scale,
                                 const void* packed_weight, int M, int D, int V, void* logits,
                                 specv_dtype_t out_dtype, hipStream_t stream) {
  using namespace specv;
  const specv_status_t st = check_head_sizes(M, D, V);
  if (st != SPECV_OK) return st;
  if (!known(out_dtype)) return SPECV_EINVAL;
  if (!hidden || !hidden_scale || !packed_weight || !logits) return SPECV_EINVAL;
  if (misaligned(hidden, 16) || misaligned(packed_weight, 16) ||
      misaligned(logits, size_of(out_dtype)))
    return SPECV_EINVAL;
  const size_t n = (size_t)M * D;
  const Span o = {logits, (size_t)M * V * size_of(out_dtype)};
  if (overlap(o, {hidden, n}) || overlap(o, {hidden_scale, n / SPECV_FP8_BLOCK}) ||
      overlap(o, {packed_weight, fp8_packed_bytes(V, D)}))
    return SPECV_EINVAL;
  return status(launch_fp8_head(hidden, hidden_scale, packed_weight, M, D, V, logits,
                                out_dtype == SPECV_BF16, stream));
}

size_t specv_verify_fp8_lm_head_workspace_bytes(int B, int K, int V, int D, int top_k,
                                                float top_p) {
  const size_t n = specv_workspace_bytes(B, K, V, SPECV_BF16, top_k, top_p);
  if (n == 0 || (long long)B * (K + 1) > 0x7fffffff ||
      specv::check_head_sizes(B * (K + 1), D, V) != SPECV_OK)
    return 0;
  return n;
}

specv_status_t specv_verify_fp8_lm_head(
    const uint8_t* hidden, const uint8_t* hidden_scale, const void* packed_weight,
    const void* draft_logits, const int32_t* draft_tokens, const int32_t* draft_len,
    const float* u, const float* u_final, int B, int K, int V, int D, float temperature, int top_k,
    float top_p, int eos_id, void* target_logits, int32_t* out_tokens, int32_t* n_emitted,
    void* workspace, size_t workspace_bytes, hipStream_t stream, float* accept_prob,
    double* residual_mass, int32_t* stop_pos, int32_t* path) {
  using namespace specv;
  if (B < 1 || K < 0 || K > SPECV_MAX_K) return SPECV_EINVAL;
  if ((long long)B * (K + 1) > 0x7fffffff) return SPECV_EUNSUPPORTED;
  const specv_status_t st = check_head_sizes(B * (K + 1), D, V);
  if (st != SPECV_OK) return st;
  // every check of the verification that follows, so that a refused call
  // enqueues nothing
  if (!(temperature > 0.0f) || !std::isfinite(temperature)) return SPECV_EINVAL;
  if (top_k < 0 || !(top_p > 0.0f && top_p <= 1.0f)) return SPECV_EINVAL;
  if (eos_id < -1 || eos_id >= V) return SPECV_EINVAL;
  if (!target_logits || !draft_len || !u_final || !out_tokens || !n_emitted) return SPECV_EINVAL;
  if (K > 0 && (!draft_logits || !draft_tokens || !u)) return SPECV_EINVAL;
  if (misaligned(draft_logits, 2) || misaligned(draft_tokens, 4) || misaligned(draft_len, 4) ||
      misaligned(u, 4) || misaligned(u_final, 4) || misaligned(out_tokens, 4) ||
      misaligned(n_emitted, 4) || misaligned(accept_prob, 4) || misaligned(residual_mass, 8) ||
      misaligned(stop_pos, 4) || misaligned(path, 4))
    return SPECV_EINVAL;
  const size_t need = specv_workspace_bytes(B, K, V, SPECV_BF16, top_k, top_p);
  if (need == 0) return SPECV_EUNSUPPORTED;
  if (!workspace || misaligned(workspace, 16) || workspace_bytes < need) return SPECV_EWORKSPACE;
  // the logits are written before the verification reads its inputs
  const size_t rows = (size_t)B * (K + 1), nk = (size_t)B * K;
  const Span in[8] = {{hidden, rows * D}, {hidden_scale, rows * D / SPECV_FP8_BLOCK},
                      {packed_weight, fp8_packed_bytes(V, D)}, {draft_logits, nk * V * 2},
                      {draft_tokens, nk * 4}, {draft_len, (size_t)B * 4}, {u, nk * 4},
                      {u_final, (size_t)B * 4}};
  const Span o[8] = {{target_logits, rows * V * 2}, {out_tokens, rows * 4},
                     {n_emitted, (size_t)B * 4}, {accept_prob, nk * 4},
                     {residual_mass, (size_t)B * 8}, {stop_pos, (size_t)B * 4},
                     {path, (size_t)B * 4}, {workspace, need}};
  if (clash(o, in)) return SPECV_EINVAL;
  const specv_status_t head = specv_fp8_lm_head(hidden, hidden_scale, packed_weight, B * (K + 1), D,
                                                V, target_logits, SPECV_BF16, stream);
  if (head != SPECV_OK) return head;
  return specv_verify_debug(target_logits, draft_logits, SPECV_BF16, draft_tokens, draft_len, u,
                            u_final, B, K, V, temperature, top_k, top_p, eos_id, out_tokens,
                            n_emitted, workspace, workspace_bytes, stream, accept_prob,
                            residual_mass, stop_pos, path);
}

size_t specv_verify_probs_workspace_bytes(int B, int K, int V) {
  if (specv::check_probs_sizes(B, K, V) != SPECV_OK) return 0;
  return specv::probs_workspace_bytes(B, V);
}

specv_status_t specv_verify_probs(const void* target_probs, int64_t target_stride_b,
                                  int64_t target_stride_k, const void* draft_probs,
                                  int64_t draft_stride_b, int64_t draft_stride_k,
                                  specv_dtype_t dtype, const int32_t* draft_tokens,
                                  const int32_t* draft_len, const float* u, const float* u_final,
                                  int B, int K, int V, int eos_id, int32_t* out_tokens,
                                  int32_t* n_emitted, void* workspace, size_t workspace_bytes,
                                  hipStream_t stream, float* accept_prob, double* residual_mass,
                                  int32_t* stop_pos, int32_t* path) {
  using namespace specv;
  const specv_status_t st = check_probs_sizes(B, K, V);
  if (st != SPECV_OK) return st;
  if (!known(dtype)) return SPECV_EINVAL;
  if (eos_id < -1 || eos_id >= V) return SPECV_EINVAL;
  if (target_stride_b < 0 || target_stride_k < 0 || draft_stride_b < 0 || draft_stride_k < 0)
    return SPECV_EINVAL;
  // the furthest element must index without overflow
  const double far_t = (double)B * target_stride_b + (double)(K + 1) * target_stride_k + V;
  const double far_d = (double)B * draft_stride_b + (double)K * draft_stride_k + V;
  if (far_t > 1.0e18 || (draft_probs && far_d > 1.0e18)) return SPECV_EINVAL;
  if (!target_probs || !draft_len || !u_final || !out_tokens || !n_emitted) return SPECV_EINVAL;
  if (K > 0 && (!draft_tokens || !u)) return SPECV_EINVAL;
  const size_t esz = size_of(dtype);
  if (misaligned(target_probs, esz) || misaligned(draft_probs, esz) ||
      misaligned(draft_tokens, 4) || misaligned(draft_len, 4) || misaligned(u, 4) ||
      misaligned(u_final, 4) || misaligned(out_tokens, 4) || misaligned(n_emitted, 4) ||
      misaligned(accept_prob, 4) || misaligned(residual_mass, 8) || misaligned(stop_pos, 4) ||
      misaligned(path, 4))
    return SPECV_EINVAL;
  const size_t need = probs_workspace_bytes(B, V), nk = (size_t)B * K;
  if (need > 0 && (!workspace || misaligned(workspace, 16) || workspace_bytes < need))
    return SPECV_EWORKSPACE;
  // the waves of a request read its inputs while one of them writes its outputs
  const Span in[4] = {{draft_tokens, nk * 4}, {draft_len, (size_t)B * 4}, {u, nk * 4},
                      {u_final, (size_t)B * 4}};
  const Span o[7] = {{out_tokens, (nk + B) * 4}, {n_emitted, (size_t)B * 4}, {accept_prob, nk * 4},
                     {residual_mass, (size_t)B * 8}, {stop_pos, (size_t)B * 4},
                     {path, (size_t)B * 4}, {workspace, need}};
  if (clash(o, in)) return SPECV_EINVAL;
  const Rows t = {target_probs, target_stride_b * esz, target_stride_k * esz, B, K + 1, V * esz};
  const Rows d = {draft_probs, draft_stride_b * esz, draft_stride_k * esz, B, K, V * esz};
  for (const Span& s : o)
    if (overlaps_rows(s, t) || overlaps_rows(s, d)) return SPECV_EINVAL;
  return status(launch_verify_probs(dtype == SPECV_BF16, target_probs, target_stride_b,
                                    target_stride_k, draft_probs, draft_stride_b, draft_stride_k,
                                    draft_tokens, draft_len, u, u_final, B, K, V, eos_id,
                                    out_tokens, n_emitted, workspace, accept_prob, residual_mass,
                                    stop_pos, path, stream));
}

int specv_ops_version(void) { return 100; }

}  // extern "C"
