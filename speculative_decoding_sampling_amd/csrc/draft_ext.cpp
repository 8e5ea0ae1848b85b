// Python binding of libspecverify_draft (module _draft_native): argument checks,
// output allocation and the library call.  Arguments are positional and already
// in the order of the Python functions in draft.py, which document them; the
// last one is the HIP stream.
#include "ext_common.h"
#include "specverify_draft.h"

namespace {

constexpr int kRun = 128;                // columns of an 8-bit scale and of a product's run

// x, out, out_scale, stream
PyObject* quantize_fp4(PyObject* const* a) {
  const Tensor& x = gpu(a[0], "x", 1, 8);
  const c10::Device dev = x.device();
  const int64_t D = x.sizes().back();
  const specv_dtype_t xc = value_code(x, "x");
  match(x, "x", x.scalar_type(), x.sizes(), dev);
  if (D < 1 || D % SPECV_FP4_BLOCK)
    refuse(PyExc_ValueError, "the last dimension must be a multiple of %d, got %ld",
           SPECV_FP4_BLOCK, (long)D);
  const int rows = dim(x.numel() / D, "the number of rows"), Di = dim(D, "D");
  const hipStream_t stream = stream_of(a[3]);
  const Tensor q = output(a[1], "out", ScalarType::Float4_e2m1fn_x2, with_last(x, D / 2), dev);
  const Tensor s = output(a[2], "out_scale", ScalarType::Float8_e8m0fnu,
                          with_last(x, D / SPECV_FP4_BLOCK), dev);
  return run(dev, [&] {
    return specv_fp4_quantize(ptr(x), xc, rows, Di, as<uint8_t>(ptr(q)), as<uint8_t>(ptr(s)),
                              stream);
  }, {q, s});
}

// weight, scale, stream
PyObject* pack_fp4_lm_head(PyObject* const* a) {
  const Tensor& w = gpu(a[0], "weight", 2, 2);
  const c10::Device dev = w.device();
  const int64_t V = w.size(0), D = 2 * w.size(1);
  match(w, "weight", ScalarType::Float4_e2m1fn_x2, {V, D / 2}, dev);
  const int Vi = dim(V, "V"), Di = dim(D, "D");
  const size_t n = specv_fp4_lm_head_packed_weight_bytes(Vi, Di);
  if (n == 0) return PyLong_FromLong(SPECV_EINVAL);
  const Tensor& s = match(tensor(a[1], "scale"), "scale", ScalarType::Float8_e8m0fnu,
                          {V, D / SPECV_FP4_BLOCK}, dev);
  const hipStream_t stream = stream_of(a[2]);
  const Tensor p = fresh(at::kByte, {(int64_t)n}, dev);
  return run(dev, [&] {
    return specv_fp4_lm_head_pack_weight(as<uint8_t>(ptr(w)), as<uint8_t>(ptr(s)), ptr(p), Vi, Di,
                                         stream);
  }, {p});
}

// hidden, hidden_scale, packed data, V, D, code, logits, stream
PyObject* fp4_lm_head(PyObject* const* a) {
  const Tensor& h = gpu(a[0], "hidden", 1, 8);
  const c10::Device dev = h.device();
  const int V = integer(a[3]), D = integer(a[4]);
  const bool h8 = h.scalar_type() == ScalarType::Float8_e4m3fn;
  if (!h8 && h.scalar_type() != ScalarType::Float4_e2m1fn_x2)
    refuse(PyExc_TypeError, "hidden must be float8_e4m3fn or float4_e2m1fn_x2, got %s",
           type_name(h.scalar_type()));
  const int64_t last = h.sizes().back(), hd = h8 ? last : 2 * last;
  if (hd != D) refuse(PyExc_ValueError, "packed weight has D=%d, hidden D=%ld", D, (long)hd);
  match(h, "hidden", h.scalar_type(), h.sizes(), dev);
  const Tensor& s = match(tensor(a[1], "hidden_scale"), "hidden_scale", ScalarType::Float8_e8m0fnu,
                          with_last(h, D / (h8 ? kRun : SPECV_FP4_BLOCK)), dev);
  const Tensor& p = match(tensor(a[2], "packed"), "packed", at::kByte,
                          {(int64_t)specv_fp4_lm_head_packed_weight_bytes(V, D)}, dev);
  const int M = dim(last ? h.numel() / last : 0, "the number of rows");
  const specv_dtype_t code = (specv_dtype_t)integer(a[5]);
  const hipStream_t stream = stream_of(a[7]);
  const Tensor z = output(a[6], "logits",
                          code == SPECV_BF16 ? ScalarType::BFloat16 : ScalarType::Float,
                          with_last(h, V), dev);
  return run(dev, [&] {
    return specv_fp4_lm_head(as<uint8_t>(ptr(h)), h8 ? SPECV_HIDDEN_E4M3 : SPECV_HIDDEN_E2M1,
                             as<uint8_t>(ptr(s)), ptr(p), M, D, V, ptr(z), code, stream);
  }, {z});
}

// A tensor of the call's rows with free strides: [B, ...] or [B, L, ...].
struct Strided {
  const Tensor* t = nullptr;
  int64_t sb = 0, sl = 0;
};
Strided strided(const Tensor& t, const char* name, ScalarType type, at::IntArrayRef shape, bool two,
                bool rows, c10::Device dev) {
  check_device(t, name, dev);
  if (t.scalar_type() != type)
    refuse(PyExc_TypeError, "%s must be %s, got %s", name, type_name(type),
           type_name(t.scalar_type()));
  check_shape(t, name, shape);
  if (rows && t.numel() && t.sizes().back() > 1 && t.strides().back() != 1)
    refuse(PyExc_ValueError, "the rows of %s must be contiguous", name);
  return {&t, t.stride(0), two ? t.stride(1) : 0};
}

// One parameter of the filters: a number, or a [B] tensor.
template <typename T>
void filter_arg(PyObject* o, const char* name, ScalarType type, int64_t B, c10::Device dev,
                const T*& array, T& value) {
  array = nullptr;
  value = T();
  if (THPVariable_Check(o)) {
    array = as<const T>(ptr(match(THPVariable_Unpack(o), name, type, {B}, dev)));
  } else if constexpr (std::is_same_v<T, float>) {
    value = (float)real(o);
  } else {
    value = integer(o);
  }
}

// logits, temperature, top_k, top_p, min_p, u, out_tokens, probs, probs code (-1:
// none), workspace, stream
PyObject* filter(PyObject* const* a) {
  const Tensor& z = gpu(a[0], "logits", 2, 3);
  const c10::Device dev = z.device();
  const bool two = z.dim() == 3;
  const int64_t B = z.size(0), L = two ? z.size(1) : 1, V = z.sizes().back();
  const specv_dtype_t code = value_code(z, "logits");
  const Strided zs = strided(z, "logits", z.scalar_type(), z.sizes(), two, true, dev);
  const int Bi = dim(B, "B"), Li = dim(L, "L"), Vi = dim(V, "V");
  specv_filters_t f;
  filter_arg(a[1], "temperature", at::kFloat, B, dev, f.temperature_array, f.temperature);
  filter_arg(a[2], "top_k", at::kInt, B, dev, f.top_k_array, f.top_k);
  filter_arg(a[3], "top_p", at::kFloat, B, dev, f.top_p_array, f.top_p);
  filter_arg(a[4], "min_p", at::kFloat, B, dev, f.min_p_array, f.min_p);
  const at::IntArrayRef lead = z.sizes().slice(0, z.dim() - 1);
  const Tensor* u = maybe(a[5], "u");
  Strided us, ts, ps;
  Tensor tokens, probs;
  if (u) {
    us = strided(*u, "u", at::kFloat, lead, two, false, dev);
    const Tensor* given = maybe(a[6], "out_tokens");
    tokens = given ? *given : fresh(at::kInt, lead, dev);
    ts = strided(tokens, "out_tokens", at::kInt, lead, two, false, dev);
  } else if (a[6] != Py_None) {
    refuse(PyExc_ValueError, "out_tokens needs u");
  }
  const int pcode = integer(a[8]);
  if (pcode >= 0) {
    const ScalarType type = pcode == SPECV_BF16 ? ScalarType::BFloat16 : ScalarType::Float;
    const Tensor* given = maybe(a[7], "probs");
    probs = given ? *given : fresh(type, z.sizes(), dev);
    ps = strided(probs, "probs", type, z.sizes(), two, true, dev);
  }
  const hipStream_t stream = stream_of(a[10]);
  const Tensor* given = maybe(a[9], "workspace");
  const Tensor ws = given ? workspace_arg(*given, dev)
                          : fresh(at::kByte, {(int64_t)specv_filter_workspace_bytes(Bi, Li, Vi, code)},
                                  dev);
  auto call = [&] {
    return specv_filter(ptr(z), zs.sb, zs.sl, code, Bi, Li, Vi, &f, u ? as<const float>(ptr(*u)) : nullptr,
                        us.sb, us.sl, ts.t ? as<int32_t>(ptr(tokens)) : nullptr, ts.sb, ts.sl,
                        ps.t ? ptr(probs) : nullptr, ps.sb, ps.sl,
                        ps.t ? (specv_dtype_t)pcode : SPECV_F32, ptr(ws), ws.nbytes(), stream);
  };
  if (ps.t && ts.t) return run(dev, call, {probs, tokens});
  return ps.t ? run(dev, call, {probs}) : run(dev, call, {tokens});
}

PyMethodDef kMethods[] = {
    method<quantize_fp4, 4>("quantize_fp4"),
    method<pack_fp4_lm_head, 3>("pack_fp4_lm_head"),
    method<fp4_lm_head, 8>("fp4_lm_head"),
    method<filter, 11>("filter"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_draft_native", nullptr, -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__draft_native() { return PyModule_Create(&kModule); }
