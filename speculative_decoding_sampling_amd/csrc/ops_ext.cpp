// Python binding of libspecverify_ops (module _ops_native): argument checks,
// output allocation and the library call.
//
// The operators take a few microseconds on the GPU; marshalled through ctypes
// a call costs the host 9 to 14 us, here 4.5 to 6.  Arguments are positional and
// already in the order of the Python functions in ops.py, which document them;
// the last one is the HIP stream.  A library error comes back as its status
// code, an argument error is raised.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/core/DeviceGuard.h>

#include <initializer_list>

#include "specverify_ops.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Refused {};                       // a Python exception is set

template <typename... A>
[[noreturn]] void refuse(PyObject* type, const char* fmt, A... a) {
  PyErr_Format(type, fmt, a...);
  throw Refused{};
}

const char* type_name(ScalarType t) { return c10::toString(t); }

// A tensor argument, or none.
const Tensor* maybe(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a torch.Tensor", name);
  return &THPVariable_Unpack(o);
}
const Tensor& tensor(PyObject* o, const char* name) {
  const Tensor* t = maybe(o, name);
  if (!t) refuse(PyExc_TypeError, "%s must be a torch.Tensor", name);
  return *t;
}
// A GPU tensor with lo to hi dimensions.
const Tensor& gpu(PyObject* o, const char* name, int lo, int hi) {
  const Tensor& t = tensor(o, name);
  if (!t.is_cuda() || t.dim() < lo || t.dim() > hi)
    refuse(PyExc_ValueError, "%s must be a GPU tensor of %d to %d dimensions", name, lo, hi);
  return t;
}

void check_device(const Tensor& t, const char* name, c10::Device dev) {
  if (t.device() != dev)
    refuse(PyExc_ValueError, "%s is on %s, expected %s", name, t.device().str().c_str(),
           dev.str().c_str());
}
void check_shape(const Tensor& t, const char* name, at::IntArrayRef shape) {
  if (t.sizes() != shape) {
    std::string got, want;
    for (int64_t n : t.sizes()) got += std::to_string(n) + ",";
    for (int64_t n : shape) want += std::to_string(n) + ",";
    refuse(PyExc_ValueError, "%s has shape (%s), expected (%s)", name, got.c_str(), want.c_str());
  }
}
const Tensor& match(const Tensor& t, const char* name, ScalarType type, at::IntArrayRef shape,
                    c10::Device dev) {
  check_device(t, name, dev);
  if (t.scalar_type() != type)
    refuse(PyExc_TypeError, "%s must be %s, got %s", name, type_name(type),
           type_name(t.scalar_type()));
  check_shape(t, name, shape);
  if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
  return t;
}
// A new tensor, straight from the allocator: the dispatcher takes a third of at::empty,
// and a call makes up to six (two: 5.1 -> 4.6 us a call).
Tensor fresh(ScalarType type, at::IntArrayRef shape, c10::Device dev) {
  return Tensor(at::detail::empty_cuda(shape, type, dev, std::nullopt));
}
// The argument where it is given, a new tensor otherwise.
Tensor output(PyObject* o, const char* name, ScalarType type, at::IntArrayRef shape,
              c10::Device dev) {
  if (const Tensor* t = maybe(o, name)) return match(*t, name, type, shape, dev);
  return fresh(type, shape, dev);
}

specv_dtype_t value_code(const Tensor& t, const char* name) {
  if (t.scalar_type() == ScalarType::BFloat16) return SPECV_BF16;
  if (t.scalar_type() == ScalarType::Float) return SPECV_F32;
  refuse(PyExc_TypeError, "%s must be bfloat16 or float32, got %s", name,
         type_name(t.scalar_type()));
}

void* ptr(const Tensor& t) { return t.numel() ? t.data_ptr() : nullptr; }
void* ptr(const Tensor* t) { return t ? ptr(*t) : nullptr; }
template <typename T>
T* as(void* p) { return static_cast<T*>(p); }

double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{};
  return v;
}
int integer(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{};
  if (v != (int)v) refuse(PyExc_ValueError, "%ld is out of range", v);
  return (int)v;
}
hipStream_t stream_of(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw Refused{};
  return static_cast<hipStream_t>(p);
}

at::DimVector with_last(const Tensor& t, int64_t last) {
  at::DimVector s(t.sizes().begin(), t.sizes().end());
  s.back() = last;
  return s;
}

// int arguments of the C ABI
int dim(int64_t n, const char* name) {
  if (n > 0x7fffffff) refuse(PyExc_ValueError, "%s is too large", name);
  return (int)n;
}

PyObject* tuple(std::initializer_list<Tensor> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (!r) throw Refused{};
  Py_ssize_t i = 0;
  for (const Tensor& t : ts) PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(t));
  return r;
}

// The library call on the tensors' device, without the interpreter's lock;
// its status where it is an error, else the outputs.
template <typename F>
PyObject* run(c10::Device dev, F call, std::initializer_list<Tensor> outs) {
  specv_status_t st;
  {
    const c10::DeviceGuard guard(dev);
    Py_BEGIN_ALLOW_THREADS
    st = call();
    Py_END_ALLOW_THREADS
  }
  return st == SPECV_OK ? tuple(outs) : PyLong_FromLong(st);
}

// x, residual, weight, post_weight, gate, scale, eps, code, residual_out, out,
// out_scale, stream
PyObject* hidden_norm(PyObject* const* a) {
  const Tensor& x = gpu(a[0], "x", 1, 8);
  const c10::Device dev = x.device();
  const at::IntArrayRef shape = x.sizes();
  const int64_t D = shape.back(), M = D ? x.numel() / D : 0;
  const Tensor &r = tensor(a[1], "residual"), &w = tensor(a[2], "weight");
  const specv_dtype_t xc = value_code(x, "x"), rc = value_code(r, "residual"),
                      wc = value_code(w, "weight");
  match(x, "x", x.scalar_type(), shape, dev);
  match(r, "residual", r.scalar_type(), shape, dev);
  match(w, "weight", w.scalar_type(), {D}, dev);
  const Tensor *pw = maybe(a[3], "post_weight"), *gate = maybe(a[4], "gate");
  if (pw) match(*pw, "post_weight", w.scalar_type(), {D}, dev);
  int64_t rows = 1;
  if (gate) {
    gpu(a[4], "gate", 1, 2);
    if (gate->dim() == 2) {
      rows = gate->size(0);
      match(*gate, "gate", w.scalar_type(), {rows, D}, dev);
      if (rows < 1 || M % rows)
        refuse(PyExc_ValueError, "gate has %ld rows, which do not divide the %ld rows of x",
               (long)rows, (long)M);
    } else {
      match(*gate, "gate", w.scalar_type(), {D}, dev);
    }
  }
  const int code = integer(a[7]);
  const bool fp8 = code == SPECV_OUT_E4M3;
  if (fp8 && D % SPECV_FP8_BLOCK)
    refuse(PyExc_ValueError, "8-bit output needs D a multiple of %d, got %ld", SPECV_FP8_BLOCK,
           (long)D);
  if (!fp8 && a[10] != Py_None) refuse(PyExc_ValueError, "out_scale goes with 8-bit output only");
  const int Mi = dim(M, "the number of rows"), Di = dim(D, "D"), Gi = dim(rows, "gate");
  const float scale = (float)real(a[5]), eps = (float)real(a[6]);
  const hipStream_t stream = stream_of(a[11]);
  const Tensor r_out = output(a[8], "residual_out", r.scalar_type(), shape, dev);
  const Tensor out = output(a[9], "out",
                            fp8 ? ScalarType::Float8_e4m3fn
                                : code == SPECV_OUT_BF16 ? ScalarType::BFloat16 : ScalarType::Float,
                            shape, dev);
  Tensor s;
  if (fp8)
    s = output(a[10], "out_scale", ScalarType::Float8_e8m0fnu, with_last(x, D / SPECV_FP8_BLOCK),
               dev);
  auto call = [&] {
    return specv_hidden_norm(ptr(x), xc, ptr(r), rc, ptr(pw), ptr(gate), Gi, ptr(w), wc, Mi, Di,
                             scale, eps, ptr(r_out), ptr(out), (specv_out_t)code,
                             fp8 ? as<uint8_t>(ptr(s)) : nullptr, stream);
  };
  return fp8 ? run(dev, call, {r_out, out, s}) : run(dev, call, {r_out, out});
}

// x, out, out_scale, stream
PyObject* quantize_fp8(PyObject* const* a) {
  const Tensor& x = gpu(a[0], "x", 1, 8);
  const c10::Device dev = x.device();
  const int64_t D = x.sizes().back();
  const specv_dtype_t xc = value_code(x, "x");
  match(x, "x", x.scalar_type(), x.sizes(), dev);
  if (D < 1 || D % SPECV_FP8_BLOCK)
    refuse(PyExc_ValueError, "the last dimension must be a multiple of %d, got %ld",
           SPECV_FP8_BLOCK, (long)D);
  const int rows = dim(x.numel() / D, "the number of rows"), Di = dim(D, "D");
  const hipStream_t stream = stream_of(a[3]);
  const Tensor q = output(a[1], "out", ScalarType::Float8_e4m3fn, x.sizes(), dev);
  const Tensor s = output(a[2], "out_scale", ScalarType::Float8_e8m0fnu,
                          with_last(x, D / SPECV_FP8_BLOCK), dev);
  return run(dev, [&] {
    return specv_fp8_quantize(ptr(x), xc, rows, Di, as<uint8_t>(ptr(q)), as<uint8_t>(ptr(s)),
                              stream);
  }, {q, s});
}

// weight, scale, stream
PyObject* pack_fp8_lm_head(PyObject* const* a) {
  const Tensor& w = gpu(a[0], "weight", 2, 2);
  const c10::Device dev = w.device();
  const int64_t V = w.size(0), D = w.size(1);
  match(w, "weight", ScalarType::Float8_e4m3fn, {V, D}, dev);
  const int Vi = dim(V, "V"), Di = dim(D, "D");
  const size_t n = specv_fp8_lm_head_packed_weight_bytes(Vi, Di);
  if (n == 0) return PyLong_FromLong(SPECV_EINVAL);
  const Tensor& s = match(tensor(a[1], "scale"), "scale", ScalarType::Float8_e8m0fnu,
                          {V, D / SPECV_FP8_BLOCK}, dev);
  const hipStream_t stream = stream_of(a[2]);
  const Tensor p = fresh(at::kByte, {(int64_t)n}, dev);
  return run(dev, [&] {
    return specv_fp8_lm_head_pack_weight(as<uint8_t>(ptr(w)), as<uint8_t>(ptr(s)), ptr(p), Vi, Di,
                                         stream);
  }, {p});
}

// hidden with its scale and the packed weight of V and D, checked together
struct Head {
  const Tensor &h, &s, &p;
  int M, D, V;
};
Head head_args(PyObject* const* a, int lo, int hi) {
  const Tensor& h = gpu(a[0], "hidden", lo, hi);
  const c10::Device dev = h.device();
  const int V = integer(a[3]), D = integer(a[4]);
  if (h.sizes().back() != D)
    refuse(PyExc_ValueError, "packed weight has D=%d, hidden D=%ld", D, (long)h.sizes().back());
  match(h, "hidden", ScalarType::Float8_e4m3fn, h.sizes(), dev);
  const Tensor& s = match(tensor(a[1], "hidden_scale"), "hidden_scale",
                          ScalarType::Float8_e8m0fnu, with_last(h, D / SPECV_FP8_BLOCK), dev);
  const Tensor& p = match(tensor(a[2], "packed"), "packed", at::kByte,
                          {(int64_t)specv_fp8_lm_head_packed_weight_bytes(V, D)}, dev);
  return {h, s, p, dim(D ? h.numel() / D : 0, "the number of rows"), D, V};
}

// hidden, hidden_scale, packed data, V, D, code, logits, stream
PyObject* fp8_lm_head(PyObject* const* a) {
  const Head n = head_args(a, 1, 8);
  const c10::Device dev = n.h.device();
  const specv_dtype_t code = (specv_dtype_t)integer(a[5]);
  const hipStream_t stream = stream_of(a[7]);
  const Tensor z = output(a[6], "logits",
                          code == SPECV_BF16 ? ScalarType::BFloat16 : ScalarType::Float,
                          with_last(n.h, n.V), dev);
  return run(dev, [&] {
    return specv_fp8_lm_head(as<uint8_t>(ptr(n.h)), as<uint8_t>(ptr(n.s)), ptr(n.p), n.M, n.D, n.V,
                             ptr(z), code, stream);
  }, {z});
}

// What both verifications take besides their distributions.
struct Round {
  const Tensor &tokens, &len, &u, &uf;
};
Round round_args(PyObject* const* a, int64_t B, int64_t K, c10::Device dev) {
  return {match(tensor(a[0], "draft_tokens"), "draft_tokens", at::kInt, {B, K}, dev),
          match(tensor(a[1], "draft_len"), "draft_len", at::kInt, {B}, dev),
          match(tensor(a[2], "u"), "u", at::kFloat, {B, K}, dev),
          match(tensor(a[3], "u_final"), "u_final", at::kFloat, {B}, dev)};
}
struct Outputs {
  Tensor tokens, n, alpha, mass, stop, path;
  Outputs(PyObject* o_tokens, PyObject* o_n, bool debug, int64_t B, int64_t K, c10::Device dev) {
    tokens = output(o_tokens, "out_tokens", at::kInt, {B, K + 1}, dev);
    n = output(o_n, "n_emitted", at::kInt, {B}, dev);
    if (!debug) return;
    alpha = fresh(at::kFloat, {B, K}, dev);
    mass = fresh(at::kDouble, {B}, dev);
    stop = fresh(at::kInt, {B}, dev);
    path = fresh(at::kInt, {B}, dev);
  }
  void* opt(const Tensor& t) const { return t.defined() ? ptr(t) : nullptr; }
};

const Tensor& workspace_arg(const Tensor& t, c10::Device dev) {
  check_device(t, "workspace", dev);
  if (!t.is_contiguous()) refuse(PyExc_ValueError, "workspace must be contiguous");
  return t;
}

// hidden, hidden_scale, packed data, V, D, draft_logits, draft_tokens,
// draft_len, u, u_final, temperature, eos_id, top_k, top_p, target_logits,
// out_tokens, n_emitted, workspace, debug, stream
PyObject* verify_fp8_lm_head(PyObject* const* a) {
  const Head n = head_args(a, 3, 3);
  const c10::Device dev = n.h.device();
  const int64_t B = n.h.size(0), K = n.h.size(1) - 1;
  const Tensor& d = match(tensor(a[5], "draft_logits"), "draft_logits", ScalarType::BFloat16,
                          {B, K, n.V}, dev);
  const Round r = round_args(a + 6, B, K, dev);
  const float T = (float)real(a[10]), top_p = (float)real(a[13]);
  const int eos = integer(a[11]), top_k = integer(a[12]);
  const bool debug = PyObject_IsTrue(a[18]);
  const hipStream_t stream = stream_of(a[19]);
  const Tensor z = output(a[14], "target_logits", ScalarType::BFloat16, {B, K + 1, n.V}, dev);
  const Outputs o(a[15], a[16], debug, B, K, dev);
  const Tensor& ws = workspace_arg(tensor(a[17], "workspace"), dev);
  auto call = [&] {
    return specv_verify_fp8_lm_head(
        as<uint8_t>(ptr(n.h)), as<uint8_t>(ptr(n.s)), ptr(n.p), ptr(d), as<int32_t>(ptr(r.tokens)),
        as<int32_t>(ptr(r.len)), as<float>(ptr(r.u)), as<float>(ptr(r.uf)), (int)B, (int)K, n.V,
        n.D, T, top_k, top_p, eos, ptr(z), as<int32_t>(ptr(o.tokens)), as<int32_t>(ptr(o.n)),
        ptr(ws), ws.nbytes(), stream, as<float>(o.opt(o.alpha)), as<double>(o.opt(o.mass)),
        as<int32_t>(o.opt(o.stop)), as<int32_t>(o.opt(o.path)));
  };
  return debug ? run(dev, call, {z, o.tokens, o.n, o.alpha, o.mass, o.stop, o.path})
               : run(dev, call, {z, o.tokens, o.n});
}

// Strides of a probability tensor [B, k, V] whose rows are contiguous.
void row_strides(const Tensor& t, const char* name, at::IntArrayRef shape, c10::Device dev,
                 int64_t& sb, int64_t& sk) {
  check_device(t, name, dev);
  check_shape(t, name, shape);
  if (t.stride(2) != 1 && shape[2] > 1 && t.numel())
    refuse(PyExc_ValueError, "the rows of %s must be contiguous", name);
  sb = t.stride(0);
  sk = t.stride(1);
}

// target_probs, draft_probs, draft_tokens, draft_len, u, u_final, eos_id,
// out_tokens, n_emitted, workspace, debug, stream
PyObject* verify_probs(PyObject* const* a) {
  const Tensor& t = gpu(a[0], "target_probs", 3, 3);
  const c10::Device dev = t.device();
  const int64_t B = t.size(0), K = t.size(1) - 1, V = t.size(2);
  const specv_dtype_t code = value_code(t, "target_probs");
  int64_t tsb = 0, tsk = 0, dsb = 0, dsk = 0;
  row_strides(t, "target_probs", {B, K + 1, V}, dev, tsb, tsk);
  const Tensor* d = maybe(a[1], "draft_probs");
  if (d) {
    if (d->dim() != 3) refuse(PyExc_ValueError, "draft_probs must have 3 dimensions");
    row_strides(*d, "draft_probs", {B, K, V}, dev, dsb, dsk);
    if (d->scalar_type() != t.scalar_type())
      refuse(PyExc_TypeError, "draft_probs must be %s, got %s", type_name(t.scalar_type()),
             type_name(d->scalar_type()));
  }
  const Round r = round_args(a + 2, B, K, dev);
  const int Bi = dim(B, "B"), Ki = dim(K, "K"), Vi = dim(V, "V"), eos = integer(a[6]);
  const bool debug = PyObject_IsTrue(a[10]);
  const hipStream_t stream = stream_of(a[11]);
  const Outputs o(a[7], a[8], debug, B, K, dev);
  const Tensor* given = maybe(a[9], "workspace");
  Tensor ws;
  if (given) {
    ws = workspace_arg(*given, dev);
  } else if (const size_t n = specv_verify_probs_workspace_bytes(Bi, Ki, Vi)) {
    ws = fresh(at::kByte, {(int64_t)n}, dev);
  }
  auto call = [&] {
    return specv_verify_probs(
        ptr(t), tsb, tsk, ptr(d), dsb, dsk, code, as<int32_t>(ptr(r.tokens)),
        as<int32_t>(ptr(r.len)), as<float>(ptr(r.u)), as<float>(ptr(r.uf)), Bi, Ki, Vi, eos,
        as<int32_t>(ptr(o.tokens)), as<int32_t>(ptr(o.n)), o.opt(ws), ws.defined() ? ws.nbytes() : 0,
        stream, as<float>(o.opt(o.alpha)), as<double>(o.opt(o.mass)), as<int32_t>(o.opt(o.stop)),
        as<int32_t>(o.opt(o.path)));
  };
  return debug ? run(dev, call, {o.tokens, o.n, o.alpha, o.mass, o.stop, o.path})
               : run(dev, call, {o.tokens, o.n});
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)),
          METH_FASTCALL, nullptr};
}

PyMethodDef kMethods[] = {
    method<hidden_norm, 12>("hidden_norm"),
    method<quantize_fp8, 4>("quantize_fp8"),
    method<pack_fp8_lm_head, 3>("pack_fp8_lm_head"),
    method<fp8_lm_head, 8>("fp8_lm_head"),
    method<verify_fp8_lm_head, 20>("verify_fp8_lm_head"),
    method<verify_probs, 12>("verify_probs"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_ops_native", nullptr, -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__ops_native() { return PyModule_Create(&kModule); }
