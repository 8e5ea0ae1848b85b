// What the Python bindings of the operators share (host C++ against torch's
// headers): argument checks, output allocation, the call itself and the entry
// points.  Included once by a module, whose own namespace keeps it.
#pragma once

#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/core/DeviceGuard.h>

#include <initializer_list>

#include "specverify.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Refused {};                       // a Python exception is set

template <typename... A>
[[noreturn]] void refuse(PyObject* type, const char* fmt, A... a) {
  PyErr_Format(type, fmt, a...);
  throw Refused{};
}

inline const char* type_name(ScalarType t) { return c10::toString(t); }

// A tensor argument, or none.
inline const Tensor* maybe(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a torch.Tensor", name);
  return &THPVariable_Unpack(o);
}
inline const Tensor& tensor(PyObject* o, const char* name) {
  const Tensor* t = maybe(o, name);
  if (!t) refuse(PyExc_TypeError, "%s must be a torch.Tensor", name);
  return *t;
}
// A GPU tensor with lo to hi dimensions.
inline const Tensor& gpu(PyObject* o, const char* name, int lo, int hi) {
  const Tensor& t = tensor(o, name);
  if (!t.is_cuda() || t.dim() < lo || t.dim() > hi)
    refuse(PyExc_ValueError, "%s must be a GPU tensor of %d to %d dimensions", name, lo, hi);
  return t;
}

inline void check_device(const Tensor& t, const char* name, c10::Device dev) {
  if (t.device() != dev)
    refuse(PyExc_ValueError, "%s is on %s, expected %s", name, t.device().str().c_str(),
           dev.str().c_str());
}
inline void check_shape(const Tensor& t, const char* name, at::IntArrayRef shape) {
  if (t.sizes() != shape) {
    std::string got, want;
    for (int64_t n : t.sizes()) got += std::to_string(n) + ",";
    for (int64_t n : shape) want += std::to_string(n) + ",";
    refuse(PyExc_ValueError, "%s has shape (%s), expected (%s)", name, got.c_str(), want.c_str());
  }
}
inline const Tensor& match(const Tensor& t, const char* name, ScalarType type, at::IntArrayRef shape,
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
inline Tensor fresh(ScalarType type, at::IntArrayRef shape, c10::Device dev) {
  return Tensor(at::detail::empty_cuda(shape, type, dev, std::nullopt));
}
// The argument where it is given, a new tensor otherwise.
inline Tensor output(PyObject* o, const char* name, ScalarType type, at::IntArrayRef shape,
              c10::Device dev) {
  if (const Tensor* t = maybe(o, name)) return match(*t, name, type, shape, dev);
  return fresh(type, shape, dev);
}

inline specv_dtype_t value_code(const Tensor& t, const char* name) {
  if (t.scalar_type() == ScalarType::BFloat16) return SPECV_BF16;
  if (t.scalar_type() == ScalarType::Float) return SPECV_F32;
  refuse(PyExc_TypeError, "%s must be bfloat16 or float32, got %s", name,
         type_name(t.scalar_type()));
}

inline void* ptr(const Tensor& t) { return t.numel() ? t.data_ptr() : nullptr; }
inline void* ptr(const Tensor* t) { return t ? ptr(*t) : nullptr; }
template <typename T>
T* as(void* p) { return static_cast<T*>(p); }

inline double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{};
  return v;
}
inline int integer(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{};
  if (v != (int)v) refuse(PyExc_ValueError, "%ld is out of range", v);
  return (int)v;
}
inline hipStream_t stream_of(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw Refused{};
  return static_cast<hipStream_t>(p);
}

inline at::DimVector with_last(const Tensor& t, int64_t last) {
  at::DimVector s(t.sizes().begin(), t.sizes().end());
  s.back() = last;
  return s;
}

// int arguments of the C ABI
inline int dim(int64_t n, const char* name) {
  if (n > 0x7fffffff) refuse(PyExc_ValueError, "%s is too large", name);
  return (int)n;
}

inline PyObject* tuple(std::initializer_list<Tensor> ts) {
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

inline const Tensor& workspace_arg(const Tensor& t, c10::Device dev) {
  check_device(t, "workspace", dev);
  if (!t.is_contiguous()) refuse(PyExc_ValueError, "workspace must be contiguous");
  return t;
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

}  // namespace
