// What the compiled bindings share: argument checks, new tensors for what is not given, results and errors.
#pragma once

#include <torch/csrc/python_headers.h>

#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/pybind.h>

#include <cmath>
#include <string>

#include "medusa.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Refused {
  PyObject* type;
  std::string text;
};

std::string list_of(at::IntArrayRef s) {
  std::string r = "[";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + "]";
}

// One call: its name, and the device and type its tensors share.
struct Call {
  const char* what;
  c10::Device dev = c10::Device(c10::kCPU);
  ScalarType ty = ScalarType::Undefined;

  [[noreturn]] void refuse(const std::string& text, PyObject* type = PyExc_ValueError) const {
    throw Refused{type, std::string(what) + ": " + text};
  }
  const Tensor& tensor(PyObject* o, const char* name) const {
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor", PyExc_TypeError);
    return THPVariable_Unpack(o);
  }
  // The tensor all others must be like.
  int lead(const Tensor& t, const char* name) {
    ty = t.scalar_type();
    if (ty != ScalarType::BFloat16 && ty != ScalarType::Float)
      refuse(std::string("tensors must be bfloat16 or float32, not ") + c10::toString(ty), PyExc_TypeError);
    if (!t.is_cuda()) refuse(std::string(name) + " must be on a GPU");
    dev = t.device();
    return ty == ScalarType::BFloat16 ? MEDUSA_BF16 : MEDUSA_F32;
  }
  void like(const Tensor& t, const char* name, ScalarType dt) const {
    if (t.device() != dev) refuse(std::string(name) + " must be on the GPU of the other tensors (" + dev.str() + "), not on " + t.device().str());
    if (t.scalar_type() != dt) refuse(std::string(name) + " must be " + c10::toString(dt) + ", not " + c10::toString(t.scalar_type()));
  }
  const Tensor& dense(const Tensor& t, const char* name, ScalarType dt, at::IntArrayRef shape) const {
    like(t, name, dt);
    if (!t.is_contiguous()) refuse(std::string(name) + " must be dense");
    if (t.sizes() != shape) refuse(std::string(name) + " must be " + list_of(shape) + ", not " + list_of(t.sizes()));
    return t;
  }
  // n words of int32, in any dense shape.
  int32_t* words(const Tensor& t, const char* name, int64_t n) const {
    like(t, name, ScalarType::Int);
    if (!t.is_contiguous() || t.numel() != n) refuse(std::string(name) + " must be dense and hold " + std::to_string(n) + " values");
    return static_cast<int32_t*>(t.data_ptr());
  }
  int32_t* words(PyObject* o, const char* name, int64_t n) const { return words(tensor(o, name), name, n); }
  // Elements from one token to the next of t [nl, T, H, d], whose heads are dense and whose layers are T tokens apart.
  int64_t token_stride(const Tensor& t, const char* name, int64_t nl, int64_t T, int64_t H, int64_t d) const {
    const int64_t shape[4] = {nl, T, H, d};
    if (t.sizes() != at::IntArrayRef(shape, 4)) refuse(std::string(name) + " must be " + list_of(at::IntArrayRef(shape, 4)) + ", not " + list_of(t.sizes()));
    const int64_t ld = T > 1 ? t.stride(1) : nl > 1 ? t.stride(0) : H * d;
    if (t.stride(3) != 1 || (H > 1 && t.stride(2) != d) || (nl > 1 && t.stride(0) != T * ld))
      refuse(std::string(name) + " must have dense heads and evenly spaced tokens (strides " + list_of(t.strides()) + ")");
    return ld;
  }
  int64_t rows(const Tensor& t, const char* name, int64_t nl, int64_t T, int64_t H, int64_t d) const {
    const int64_t ld = token_stride(t, name, nl, T, H, d);
    like(t, name, ty);
    return ld;
  }
  void dims(const Tensor& t, const char* name, int64_t n, const char* shape) const {
    if (t.dim() != n) refuse(std::string(name) + " must be " + shape + ", not " + list_of(t.sizes()));
  }
  Tensor fresh(at::IntArrayRef shape, ScalarType dt) const { return at::empty(shape, at::TensorOptions().dtype(dt).device(dev)); }
  medusa_stream_t stream() const { return reinterpret_cast<medusa_stream_t>(c10::cuda::getCurrentCUDAStream(dev.index()).stream()); }
};

// An output: the given tensor, checked, or a new one.
struct Out {
  PyObject* given = nullptr;
  Tensor t;
  bool there = false;
  Out() = default;
  Out(const Call& c, PyObject* o, const char* name, at::IntArrayRef shape, ScalarType dt, bool wanted = true) {
    if (o != Py_None) {
      given = o;
      t = c.dense(c.tensor(o, name), name, dt, shape);
    } else if (wanted) {
      t = c.fresh(shape, dt);
    }
    there = t.defined();
  }
  void* ptr() const { return there ? t.data_ptr() : nullptr; }
  PyObject* object() const {
    if (!there) Py_RETURN_NONE;
    if (given) return Py_NewRef(given);
    return THPVariable_Wrap(t);
  }
};

int32_t* status_word(const Call& c, PyObject* o) {
  if (o == Py_None) return nullptr;
  const Tensor& t = c.tensor(o, "d_status");
  c.like(t, "d_status", ScalarType::Int);
  return static_cast<int32_t*>(t.data_ptr());
}

struct Workspace {
  Tensor t;
  size_t n;
  Workspace(const Call& c, PyObject* o, size_t need) : n(need) {
    if (o == Py_None) {
      t = c.fresh({(int64_t)need}, ScalarType::Byte);
      return;
    }
    t = c.tensor(o, "ws");
    if (t.device() != c.dev || !t.is_contiguous() || t.nbytes() < need)
      c.refuse("the workspace must be " + std::to_string(need) + " dense bytes on " + c.dev.str());
    n = t.nbytes();
  }
};

float number(const Call& c, PyObject* o, double otherwise) {
  if (o == Py_None) return (float)otherwise;
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw python_error();
  return (float)x;
}
bool flag(PyObject* o) {
  const int yes = PyObject_IsTrue(o);
  if (yes < 0) throw python_error();
  return yes == 1;
}
int small(const Call& c, int64_t n, const char* name) {
  if (n < 0 || n > 0x7fffffff) c.refuse(std::string(name) + " is out of range");
  return (int)n;
}
// (first, second), or the status that a refused call returned.
PyObject* result(medusa_status st, const Out& first, const Out& second) {
  if (st != MEDUSA_OK) return PyLong_FromLong(st);
  PyObject* pair = PyTuple_New(2);
  if (!pair) return nullptr;
  PyTuple_SET_ITEM(pair, 0, first.object());
  PyTuple_SET_ITEM(pair, 1, second.object());
  return pair;
}

template <typename F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F&& body) {
  HANDLE_TH_ERRORS
  if (got != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", want, got);
    return nullptr;
  }
  try {
    return body();
  } catch (const Refused& r) {
    PyErr_SetString(r.type, r.text.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// The library call, other Python threads running meanwhile.
template <typename F>
medusa_status enqueue(F&& f) {
  pybind11::gil_scoped_release off;
  return f();
}

}  // namespace
