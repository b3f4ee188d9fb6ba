// The paged-cache calls on torch tensors: argument checks, new tensors for what
// is not given, and marshalling.
//
// A decoding step makes these calls once per layer and their kernels run for a few
// microseconds.  Checked and marshalled in Python (some sixty attribute reads and
// three allocations a call) an attention call took the host 25 us, here 9, of which 6
// are its two launches; rotation 15 and 5 us, append 16 and 5, compaction 14 and 4.
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

// Pools, table and lengths of a call over B sequences.
struct Pools {
  int64_t nl, n_pages, ps, hkv, d, B, max_pages;
  const Tensor *k, *v, *table;
  Pools(const Call& c, PyObject* kp, PyObject* vp, PyObject* tab) {
    k = &c.tensor(kp, "k_pages");
    v = &c.tensor(vp, "v_pages");
    table = &c.tensor(tab, "page_table");
    c.dims(*k, "k_pages", 5, "[nl, n_pages, page_size, Hkv, d]");
    c.dims(*table, "page_table", 2, "[B, max_pages]");
    nl = k->size(0);
    n_pages = k->size(1);
    ps = k->size(2);
    hkv = k->size(3);
    d = k->size(4);
    B = table->size(0);
    max_pages = table->size(1);
  }
  void check(const Call& c) const {
    c.dense(*k, "k_pages", c.ty, k->sizes());
    c.dense(*v, "v_pages", c.ty, k->sizes());
    c.words(*table, "page_table", table->numel());
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
const medusa_rope_plan* plan_at(PyObject* o) {
  if (o == Py_None) return nullptr;
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw python_error();
  return static_cast<const medusa_rope_plan*>(p);
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

// q, k, pos, plan, q_out, k_out, inverse
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject* {
    Call c{"medusa_rope"};
    const bool inverse = flag(a[6]);
    const Tensor& q = c.tensor(a[0], "q");
    const int dt = c.lead(q, "q");
    c.dims(q, "q", 4, "[nl, T, Hq, d]");
    const int64_t nl = q.size(0), T = q.size(1), hq = q.size(2), d = q.size(3);
    const int64_t ldq = c.rows(q, "q", nl, T, hq, d);
    int64_t hkv = 0, ldk = 0;
    const void* k = nullptr;
    if (a[1] != Py_None) {
      const Tensor& t = c.tensor(a[1], "k");
      c.dims(t, "k", 4, "[nl, T, Hkv, d]");
      hkv = t.size(2);
      ldk = c.rows(t, "k", nl, T, hkv, d);
      k = t.data_ptr();
    } else if (a[5] != Py_None) {
      c.refuse("k_out needs k");
    }
    const int32_t* pos = c.words(a[2], "pos", T);
    c10::DeviceGuard on(c.dev);
    const Out qo(c, a[4], "q_out", {nl, T, hq, d}, c.ty), ko(c, a[5], "k_out", {nl, T, hkv, d}, c.ty, k != nullptr);
    const medusa_rope_plan* plan = plan_at(a[3]);
    const medusa_status st = enqueue([&] {
      return medusa_rope(q.data_ptr(), ldq, k, ldk, pos, plan, inverse, small(c, nl, "nl"), small(c, T, "T"), small(c, hq, "Hq"),
                         small(c, hkv, "Hkv"), small(c, d, "d"), (medusa_dtype)dt, qo.ptr(), ko.ptr(), c.stream());
    });
    return result(st, qo, ko);
  });
}

// k, v, k_pages, v_pages, page_table, q_start, prefix_len, q, pos, plan, q_out, d_status
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    Call c{"medusa_paged_append"};
    const Tensor &k = c.tensor(a[0], "k"), &v = c.tensor(a[1], "v");
    const int dt = c.lead(k, "k");
    const Pools p(c, a[2], a[3], a[4]);
    c.dims(k, "k", 4, "[nl, T, Hkv, d]");
    c.dims(v, "v", 4, "[nl, T, Hkv, d]");
    const int64_t T = k.size(1), ldk = c.rows(k, "k", p.nl, T, p.hkv, p.d), ldv = c.rows(v, "v", p.nl, T, p.hkv, p.d);
    p.check(c);
    const int32_t *start = c.words(a[5], "q_start", p.B + 1), *len = c.words(a[6], "prefix_len", p.B);
    const int32_t* pos = a[8] == Py_None ? nullptr : c.words(a[8], "pos", T);
    int32_t* status = status_word(c, a[11]);
    c10::DeviceGuard on(c.dev);
    int64_t hq = 0, ldq = 0;
    const void* q = nullptr;
    Out qo;
    if (a[7] != Py_None) {
      const Tensor& t = c.tensor(a[7], "q");
      c.dims(t, "q", 4, "[nl, T, Hq, d]");
      hq = t.size(2);
      ldq = c.rows(t, "q", p.nl, T, hq, p.d);
      q = t.data_ptr();
      qo = Out(c, a[10], "q_out", {p.nl, T, hq, p.d}, c.ty);
    } else if (a[10] != Py_None) {
      c.refuse("q_out needs q");
    }
    const medusa_rope_plan* plan = plan_at(a[9]);
    const medusa_status st = enqueue([&] {
      return medusa_paged_append(q, ldq, k.data_ptr(), ldk, v.data_ptr(), ldv, pos, plan, static_cast<int32_t*>(p.table->data_ptr()), start, len,
                                 small(c, p.nl, "nl"), small(c, T, "T"), small(c, p.B, "B"), small(c, hq, "Hq"), small(c, p.hkv, "Hkv"),
                                 small(c, p.d, "d"), small(c, p.n_pages, "n_pages"), small(c, p.ps, "page_size"),
                                 small(c, p.max_pages, "max_pages"), (medusa_dtype)dt, qo.ptr(), p.k->data_ptr(), p.v->data_ptr(), status, c.stream());
    });
    return result(st, qo, Out());
  });
}

// q, k_pages, v_pages, page_table, q_start, prefix_len, scale, out, lse, want_lse, ws, d_status
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    Call c{"medusa_paged_attention"};
    const bool want_lse = flag(a[9]);
    const Tensor& q = c.tensor(a[0], "q");
    const int dt = c.lead(q, "q");
    const Pools p(c, a[1], a[2], a[3]);
    c.dims(q, "q", 4, "[nl, T, Hq, d]");
    const int64_t T = q.size(1), hq = q.size(2), ldq = c.rows(q, "q", p.nl, T, hq, p.d);
    p.check(c);
    const int32_t *start = c.words(a[4], "q_start", p.B + 1), *len = c.words(a[5], "prefix_len", p.B);
    int32_t* status = status_word(c, a[11]);
    c10::DeviceGuard on(c.dev);
    const Out out(c, a[7], "out", {p.nl, T, hq, p.d}, c.ty);
    const Out lse(c, a[8], "lse", {p.nl, T, hq}, ScalarType::Float, want_lse);
    const int nl = small(c, p.nl, "nl"), t = small(c, T, "T"), b = small(c, p.B, "B"), h = small(c, hq, "Hq"), hk = small(c, p.hkv, "Hkv"),
              d = small(c, p.d, "d"), np = small(c, p.n_pages, "n_pages"), ps = small(c, p.ps, "page_size"), mp = small(c, p.max_pages, "max_pages");
    const float scale = number(c, a[6], 1.0 / std::sqrt((double)(d > 0 ? d : 1)));
    const Workspace ws(c, a[10], medusa_paged_attention_workspace_size(nl, t, b, h, hk, d, ps, (medusa_dtype)dt));
    const medusa_status st = enqueue([&] {
      return medusa_paged_attention(q.data_ptr(), ldq, p.k->data_ptr(), p.v->data_ptr(), static_cast<int32_t*>(p.table->data_ptr()), start, len, nl, t, b,
                                    h, hk, d, np, ps, mp, scale, (medusa_dtype)dt, out.ptr(), static_cast<float*>(lse.ptr()), ws.t.data_ptr(), ws.n,
                                    status, c.stream());
    });
    return result(st, out, lse);
  });
}

// q, k_pages, v_pages, page_table, kt, vt, mask, prefix_len, scale, out, lse, want_lse, ws, d_status
PyObject* tree_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> PyObject* {
    Call c{"medusa_paged_tree_attention"};
    const bool want_lse = flag(a[11]);
    const Tensor &q = c.tensor(a[0], "q"), &kt = c.tensor(a[4], "kt"), &vt = c.tensor(a[5], "vt");
    const int dt = c.lead(q, "q");
    const Pools p(c, a[1], a[2], a[3]);
    c.dims(q, "q", 5, "[nl, B, N, Hq, d]");
    const int64_t N = q.size(2), hq = q.size(3);
    const int64_t rows[5] = {p.nl, p.B, N, p.hkv, p.d};
    c.dense(q, "q", c.ty, {p.nl, p.B, N, hq, p.d});
    c.dense(kt, "kt", c.ty, rows);
    c.dense(vt, "vt", c.ty, rows);
    p.check(c);
    const Tensor& mask = c.dense(c.tensor(a[6], "mask"), "mask", ScalarType::Int, {N, (N + 31) / 32});
    const int32_t* len = c.words(a[7], "prefix_len", p.B);
    int32_t* status = status_word(c, a[13]);
    c10::DeviceGuard on(c.dev);
    const Out out(c, a[9], "out", {p.nl, p.B, N, hq, p.d}, c.ty);
    const Out lse(c, a[10], "lse", {p.nl, p.B, N, hq}, ScalarType::Float, want_lse);
    const int nl = small(c, p.nl, "nl"), b = small(c, p.B, "B"), nn = small(c, N, "N"), t = small(c, p.B * N, "B * N"), h = small(c, hq, "Hq"),
              hk = small(c, p.hkv, "Hkv"), d = small(c, p.d, "d"), np = small(c, p.n_pages, "n_pages"), ps = small(c, p.ps, "page_size"),
              mp = small(c, p.max_pages, "max_pages");
    const float scale = number(c, a[8], 1.0 / std::sqrt((double)(d > 0 ? d : 1)));
    const Workspace ws(c, a[12], medusa_paged_attention_workspace_size(nl, t, b, h, hk, d, ps, (medusa_dtype)dt));
    const medusa_status st = enqueue([&] {
      return medusa_paged_tree_attention(q.data_ptr(), p.k->data_ptr(), p.v->data_ptr(), static_cast<int32_t*>(p.table->data_ptr()), kt.data_ptr(),
                                         vt.data_ptr(), static_cast<uint32_t*>(mask.data_ptr()), len, nl, b, nn, h, hk, d, np, ps, mp, scale,
                                         (medusa_dtype)dt, out.ptr(), static_cast<float*>(lse.ptr()), ws.t.data_ptr(), ws.n, status, c.stream());
    });
    return result(st, out, lse);
  });
}

// k_pages, v_pages, page_table, kt, vt, path_nodes, accept_len, prefix_len, new_len, d_status
PyObject* compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    Call c{"medusa_paged_compact"};
    const Tensor &kt = c.tensor(a[3], "kt"), &vt = c.tensor(a[4], "vt"), &path = c.tensor(a[5], "path_nodes");
    const int dt = c.lead(kt, "kt");
    const Pools p(c, a[0], a[1], a[2]);
    c.dims(kt, "kt", 5, "[nl, B, N, Hkv, d]");
    c.dims(path, "path_nodes", 2, "[B, Dmax + 1]");
    const int64_t N = kt.size(2), rows[5] = {p.nl, p.B, N, p.hkv, p.d};
    c.dense(kt, "kt", c.ty, rows);
    c.dense(vt, "vt", c.ty, rows);
    p.check(c);
    const int32_t *nodes = static_cast<int32_t*>(c.dense(path, "path_nodes", ScalarType::Int, {p.B, path.size(1)}).data_ptr()),
                  *acc = c.words(a[6], "accept_len", p.B), *len = c.words(a[7], "prefix_len", p.B);
    int32_t* status = status_word(c, a[9]);
    c10::DeviceGuard on(c.dev);
    const Out nlen(c, a[8], "new_len", {p.B}, ScalarType::Int);
    const medusa_status st = enqueue([&] {
      return medusa_paged_compact(p.k->data_ptr(), p.v->data_ptr(), static_cast<int32_t*>(p.table->data_ptr()), kt.data_ptr(), vt.data_ptr(), nodes, acc, len,
                                  static_cast<int32_t*>(nlen.ptr()), small(c, p.nl, "nl"), small(c, p.B, "B"), small(c, N, "N"), small(c, p.hkv, "Hkv"),
                                  small(c, p.d, "d"), small(c, p.n_pages, "n_pages"), small(c, p.ps, "page_size"), small(c, p.max_pages, "max_pages"),
                                  (int)path.size(1) - 1, (medusa_dtype)dt, status, c.stream());
    });
    return result(st, nlen, Out());
  });
}

// what, name, t, nl, T, H, d: the stride the calls pass for t, refused as they refuse it
PyObject* token_stride(PyObject*, PyObject* args) {
  const char *what, *name;
  PyObject* t;
  long long nl, T, H, d;
  if (!PyArg_ParseTuple(args, "ssOLLLL", &what, &name, &t, &nl, &T, &H, &d)) return nullptr;
  return guarded(0, 0, [&]() -> PyObject* {
    Call c{what};
    const Tensor& x = c.tensor(t, name);
    c.dims(x, name, 4, "[nl, T, H, d]");
    return PyLong_FromLongLong(c.token_stride(x, name, nl, T, H, d));
  });
}

PyMethodDef methods[] = {
    {"rope", (PyCFunction)(void (*)())rope, METH_FASTCALL, nullptr},
    {"append", (PyCFunction)(void (*)())append, METH_FASTCALL, nullptr},
    {"attention", (PyCFunction)(void (*)())attention, METH_FASTCALL, nullptr},
    {"tree_attention", (PyCFunction)(void (*)())tree_attention, METH_FASTCALL, nullptr},
    {"compact", (PyCFunction)(void (*)())compact, METH_FASTCALL, nullptr},
    {"token_stride", token_stride, METH_VARARGS, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "paged_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit_paged_binding() { return PyModule_Create(&module); }
