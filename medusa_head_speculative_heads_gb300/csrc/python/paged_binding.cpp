// The paged-cache calls on torch tensors: argument checks, new tensors for what
// is not given, and marshalling.
//
// A decoding step makes these calls once per layer and their kernels run for a few
// microseconds.  Checked and marshalled in Python (some sixty attribute reads and
// three allocations a call) an attention call took the host 25 us, here 9, of which 6
// are its two launches; rotation 15 and 5 us, append 16 and 5, compaction 14 and 4.
#include "torch_call.h"

namespace {

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

const medusa_rope_plan* plan_at(PyObject* o) {
  if (o == Py_None) return nullptr;
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw python_error();
  return static_cast<const medusa_rope_plan*>(p);
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
