// The calls around a verify pass's output on torch tensors: argument checks, new tensors for
// what is not given, and marshalling.  A decoding step makes the linear calls several times a layer,
// and their kernels run for a few microseconds.
#include "torch_call.h"

namespace {

// A matrix of evenly spaced rows, each dense: elements from one row to the next.
int64_t row_stride(const Call& c, const Tensor& t, const char* name, int64_t rows, int64_t cols) {
  const int64_t ld = rows > 1 ? t.stride(-2) : cols;
  if ((cols > 1 && t.stride(-1) != 1) || ld < cols) c.refuse(std::string(name) + " must have dense rows (strides " + list_of(t.strides()) + ")");
  return ld;
}

// w, group, symmetric
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 3, [&]() -> PyObject* {
    Call c{"medusa_w4_quantize"};
    const bool symmetric = flag(a[2]);
    const int64_t group = PyLong_AsLongLong(a[1]);
    if (group == -1 && PyErr_Occurred()) throw python_error();
    const Tensor& w = c.tensor(a[0], "w");
    const int dt = c.lead(w, "w");
    c.dims(w, "w", 2, "[Nout, K]");
    const int64_t N = w.size(0), K = w.size(1);
    c.dense(w, "w", c.ty, {N, K});
    if ((group != 32 && group != 64 && group != 128) || K % group || K < 1 || N < 1)
      c.refuse("group must be 32, 64 or 128 and divide K, not " + std::to_string(group) + " of w " + list_of(w.sizes()));
    c10::DeviceGuard on(c.dev);
    const Tensor q = c.fresh({N, K / 8}, ScalarType::Int), s = c.fresh({K / group, N}, ScalarType::BFloat16);
    Out z;
    if (!symmetric) z = Out(c, Py_None, "zeros", {K / group, N}, ScalarType::Byte);
    const medusa_status st = enqueue([&] {
      return medusa_w4_quantize(w.data_ptr(), small(c, N, "Nout"), small(c, K, "K"), (int)group, symmetric, (medusa_dtype)dt,
                                static_cast<uint32_t*>(q.data_ptr()), s.data_ptr(), static_cast<uint8_t*>(z.ptr()), c.stream());
    });
    if (st != MEDUSA_OK) return PyLong_FromLong(st);
    PyObject* r = PyTuple_New(3);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(q));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(s));
    PyTuple_SET_ITEM(r, 2, z.object());
    return r;
  });
}

// x, qweight, scales, zeros, y, fp32 (a truth value; anything else: a type that y cannot have), d_status
PyObject* linear_w4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject* {
    Call c{"medusa_linear_w4"};
    const Tensor &x = c.tensor(a[0], "x"), &q = c.tensor(a[1], "qweight"), &s = c.tensor(a[2], "scales");
    if (!PyBool_Check(a[5])) c.refuse("y is bfloat16 or float32", PyExc_TypeError);
    c.lead(x, "x");
    if (c.ty != ScalarType::BFloat16) c.refuse("x must be bfloat16", PyExc_TypeError);
    c.dims(x, "x", 2, "[T, K]");
    c.dims(q, "qweight", 2, "[Nout, K / 8]");
    c.dims(s, "scales", 2, "[K / group, Nout]");
    const int64_t T = x.size(0), K = x.size(1), N = q.size(0), ng = s.size(0), ldx = row_stride(c, x, "x", T, K);
    if (K < 1 || ng < 1 || K % ng || (K / ng != 32 && K / ng != 64 && K / ng != 128))
      c.refuse("scales of " + std::to_string(ng) + " groups do not fit x of " + std::to_string(K) + " columns: a group is 32, 64 or 128 of them");
    c.dense(q, "qweight", ScalarType::Int, {N, K / 8});
    c.dense(s, "scales", ScalarType::BFloat16, {ng, N});
    const uint8_t* zeros = nullptr;
    if (a[3] != Py_None) zeros = static_cast<uint8_t*>(c.dense(c.tensor(a[3], "zeros"), "zeros", ScalarType::Byte, {ng, N}).data_ptr());
    int32_t* status = status_word(c, a[6]);
    c10::DeviceGuard on(c.dev);
    ScalarType out = a[5] == Py_True ? ScalarType::Float : ScalarType::BFloat16;
    if (a[4] != Py_None) {
      const ScalarType given = c.tensor(a[4], "y").scalar_type();
      if (given == ScalarType::Float) out = given;  // a y of that type asks for it
    }
    const Out y(c, a[4], "y", {T, N}, out);
    const int t = small(c, T, "T"), k = small(c, K, "K"), nn = small(c, N, "Nout"), g = (int)(K / ng);
    const medusa_status st = enqueue([&] {
      return medusa_linear_w4(x.data_ptr(), ldx, static_cast<uint32_t*>(q.data_ptr()), s.data_ptr(), zeros, t, k, nn, g, y.ptr(),
                              out == ScalarType::Float ? MEDUSA_F32 : MEDUSA_BF16, status, c.stream());
    });
    return st != MEDUSA_OK ? PyLong_FromLong(st) : y.object();
  });
}

// logits, counts, prompt_bits, repetition, frequency, presence, bias, mask, mask_row, tokens, topology, out, d_status
PyObject* logits(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject* {
    Call c{"medusa_logits_process"};
    const Tensor& z = c.tensor(a[0], "logits");
    const int dt = c.lead(z, "logits");
    c.dims(z, "logits", 3, "[B, N, V]");
    const int64_t B = z.size(0), N = z.size(1), V = z.size(2), W = (V + 31) / 32;
    if (B < 1 || N < 1 || V < 1) c.refuse("logits must not be empty, but are " + list_of(z.sizes()));
    const int64_t ld = N > 1 ? z.stride(1) : B > 1 ? z.stride(0) : V;
    if ((V > 1 && z.stride(2) != 1) || ld < V || (B > 1 && N > 1 && z.stride(0) != N * ld))
      c.refuse("logits must have dense, evenly spaced rows (strides " + list_of(z.strides()) + ")");
    medusa_logits_rules r{};
    auto given = [&](int i) { return a[i] != Py_None; };
    auto floats = [&](int i, const char* name) -> const float* {
      return given(i) ? static_cast<float*>(c.dense(c.tensor(a[i], name), name, ScalarType::Float, {B}).data_ptr()) : nullptr;
    };
    auto ints = [&](int i, const char* name, at::IntArrayRef shape) -> int32_t* {
      return given(i) ? static_cast<int32_t*>(c.dense(c.tensor(a[i], name), name, ScalarType::Int, shape).data_ptr()) : nullptr;
    };
    r.counts = ints(1, "counts", {B, V});
    r.prompt_bits = reinterpret_cast<uint32_t*>(ints(2, "prompt_bits", {B, W}));
    r.repetition = floats(3, "repetition");
    r.frequency = floats(4, "frequency");
    r.presence = floats(5, "presence");
    if (given(6)) {
      const Tensor& b = c.tensor(a[6], "bias");
      const int64_t one[1] = {V}, each[2] = {B, V};
      c.dense(b, "bias", ScalarType::Float, b.dim() == 1 ? at::IntArrayRef(one, 1) : at::IntArrayRef(each, 2));
      r.bias = static_cast<float*>(b.data_ptr());
      r.bias_rows = b.dim() == 1 ? 1 : small(c, B, "B");
    }
    if (given(7)) {
      const Tensor& m = c.tensor(a[7], "mask");
      c.dims(m, "mask", 2, "[M, ceil(V / 32)]");
      const int64_t M = given(8) ? m.size(0) : B * N;
      if (M < 1) c.refuse("mask must have rows: one without any has no address, and would be none");
      r.mask = reinterpret_cast<uint32_t*>(ints(7, "mask", {M, W}));
      r.n_masks = small(c, M, "M");
      r.mask_row = ints(8, "mask_row", {B, N});
    } else if (given(8)) {
      c.refuse("mask_row needs mask");
    }
    const medusa_dev_topology* topo = nullptr;
    const int32_t* tokens = nullptr;
    if (given(10)) {
      topo = static_cast<const medusa_dev_topology*>(PyLong_AsVoidPtr(a[10]));
      if (!topo) {
        if (PyErr_Occurred()) throw python_error();
        c.refuse("topo must be a device topology");
      }
      if (!given(9)) c.refuse("topo needs tokens");
      if (topo->n_nodes != N) c.refuse("logits of " + std::to_string(N) + " nodes do not fit a tree of " + std::to_string(topo->n_nodes));
      tokens = ints(9, "tokens", {B, N});
    } else if (given(9)) {
      c.refuse("tokens need topo");
    }
    int32_t* status = status_word(c, a[12]);
    c10::DeviceGuard on(c.dev);
    const Out out(c, a[11], "out", {B, N, V}, ScalarType::Float);
    const medusa_status st = enqueue([&] {
      return medusa_logits_process(z.data_ptr(), ld, (medusa_dtype)dt, &r, tokens, topo, small(c, B, "B"), small(c, N, "N"), small(c, V, "V"),
                                   static_cast<float*>(out.ptr()), status, c.stream());
    });
    return st != MEDUSA_OK ? PyLong_FromLong(st) : out.object();
  });
}

// The tensor that all others of a call on int32 words must be like.
const Tensor& words_lead(Call& c, PyObject* o, const char* name) {
  const Tensor& t = c.tensor(o, name);
  if (t.scalar_type() != ScalarType::Int) c.refuse(std::string(name) + " must be Int, not " + c10::toString(t.scalar_type()), PyExc_TypeError);
  if (!t.is_cuda()) c.refuse(std::string(name) + " must be on a GPU");
  c.dev = t.device();
  return t;
}

// tokens, V, counts, prompt_bits, d_status
PyObject* count_tokens(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject* {
    Call c{"medusa_count_tokens"};
    const int64_t V = PyLong_AsLongLong(a[1]);
    if (V == -1 && PyErr_Occurred()) throw python_error();
    const Tensor& t = words_lead(c, a[0], "tokens");
    c.dims(t, "tokens", 2, "[B, S]");
    const int64_t B = t.size(0), S = t.size(1);
    c.dense(t, "tokens", ScalarType::Int, {B, S});
    if (V < 1 || B < 1) c.refuse("V and B must be at least 1");
    if (a[2] == Py_None && a[3] == Py_None) c.refuse("counts or prompt_bits must be given");
    int32_t *counts = nullptr, *bits = nullptr;
    if (a[2] != Py_None) counts = static_cast<int32_t*>(c.dense(c.tensor(a[2], "counts"), "counts", ScalarType::Int, {B, V}).data_ptr());
    if (a[3] != Py_None) bits = static_cast<int32_t*>(c.dense(c.tensor(a[3], "prompt_bits"), "prompt_bits", ScalarType::Int, {B, (V + 31) / 32}).data_ptr());
    int32_t* status = status_word(c, a[4]);
    c10::DeviceGuard on(c.dev);
    return PyLong_FromLong(enqueue([&] {
      return medusa_count_tokens(static_cast<int32_t*>(t.data_ptr()), small(c, B, "B"), small(c, S, "S"), small(c, V, "V"), counts,
                                 reinterpret_cast<uint32_t*>(bits), status, c.stream());
    }));
  });
}

// counts, tokens, path_nodes, accept_len, d_status
PyObject* count_accepted(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject* {
    Call c{"medusa_count_accepted"};
    const Tensor& counts = words_lead(c, a[0], "counts");
    const Tensor &tokens = c.tensor(a[1], "tokens"), &path = c.tensor(a[2], "path_nodes");
    c.dims(counts, "counts", 2, "[B, V]");
    c.dims(tokens, "tokens", 2, "[B, N]");
    c.dims(path, "path_nodes", 2, "[B, Dmax + 1]");
    const int64_t B = counts.size(0), V = counts.size(1), N = tokens.size(1), D1 = path.size(1);
    c.dense(counts, "counts", ScalarType::Int, {B, V});
    c.dense(tokens, "tokens", ScalarType::Int, {B, N});
    c.dense(path, "path_nodes", ScalarType::Int, {B, D1});
    const int32_t* len = c.words(a[3], "accept_len", B);
    int32_t* status = status_word(c, a[4]);
    c10::DeviceGuard on(c.dev);
    return PyLong_FromLong(enqueue([&] {
      return medusa_count_accepted(static_cast<int32_t*>(tokens.data_ptr()), static_cast<int32_t*>(path.data_ptr()), len, small(c, B, "B"),
                                   small(c, N, "N"), small(c, D1, "Dmax + 1") - 1, small(c, V, "V"), static_cast<int32_t*>(counts.data_ptr()), status,
                                   c.stream());
    }));
  });
}

PyMethodDef methods[] = {
    {"quantize", (PyCFunction)(void (*)())quantize, METH_FASTCALL, nullptr},
    {"linear_w4", (PyCFunction)(void (*)())linear_w4, METH_FASTCALL, nullptr},
    {"logits", (PyCFunction)(void (*)())logits, METH_FASTCALL, nullptr},
    {"count_tokens", (PyCFunction)(void (*)())count_tokens, METH_FASTCALL, nullptr},
    {"count_accepted", (PyCFunction)(void (*)())count_accepted, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "verify_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit_verify_binding() { return PyModule_Create(&module); }
