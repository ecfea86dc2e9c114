// The common form of the decode-side calls, from torch tensors to the C ABI.
//
// A decode step makes these calls at a rate of some 10^5 a second, and checking
// and marshalling the arguments in Python takes longer than the kernels run.  Each
// function here handles the form in which everything is as it should be: tensors
// of the right types and shapes on the current GPU, outputs to be allocated, the
// current stream.  It returns None for anything else, without having done
// anything, and binding.py then takes its own path, which says what is wrong or
// serves the rarer forms.  A status of the C ABI other than TQ_OK comes back as an
// int.
//
// Build: bit_mixed_precision_amd/build_lib.py.  The C entry points are handed
// over by address, so that the library that binding.py loaded is the one that runs.

#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstring>
#include <initializer_list>

#include "tq.h"

namespace {

struct Entries {
  decltype(&tq_rope) rope;
  decltype(&tq_rope_append) rope_append;
  decltype(&tq_paged_attention) paged_attention;
  decltype(&tq_paged_attention_workspace) paged_attention_workspace;
  decltype(&tq_pages_workspace) pages_workspace;
  decltype(&tq_pages_fork) pages_fork;
  decltype(&tq_pages_grow) pages_grow;
  decltype(&tq_pages_compact) pages_compact;
};
Entries c{};
PyObject* raw_stream = nullptr;  // device index -> HIP stream as an int

// A tensor argument, or nullptr.
const at::Tensor* tensor(PyObject* o) {
  return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr;
}

bool tensors(PyObject* const* args, std::initializer_list<int> which, const at::Tensor** out) {
  for (int i : which) {
    if (!(out[i] = tensor(args[i]))) return false;
  }
  return true;
}

int kind(const at::Tensor& t, bool f32) {
  switch (t.scalar_type()) {
    case at::kHalf: return TQ_F16;
    case at::kBFloat16: return TQ_BF16;
    case at::kFloat: return f32 ? TQ_F32 : -1;
    default: return -1;
  }
}

// A flag that the C ABI takes as it is: a bool, or the int 0 or 1; -1 for the rest,
// which binding.py looks at.
int flag(PyObject* o) {
  if (!PyLong_Check(o)) return -1;  // bools are ints
  int overflow = 0;
  const long v = PyLong_AsLongAndOverflow(o, &overflow);
  return !overflow && (v == 0 || v == 1) ? (int)v : -1;
}

bool on(const at::Tensor& t, const at::Device& d) { return t.device() == d; }

// t is on the GPU that is current.
bool current(const at::Tensor& t) {
  if (!t.is_cuda()) return false;
  static const c10::impl::VirtualGuardImpl guard(c10::DeviceType::CUDA);
  return guard.getDevice() == t.device();
}

bool int32s(const at::Tensor& t, at::IntArrayRef shape, const at::Device& d) {
  return t.scalar_type() == at::kInt && t.sizes() == shape && t.is_contiguous() && on(t, d);
}

// [tokens][heads][D], the numbers of a head adjacent
bool heads(const at::Tensor& t) { return t.dim() == 3 && (t.stride(2) == 1 || t.size(2) <= 1); }

// cosines and sines [positions][rot / 2][2]
bool angles(const at::Tensor& t, const at::Device& d) {
  return t.dim() == 3 && t.size(2) == 2 && t.scalar_type() == at::kFloat && t.is_contiguous() &&
         on(t, d);
}

bool matrix(const at::Tensor& t, const at::Device& d) {
  return t.dim() == 2 && t.scalar_type() == at::kInt && t.is_contiguous() && on(t, d);
}

// the halves of a paged cache [pages][slots][heads][D], as like's type
bool cache(const at::Tensor& k, const at::Tensor& v, const at::Tensor& like, const at::Device& d) {
  return k.dim() == 4 && k.size(3) == like.size(2) && (k.stride(3) == 1 || k.size(3) <= 1) &&
         k.scalar_type() == like.scalar_type() && v.scalar_type() == like.scalar_type() &&
         k.sizes() == v.sizes() && k.strides() == v.strides() && on(k, d) && on(v, d);
}

// [planes][pages][...] without gaps
bool pool_of(const at::Tensor& t, int64_t* planes, int64_t* pages, int64_t* bytes) {
  if (t.dim() < 3 || !t.is_contiguous()) return false;
  *planes = t.size(0);
  *pages = t.size(1);
  *bytes = t.element_size();
  for (int64_t i = 2; i < t.dim(); ++i) *bytes *= t.size(i);
  return true;
}

template <class T>
T* ptr(const at::Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}

// The current HIP stream of GPU d; *ok is false with a Python error set.
void* stream_of(const at::Device& d, bool* ok) {
  *ok = false;
  PyObject* index = PyLong_FromLong(d.index());
  if (!index) return nullptr;
  PyObject* s = PyObject_CallOneArg(raw_stream, index);
  Py_DECREF(index);
  if (!s) return nullptr;
  void* p = PyLong_AsVoidPtr(s);
  Py_DECREF(s);
  *ok = !(p == nullptr && PyErr_Occurred());
  return p;
}

PyObject* none() { Py_RETURN_NONE; }

PyObject* tuple(std::initializer_list<at::Tensor> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (!r) return nullptr;
  Py_ssize_t i = 0;
  for (const auto& t : ts) {
    PyObject* o = THPVariable_Wrap(t);
    if (!o) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// Nothing C++ throws leaves a function: allocation failures become Python errors.
template <class F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// (X, table, positions, interleaved, inverse)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor* t[3];
    if (n != 5 || !tensors(a, {0, 1, 2}, t)) return none();
    const at::Tensor &x = *t[0], &table = *t[1], &pos = *t[2];
    const int k = kind(x, true), inter = flag(a[3]), inv = flag(a[4]);
    const at::Device d = x.device();
    if (k < 0 || inter < 0 || inv < 0 || !current(x) || !heads(x) || !angles(table, d) ||
        !int32s(pos, {x.size(0)}, d))
      return none();
    bool ok;
    void* s = stream_of(d, &ok);
    if (!ok) return nullptr;
    at::Tensor y = at::empty(x.sizes(), x.options());
    const int st = c.rope(k, x.data_ptr(), x.stride(0), x.stride(1), y.data_ptr(), y.stride(0),
                          y.stride(1), ptr<float>(table), table.size(0), 2 * table.size(1),
                          ptr<int32_t>(pos), x.size(0), x.size(1), x.size(2), inter, inv, s);
    return st == TQ_OK ? THPVariable_Wrap(y) : PyLong_FromLong(st);
  });
}

// (QKV, table, positions, page_table, k_pages, v_pages, interleaved, seqs or None)
PyObject* rope_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor* t[6];
    if (n != 8 || !tensors(a, {0, 1, 2, 3, 4, 5}, t)) return none();
    const at::Tensor &x = *t[0], &table = *t[1], &pos = *t[2], &pages = *t[3], &k = *t[4],
                     &v = *t[5];
    const at::Tensor* seqs = a[7] == Py_None ? nullptr : tensor(a[7]);
    const int kd = kind(x, false), inter = flag(a[6]);
    const at::Device d = x.device();
    if (kd < 0 || inter < 0 || (a[7] != Py_None && !seqs) || !current(x) || !heads(x) ||
        (x.size(1) > 1 && x.stride(1) != x.size(2)) || !angles(table, d) || !matrix(pages, d) ||
        !int32s(pos, {x.size(0)}, d) || (seqs && !int32s(*seqs, {x.size(0)}, d)) ||
        !cache(k, v, x, d))
      return none();
    const int64_t T = x.size(0), D = x.size(2), Hkv = k.size(2), Hq = x.size(1) - 2 * Hkv;
    if (Hq < 1) return none();
    bool ok;
    void* s = stream_of(d, &ok);
    if (!ok) return nullptr;
    at::Tensor q = at::empty({T, Hq, D}, x.options());
    const int st = c.rope_append(
        kd, x.data_ptr(), x.stride(0), ptr<float>(table), table.size(0), 2 * table.size(1),
        ptr<int32_t>(pos), seqs ? ptr<int32_t>(*seqs) : nullptr, ptr<int32_t>(pages),
        pages.size(0), pages.size(1), k.data_ptr(), v.data_ptr(), k.size(0), k.size(1),
        k.stride(0), k.stride(1), k.stride(2), q.data_ptr(), T, Hq, Hkv, D, inter, s);
    return st == TQ_OK ? THPVariable_Wrap(q) : PyLong_FromLong(st);
  });
}

// (Q, k_pages, v_pages, page_table, lens, scale or None, window, return_lse)
PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor* t[5];
    if (n != 8 || !tensors(a, {0, 1, 2, 3, 4}, t)) return none();
    const at::Tensor &q = *t[0], &k = *t[1], &v = *t[2], &pages = *t[3], &lens = *t[4];
    const int kd = kind(q, false), with_lse = PyObject_IsTrue(a[7]);
    const at::Device d = q.device();
    if (kd < 0 || with_lse < 0 || !current(q) || !heads(q) || !matrix(pages, d) ||
        pages.size(0) != q.size(0) || !int32s(lens, {q.size(0)}, d) || !cache(k, v, q, d) ||
        !PyLong_Check(a[6]) || !(a[5] == Py_None || PyFloat_Check(a[5])))
      return PyErr_Occurred() ? nullptr : none();
    const int64_t B = q.size(0), Hq = q.size(1), D = q.size(2);
    const double scale = a[5] == Py_None ? 1.0 / std::sqrt((double)D) : PyFloat_AS_DOUBLE(a[5]);
    const long long window = PyLong_AsLongLong(a[6]);
    if (window == -1 && PyErr_Occurred()) return nullptr;
    const int64_t bytes =
        c.paged_attention_workspace(B, Hq, k.size(2), D, k.size(1), pages.size(1));
    if (bytes < 0) return PyLong_FromLong((long)bytes);
    bool ok;
    void* s = stream_of(d, &ok);
    if (!ok) return nullptr;
    at::Tensor out = at::empty({B, Hq, D}, q.options()), lse, ws;
    if (with_lse) lse = at::empty({B, Hq}, q.options().dtype(at::kFloat));
    if (bytes > 0) ws = at::empty({bytes}, q.options().dtype(at::kByte));
    const int st = c.paged_attention(
        kd, q.data_ptr(), q.stride(0), q.stride(1), k.data_ptr(), v.data_ptr(), k.size(0),
        k.size(1), k.stride(0), k.stride(1), k.stride(2), ptr<int32_t>(pages), pages.size(1),
        ptr<int32_t>(lens), B, Hq, k.size(2), D, scale, window, out.data_ptr(),
        with_lse ? ptr<float>(lse) : nullptr, bytes > 0 ? ws.data_ptr() : nullptr, bytes, s);
    if (st != TQ_OK) return PyLong_FromLong(st);
    return with_lse ? tuple({out, lse}) : THPVariable_Wrap(out);
  });
}

// (pool, page_table, lens, parent, page_size)
PyObject* pages_fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor* t[4];
    if (n != 5 || !tensors(a, {0, 1, 2, 3}, t) || !PyLong_Check(a[4])) return none();
    const at::Tensor &pool = *t[0], &table = *t[1], &lens = *t[2], &parent = *t[3];
    const at::Device d = pool.device();
    int64_t planes, pages, page_bytes;
    if (!current(pool) || !pool_of(pool, &planes, &pages, &page_bytes) || !matrix(table, d) ||
        !int32s(lens, {table.size(0)}, d) || parent.dim() != 1 ||
        !int32s(parent, {parent.size(0)}, d))
      return none();
    const long long size = PyLong_AsLongLong(a[4]);
    if (size == -1 && PyErr_Occurred()) return nullptr;
    const int64_t rows = parent.size(0), width = table.size(1);
    const int64_t bytes = c.pages_workspace(rows, pages);
    if (bytes < 0) return PyLong_FromLong((long)bytes);
    bool ok;
    void* s = stream_of(d, &ok);
    if (!ok) return nullptr;
    const auto o = lens.options();
    at::Tensor ws = at::empty({bytes / 4}, o), table_out = at::empty({rows, width}, o),
               lens_out = at::empty({rows}, o), refs = at::empty({pages}, o),
               lacking = at::empty({1}, o);
    const int st = c.pages_fork(pool.data_ptr(), planes, pages, page_bytes, ptr<int32_t>(table),
                                ptr<int32_t>(lens), table.size(0), ptr<int32_t>(parent), rows,
                                width, size, ptr<int32_t>(table_out), ptr<int32_t>(lens_out),
                                ptr<int32_t>(refs), ptr<int32_t>(lacking), ws.data_ptr(), bytes, s);
    return st == TQ_OK ? tuple({table_out, lens_out, refs, lacking}) : PyLong_FromLong(st);
  });
}

// (page_table, lens, add, n_pages, page_size)
PyObject* pages_grow(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor* t[3];
    if (n != 5 || !tensors(a, {0, 1, 2}, t) || !PyLong_Check(a[3]) || !PyLong_Check(a[4]))
      return none();
    const at::Tensor &table = *t[0], &lens = *t[1], &add = *t[2];
    const at::Device d = table.device();
    if (!current(table) || !matrix(table, d) || !int32s(lens, {table.size(0)}, d) ||
        !int32s(add, {table.size(0)}, d))
      return none();
    const long long pages = PyLong_AsLongLong(a[3]), size = PyLong_AsLongLong(a[4]);
    if (PyErr_Occurred()) return nullptr;
    const int64_t rows = table.size(0), width = table.size(1);
    const int64_t bytes = c.pages_workspace(rows, pages);
    if (bytes < 0) return PyLong_FromLong((long)bytes);
    bool ok;
    void* s = stream_of(d, &ok);
    if (!ok) return nullptr;
    const auto o = lens.options();
    at::Tensor ws = at::empty({bytes / 4}, o), table_out = at::empty({rows, width}, o),
               lens_out = at::empty({rows}, o), lacking = at::empty({1}, o);
    const int st = c.pages_grow(ptr<int32_t>(table), ptr<int32_t>(lens), ptr<int32_t>(add), rows,
                                width, size, pages, ptr<int32_t>(table_out),
                                ptr<int32_t>(lens_out), ptr<int32_t>(lacking), ws.data_ptr(),
                                bytes, s);
    return st == TQ_OK ? tuple({table_out, lens_out, lacking}) : PyLong_FromLong(st);
  });
}

// (pool, page_table, lens, page_size)
PyObject* pages_compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor* t[3];
    if (n != 4 || !tensors(a, {0, 1, 2}, t) || !PyLong_Check(a[3])) return none();
    const at::Tensor &pool = *t[0], &table = *t[1], &lens = *t[2];
    const at::Device d = pool.device();
    int64_t planes, pages, page_bytes;
    if (!current(pool) || !pool_of(pool, &planes, &pages, &page_bytes) || !matrix(table, d) ||
        !int32s(lens, {table.size(0)}, d))
      return none();
    const long long size = PyLong_AsLongLong(a[3]);
    if (size == -1 && PyErr_Occurred()) return nullptr;
    const int64_t rows = table.size(0), width = table.size(1);
    const int64_t bytes = c.pages_workspace(rows, pages);
    if (bytes < 0) return PyLong_FromLong((long)bytes);
    bool ok;
    void* s = stream_of(d, &ok);
    if (!ok) return nullptr;
    const auto o = lens.options();
    at::Tensor ws = at::empty({bytes / 4}, o), table_out = at::empty({rows, width}, o),
               used = at::empty({1}, o);
    const int st = c.pages_compact(pool.data_ptr(), planes, pages, page_bytes, ptr<int32_t>(table),
                                   ptr<int32_t>(lens), rows, width, size, ptr<int32_t>(table_out),
                                   ptr<int32_t>(used), ws.data_ptr(), bytes, s);
    return st == TQ_OK ? tuple({table_out, used}) : PyLong_FromLong(st);
  });
}

// bind(raw_stream, {name: address}): what the functions call
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 2 || !PyDict_Check(a[1])) {
    PyErr_SetString(PyExc_TypeError, "bind(raw_stream, addresses)");
    return nullptr;
  }
  auto take = [&](const char* name, auto* fn) {
    PyObject* o = PyDict_GetItemString(a[1], name);  // borrowed
    void* p = o ? PyLong_AsVoidPtr(o) : nullptr;
    if (!p) {
      if (!PyErr_Occurred()) PyErr_Format(PyExc_KeyError, "%s", name);
      return false;
    }
    static_assert(sizeof(*fn) == sizeof p, "");
    std::memcpy(fn, &p, sizeof p);
    return true;
  };
  Entries e{};  // all or nothing
  if (!take("tq_rope", &e.rope) || !take("tq_rope_append", &e.rope_append) ||
      !take("tq_paged_attention", &e.paged_attention) ||
      !take("tq_paged_attention_workspace", &e.paged_attention_workspace) ||
      !take("tq_pages_workspace", &e.pages_workspace) || !take("tq_pages_fork", &e.pages_fork) ||
      !take("tq_pages_grow", &e.pages_grow) || !take("tq_pages_compact", &e.pages_compact))
    return nullptr;
  c = e;
  Py_INCREF(a[0]);
  Py_XDECREF(raw_stream);
  raw_stream = a[0];
  Py_RETURN_NONE;
}

#define TQ_METHOD(name) \
  { #name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr }
PyMethodDef methods[] = {TQ_METHOD(bind),          TQ_METHOD(rope),
                         TQ_METHOD(rope_append),   TQ_METHOD(paged_attention),
                         TQ_METHOD(pages_fork),    TQ_METHOD(pages_grow),
                         TQ_METHOD(pages_compact), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tq_torch",
                      "Decode-side calls of libtq.so in their common form.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: the torch whose headers this was compiled with; binding.py calls
// nothing here under any other.
PyMODINIT_FUNC PyInit__tq_torch() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", TQ_TORCH_VERSION) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
