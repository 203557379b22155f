// Argument marshalling of the paged-cache calls (specfold_cache.h) for torch
// tensors: checks of type, device, shape and strides, then one call of the C
// ABI.  A decode step makes these calls once per layer, for kernels of a few
// microseconds, so the marshalling is compiled: about 0.1 us a tensor less than
// attribute by attribute from Python, 12 us a call in all.
//
// Every function returns the call's sf_status, or raises ValueError for a
// tensor that does not fit (nothing is called then).
#include <Python.h>

#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "specfold_cache.h"

namespace {

// What the checks need to know of an object: a PyCapsule of this.
struct State {
  sf_cache* cache;
  int device;  // -1: CPU tensors (the checks alone can be tested so)
  at::ScalarType dtype;
  int64_t nq, nkv, hd, page;
};

void free_state(PyObject* cap) { delete static_cast<State*>(PyCapsule_GetPointer(cap, "sf_cache_state")); }

struct Refused {
  std::string text;
};

std::string describe(const at::Tensor& t) {
  std::string s = std::string(c10::toString(t.scalar_type())) + " [";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  s += "] strides [";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.stride(i));
  return s + "] on " + t.device().str();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Refused{std::string(name) + " must be a tensor"};
  return THPVariable_Unpack(o);
}

[[noreturn]] void refuse(const State& s, const char* name, const at::Tensor& t, const std::string& want) {
  throw Refused{std::string(name) + " must be " + want + " on device " + std::to_string(s.device) + ": got " +
                describe(t)};
}

bool here(const State& s, const at::Tensor& t) {
  return t.layout() == c10::kStrided && (s.device < 0 ? t.device().is_cpu() : t.is_cuda() && t.get_device() == s.device);
}

// Contiguous tensor of the given type and shape; None gives a null pointer where it may.
template <size_t N>
void* fixed(const State& s, PyObject* o, const char* name, at::ScalarType type, const int64_t (&shape)[N],
            bool optional = false) {
  if (o == Py_None && optional) return nullptr;
  const at::Tensor& t = tensor(o, name);
  bool ok = t.scalar_type() == type && here(s, t) && t.dim() == (int64_t)N && t.is_contiguous();
  for (size_t i = 0; ok && i < N; ++i) ok = t.size(i) == shape[i];
  if (!ok) {
    std::string want = std::string("contiguous ") + c10::toString(type) + " [";
    for (size_t i = 0; i < N; ++i) want += (i ? ", " : "") + std::to_string(shape[i]);
    refuse(s, name, t, want + "]");
  }
  return t.data_ptr();
}

struct Rows {
  void* p;
  int64_t n, ld;
};

// [T, heads, head_dim] or [T, heads * head_dim] with contiguous rows.
Rows rows(const State& s, PyObject* o, const char* name, int64_t heads) {
  const at::Tensor& t = tensor(o, name);
  bool ok = t.scalar_type() == s.dtype && here(s, t);
  if (t.dim() == 3)
    ok = ok && t.size(1) == heads && t.size(2) == s.hd && t.stride(2) == 1 && (heads == 1 || t.stride(1) == s.hd);
  else
    ok = ok && t.dim() == 2 && t.size(1) == heads * s.hd && t.stride(1) == 1;
  if (!ok)
    refuse(s, name, t, std::string(c10::toString(s.dtype)) + " [T, " + std::to_string(heads) + ", " +
                           std::to_string(s.hd) + "] (or flattened) with contiguous rows");
  return Rows{t.data_ptr(), t.size(0), t.stride(0)};
}

struct Pools {
  void *k, *v;
  int64_t pages;
};

Pools pools(const State& s, PyObject* ko, PyObject* vo, const char* kname = "k_pages",
            const char* vname = "v_pages") {
  Pools p{};
  const at::Tensor& k = tensor(ko, kname);
  const int64_t shape[4] = {k.dim() == 4 ? k.size(0) : 0, s.page, s.nkv, s.hd};
  p.k = fixed(s, ko, kname, s.dtype, shape);
  p.v = fixed(s, vo, vname, s.dtype, shape);
  p.pages = shape[0];
  return p;
}

struct Table {
  const int32_t* p;
  int64_t S, cols, ld;
};

Table table(const State& s, PyObject* o, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != at::kInt || !here(s, t) || t.dim() != 2 || (t.size(1) > 1 && t.stride(1) != 1))
    refuse(s, name, t, "Int [S, columns] with contiguous rows");
  return Table{static_cast<const int32_t*>(t.data_ptr()), t.size(0), t.size(1), t.stride(0)};
}

void* stream_of(const State& s, PyObject* o) {
  if (o == Py_None) return s.device < 0 ? nullptr : c10::cuda::getCurrentCUDAStream(s.device).stream();
  PyObject* h = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
  if (!h) throw Refused{""};  // the attribute's own error stands
  const unsigned long long v = PyLong_AsUnsignedLongLong(h);
  Py_DECREF(h);
  if (v == (unsigned long long)-1 && PyErr_Occurred()) throw Refused{""};
  return reinterpret_cast<void*>(v);
}

int as_int(PyObject* o, const char* name) {
  int overflow = 0;
  const long v = PyLong_AsLongAndOverflow(o, &overflow);
  if (v == -1 && PyErr_Occurred()) throw Refused{""};
  if (overflow || v < INT32_MIN || v > INT32_MAX) throw Refused{std::string(name) + " does not fit 32 bits"};
  return (int)v;
}

int count(int64_t n, const char* name) {
  if (n > INT32_MAX) throw Refused{std::string(name) + " does not fit 32 bits"};
  return (int)n;
}

template <typename F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, PyObject* cap, F call) {
  if (got != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", got, want);
    return nullptr;
  }
  State* s = static_cast<State*>(PyCapsule_GetPointer(cap, "sf_cache_state"));
  if (!s) return nullptr;
  try {
    return PyLong_FromLong(call(*s));
  } catch (const Refused& r) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, r.text.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// state, qkv, index, table, k_pages, v_pages, pos, seq, q_gain, k_gain, q, stream
PyObject* py_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, n ? a[0] : Py_None, [&](const State& s) -> int {
    const Rows x = rows(s, a[1], "qkv", s.nq + 2 * s.nkv), q = rows(s, a[10], "q", s.nq);
    if (q.n != x.n) throw Refused{"q has " + std::to_string(q.n) + " rows, qkv " + std::to_string(x.n)};
    const int64_t T[1] = {x.n}, hd[1] = {s.hd};
    const Table t = table(s, a[3], "table");
    const Pools p = pools(s, a[4], a[5]);
    const void* index = fixed(s, a[2], "index", at::kInt, T);
    const void* pos = fixed(s, a[6], "pos", at::kInt, T, true);
    const void* seq = fixed(s, a[7], "seq", at::kInt, T, true);
    const void* qg = fixed(s, a[8], "q_gain", at::kFloat, hd, true);
    const void* kg = fixed(s, a[9], "k_gain", at::kFloat, hd, true);
    return sf_cache_append(s.cache, stream_of(s, a[11]), x.p, x.ld, count(x.n, "T"), (const float*)qg, (const float*)kg,
                           (const int32_t*)index, (const int32_t*)pos, (const int32_t*)seq, t.p, count(t.S, "S"),
                           count(t.cols, "columns"), t.ld, p.k, p.v, p.pages, q.p, q.ld);
  });
}

// state, q, k_pages, v_pages, table, lens, scale, out, weights, weights_out, stream
PyObject* py_attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, n ? a[0] : Py_None, [&](const State& s) -> int {
    const Table t = table(s, a[4], "table");
    const Rows q = rows(s, a[1], "q", s.nq), out = rows(s, a[7], "out", s.nq);
    if (q.n != t.S || out.n != t.S)
      throw Refused{"q has " + std::to_string(q.n) + " rows, out " + std::to_string(out.n) + ", table " +
                    std::to_string(t.S)};
    const Pools p = pools(s, a[2], a[3]);
    const int64_t S[1] = {t.S};
    const void* lens = fixed(s, a[5], "lens", at::kInt, S);
    const double scale = PyFloat_AsDouble(a[6]);
    if (scale == -1.0 && PyErr_Occurred()) throw Refused{""};
    int64_t ld_w = 0;
    const void* w_in = nullptr;
    void* w_out = nullptr;
    if (a[9] != Py_None) {
      const at::Tensor& w = tensor(a[9], "weights_out");
      ld_w = w.dim() == 3 ? w.size(2) : 0;
      const int64_t shape[3] = {t.S, s.nkv, ld_w};
      w_out = fixed(s, a[9], "weights_out", at::kFloat, shape);
      w_in = fixed(s, a[8], "weights", at::kFloat, shape, true);
    }
    return sf_cache_attend(s.cache, stream_of(s, a[10]), q.p, q.ld, p.k, p.v, p.pages, t.p, count(t.S, "S"),
                           count(t.cols, "columns"), t.ld, (const int32_t*)lens, (float)scale, out.p, out.ld,
                           (const float*)w_in, (float*)w_out, ld_w);
  });
}

double as_double(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{""};
  return v;
}

// state, k_pages, table, lens, pos_from, pos_to, stream
PyObject* py_reposition(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, n ? a[0] : Py_None, [&](const State& s) -> int {
    const Table t = table(s, a[2], "table");
    const Pools p = pools(s, a[1], a[1]);
    const int64_t S[1] = {t.S};
    const void* lens = fixed(s, a[3], "lens", at::kInt, S);
    const at::Tensor& ft = tensor(a[4], "pos_from");
    const int64_t shape[3] = {t.S, s.nkv, ft.dim() == 3 ? ft.size(2) : 0};
    const void* from = fixed(s, a[4], "pos_from", at::kInt, shape);
    const void* to = fixed(s, a[5], "pos_to", at::kInt, shape, true);
    return sf_cache_reposition(s.cache, stream_of(s, a[6]), p.k, p.pages, t.p, count(t.S, "S"), count(t.cols, "columns"),
                               t.ld, (const int32_t*)lens, (const int32_t*)from, (const int32_t*)to, shape[2]);
  });
}

// state, q, k_pages, v_pages, table, lens, starts, scale, out, lse, stream
PyObject* py_attend_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, n ? a[0] : Py_None, [&](const State& s) -> int {
    const Table t = table(s, a[4], "table");
    const Rows q = rows(s, a[1], "q", s.nq), out = rows(s, a[8], "out", s.nq);
    if (out.n != q.n) throw Refused{"out has " + std::to_string(out.n) + " rows, q " + std::to_string(q.n)};
    const Pools p = pools(s, a[2], a[3]);
    const int64_t S[1] = {t.S}, S1[1] = {t.S + 1}, ls[2] = {q.n, s.nq};
    const void* lens = fixed(s, a[5], "lens", at::kInt, S);
    const void* starts = fixed(s, a[6], "starts", at::kInt, S1);
    void* lse = fixed(s, a[9], "lse", at::kFloat, ls, true);
    return sf_cache_attend_rows(s.cache, stream_of(s, a[10]), q.p, q.ld, count(q.n, "T"), p.k, p.v, p.pages, t.p,
                                count(t.S, "S"), count(t.cols, "columns"), t.ld, (const int32_t*)lens,
                                (const int32_t*)starts, (float)as_double(a[7]), out.p, out.ld, (float*)lse);
  });
}

// state, q, k_pages, v_pages, table, lens, prefix_table, prefix_lens, starts, scale, out, lse, stream
PyObject* py_attend_shared(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, n ? a[0] : Py_None, [&](const State& s) -> int {
    const Table t = table(s, a[4], "table"), pt = table(s, a[6], "prefix_table");
    const Rows q = rows(s, a[1], "q", s.nq), out = rows(s, a[10], "out", s.nq);
    if (q.n != t.S || out.n != t.S)
      throw Refused{"q has " + std::to_string(q.n) + " rows, out " + std::to_string(out.n) + ", table " +
                    std::to_string(t.S)};
    const Pools p = pools(s, a[2], a[3]);
    const int64_t S[1] = {t.S}, G[1] = {pt.S}, G1[1] = {pt.S + 1}, ls[2] = {q.n, s.nq};
    const void* lens = fixed(s, a[5], "lens", at::kInt, S);
    const void* plens = fixed(s, a[7], "prefix_lens", at::kInt, G);
    const void* starts = fixed(s, a[8], "starts", at::kInt, G1);
    void* lse = fixed(s, a[11], "lse", at::kFloat, ls, true);
    return sf_cache_attend_shared(s.cache, stream_of(s, a[12]), q.p, q.ld, p.k, p.v, p.pages, t.p, count(t.S, "S"),
                                  count(t.cols, "columns"), t.ld, (const int32_t*)lens, pt.p, count(pt.S, "G"),
                                  count(pt.cols, "prefix columns"), pt.ld, (const int32_t*)plens,
                                  (const int32_t*)starts, (float)as_double(a[9]), out.p, out.ld, (float*)lse);
  });
}

// state, k_pages, v_pages, table, lens, weights, budget, n_first, n_recent, k_out, v_out, table_out, weights_out,
// lens_out, kept, stream
PyObject* py_evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 16, n ? a[0] : Py_None, [&](const State& s) -> int {
    const Table t = table(s, a[3], "table"), to = table(s, a[11], "table_out");
    if (to.S != t.S) throw Refused{"table_out has " + std::to_string(to.S) + " rows, table " + std::to_string(t.S)};
    const Pools p = pools(s, a[1], a[2]), po = pools(s, a[9], a[10], "k_out", "v_out");
    const int budget = as_int(a[6], "budget"), first = as_int(a[7], "n_first"), recent = as_int(a[8], "n_recent");
    const at::Tensor& wt = tensor(a[5], "weights");
    const int64_t ld_w = wt.dim() == 3 ? wt.size(2) : 0;
    const int64_t shape[3] = {t.S, s.nkv, ld_w}, S[1] = {t.S}, kept_shape[3] = {t.S, s.nkv, budget > 0 ? budget : 0};
    const void* w = fixed(s, a[5], "weights", at::kFloat, shape);
    void* w_out = fixed(s, a[12], "weights_out", at::kFloat, shape);
    const void* lens = fixed(s, a[4], "lens", at::kInt, S);
    void* lens_out = fixed(s, a[13], "lens_out", at::kInt, S);
    void* kept = fixed(s, a[14], "kept", at::kInt, kept_shape);
    return sf_cache_evict(s.cache, stream_of(s, a[15]), p.k, p.v, p.pages, t.p, count(t.S, "S"),
                          count(t.cols, "columns"), t.ld, (const int32_t*)lens, (const float*)w, ld_w, budget, first,
                          recent, po.k, po.v, po.pages, to.p, count(to.cols, "columns"), to.ld, (float*)w_out,
                          (int32_t*)lens_out, (int32_t*)kept);
  });
}

// cache (address), device, is_bf16, n_q_heads, n_kv_heads, head_dim, page_size
PyObject* py_state(PyObject*, PyObject* args) {
  unsigned long long cache;
  int device, bf16;
  long long nq, nkv, hd, page;
  if (!PyArg_ParseTuple(args, "KiiLLLL", &cache, &device, &bf16, &nq, &nkv, &hd, &page)) return nullptr;
  State* s = new (std::nothrow) State{reinterpret_cast<sf_cache*>(cache), device, bf16 ? at::kBFloat16 : at::kFloat,
                                      nq, nkv, hd, page};
  if (!s) return PyErr_NoMemory();
  PyObject* cap = PyCapsule_New(s, "sf_cache_state", free_state);
  if (!cap) delete s;
  return cap;
}

PyMethodDef methods[] = {
    {"state", py_state, METH_VARARGS, "Checks' view of a cache object."},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_append)), METH_FASTCALL, "sf_cache_append"},
    {"attend", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_attend)), METH_FASTCALL, "sf_cache_attend"},
    {"reposition", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_reposition)), METH_FASTCALL,
     "sf_cache_reposition"},
    {"attend_rows", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_attend_rows)), METH_FASTCALL,
     "sf_cache_attend_rows"},
    {"attend_shared", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_attend_shared)), METH_FASTCALL,
     "sf_cache_attend_shared"},
    {"evict", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_evict)), METH_FASTCALL, "sf_cache_evict"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_sf_torch", "Marshalling of the paged-cache calls.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__sf_torch(void) { return PyModule_Create(&module); }
