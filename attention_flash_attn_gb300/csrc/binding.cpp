// binding.cpp -- the calls of cache.py: argument checks, outputs and scratch, and the call into
// include/attn_cache_gb300.h.  A decoding step makes these calls once per layer, and in Python their checks
// and allocations alone took longer than the kernels (22 us an attention call, 14 an append; compiled, an
// append takes 6 us from call to call, its kernel included).
//
// Every function takes the address of the handle's attn_cache and the handle's k tensor (for its device)
// first.  Errors are those of the binding: TypeError, ValueError, and AttnError for a status.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdio>
#include <string>
#include <utility>

#include "../../include/attn_cache_gb300.h"

namespace {

// A Python exception that is already set.
struct Raised {};

[[noreturn]] void raise(PyObject *type, const char *fmt, ...) {
  char text[400];
  va_list v;
  va_start(v, fmt);
  vsnprintf(text, sizeof(text), fmt, v);
  va_end(v);
  PyErr_SetString(type, text);
  throw Raised{};
}

void check_status(int status, const char *where) {
  if (status == ATTN_OK) return;
  PyObject *mod = PyImport_ImportModule("attention_flash_attn_gb300._capi");
  PyObject *cls = mod ? PyObject_GetAttrString(mod, "AttnError") : nullptr;
  PyObject *err = cls ? PyObject_CallFunction(cls, "is", status, where) : nullptr;
  if (err) PyErr_SetObject(cls, err);
  Py_XDECREF(err);
  Py_XDECREF(cls);
  Py_XDECREF(mod);
  throw Raised{};
}

std::string shape_of(const at::Tensor &t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + (t.dim() == 1 ? ",)" : ")");
}

const at::Tensor &tensor(const char *where, const char *name, PyObject *o) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s: %s must be a tensor", where, name);
  return THPVariable_Unpack(o);
}
int64_t whole(PyObject *o) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw Raised{};
  return x;
}
int whole32(const char *where, const char *name, PyObject *o) {
  const int64_t x = whole(o);
  if (x > INT32_MAX || x < INT32_MIN) raise(PyExc_ValueError, "%s: %s is out of range", where, name);
  return (int)x;
}
double real(PyObject *o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw Raised{};
  return x;
}
bool truth(PyObject *o) {
  const int x = PyObject_IsTrue(o);
  if (x < 0) throw Raised{};
  return x != 0;
}

struct Cache {
  const attn_cache *c;
  const at::Tensor &k;
  Cache(PyObject *addr, PyObject *k) : c(static_cast<const attn_cache *>(PyLong_AsVoidPtr(addr))), k(tensor("AttnCache", "k", k)) {
    if (!c && PyErr_Occurred()) throw Raised{};
  }
  c10::Device device() const { return k.device(); }
};

void same_device(const char *where, const Cache &c, const at::Tensor &t) {
  if (t.device() != c.device())
    raise(PyExc_ValueError, "%s: every tensor must be on %s (got one on %s)", where, c.device().str().c_str(), t.device().str().c_str());
}

// Stride of a dimension, 0 where it is never taken (PyTorch leaves any number there).
int64_t stride(const at::Tensor &t, int d) { return t.size(d) > 1 ? t.stride(d) : 0; }

// [B, S, H, D] rows in bfloat16 or float32 with the head dimension dense; returns the dtype code.
int rows(const char *where, const char *name, const at::Tensor &t, const Cache &c) {
  const auto ty = t.scalar_type();
  if (ty != at::kBFloat16 && ty != at::kFloat) raise(PyExc_TypeError, "%s: %s must be bfloat16 or float32", where, name);
  if (t.dim() != 4 || t.size(3) != c.c->D)
    raise(PyExc_ValueError, "%s: %s must be [B, S, H, D] with the cache's D = %d, got %s", where, name, c.c->D, shape_of(t).c_str());
  if (t.stride(3) != 1) raise(PyExc_ValueError, "%s: the head dimension of %s must be contiguous", where, name);
  same_device(where, c, t);
  for (int d = 0; d < 3; ++d)
    if (t.size(d) > INT32_MAX) raise(PyExc_ValueError, "%s: %s is too large", where, name);
  return ty == at::kBFloat16 ? ATTN_DTYPE_BF16 : ATTN_DTYPE_F32;
}

void ints(const char *where, const char *name, const at::Tensor &t, int64_t B, const Cache &c) {
  if (t.scalar_type() != at::kInt || t.dim() != 1 || t.size(0) != B || !t.is_contiguous())
    raise(PyExc_ValueError, "%s: %s must be a contiguous int32 tensor of %lld entries, got %s %s", where, name, (long long)B,
          toString(t.scalar_type()), shape_of(t).c_str());
  same_device(where, c, t);
}

void page_table(const char *where, const char *name, const at::Tensor &t, int64_t B, int64_t pages, const Cache &c) {
  if (t.dim() != 2 || t.size(0) != B || t.size(1) < pages || t.size(1) > INT32_MAX || t.scalar_type() != at::kInt)
    raise(PyExc_ValueError, "%s: %s must be int32 [%lld, %s%lld pages], got %s %s", where, name, (long long)B, "at least ",
          (long long)pages, toString(t.scalar_type()), shape_of(t).c_str());
  if ((t.stride(1) != 1 && t.size(1) > 1) || (t.stride(0) < t.size(1) && B > 1))
    raise(PyExc_ValueError, "%s: the rows of %s must be dense and not overlap", where, name);
  same_device(where, c, t);
}

attn_cache_seqs sequences(const char *where, const Cache &c, int64_t B, const at::Tensor &table, const at::Tensor &lengths) {
  page_table(where, "table", table, B, 0, c);
  ints(where, "lengths", lengths, B, c);
  return {(int)B, (int)table.size(1), static_cast<const int32_t *>(table.data_ptr()), table.stride(0),
          static_cast<const int32_t *>(lengths.data_ptr())};
}

void weight_rows(const char *where, const char *name, const at::Tensor &t, int64_t B, int64_t room, const Cache &c) {
  if (t.dim() != 3 || t.scalar_type() != at::kFloat || t.size(0) != B || t.size(1) != c.c->Hkv || t.size(2) < room ||
      (t.stride(2) != 1 && t.size(2) > 1))
    raise(PyExc_ValueError, "%s: %s must be float32 [%lld, %d, at least %lld] with dense rows, got %s %s", where, name, (long long)B,
          c.c->Hkv, (long long)room, toString(t.scalar_type()), shape_of(t).c_str());
  same_device(where, c, t);
}

// Weights that a call writes: rows of [B, Hkv] that keep off one another in their first `room` elements.
void written_rows(const char *where, const char *name, const at::Tensor &t, int64_t B, int64_t room, const Cache &c) {
  weight_rows(where, name, t, B, room, c);
  int64_t n[2] = {t.size(0), t.size(1)}, s[2] = {t.stride(0), t.stride(1)};
  if (s[0] < s[1]) {
    std::swap(n[0], n[1]);
    std::swap(s[0], s[1]);
  }
  if ((n[1] > 1 && s[1] < room) || (n[0] > 1 && s[0] < (n[1] > 1 ? (n[1] - 1) * s[1] : 0) + room))
    raise(PyExc_ValueError, "%s: the rows of %s must not overlap", where, name);
}

// A given output, checked, or a new one.
at::Tensor output(const char *where, const char *name, PyObject *o, at::IntArrayRef shape, at::ScalarType ty, const Cache &c) {
  if (o == Py_None) return at::empty(shape, at::TensorOptions().dtype(ty).device(c.device()));
  const at::Tensor &t = tensor(where, name, o);
  if (t.sizes() != shape || t.scalar_type() != ty || !t.is_contiguous()) {
    std::string want = "(";
    for (size_t i = 0; i < shape.size(); ++i) want += (i ? ", " : "") + std::to_string(shape[i]);
    raise(PyExc_ValueError, "%s: %s must be a contiguous %s tensor of shape %s), got %s %s", where, name, toString(ty), want.c_str(),
          toString(t.scalar_type()), shape_of(t).c_str());
  }
  same_device(where, c, t);
  return t;
}

// The current stream of the cache's device, which is made current while this lives.
struct On {
  c10::cuda::OptionalCUDAGuard guard;
  attn_stream_t stream;
  explicit On(const Cache &c) {
    if (!c.device().is_cuda()) raise(PyExc_ValueError, "AttnCache: the cache must be on a CUDA device");
    if (c.device().index() != c10::cuda::current_device()) guard.set_index(c.device().index());
    stream = reinterpret_cast<attn_stream_t>(c10::cuda::getCurrentCUDAStream(c.device().index()).stream());
  }
};

void need_args(const char *where, Py_ssize_t n, Py_ssize_t want) {
  if (n != want) raise(PyExc_TypeError, "%s: %zd arguments instead of %zd", where, n, want);
}

PyObject *wrap(std::initializer_list<at::Tensor> ts) {
  PyObject *t = PyTuple_New((Py_ssize_t)ts.size());
  if (!t) throw Raised{};
  Py_ssize_t i = 0;
  for (const at::Tensor &x : ts) {
    PyObject *o = THPVariable_Wrap(x);
    if (!o) {
      Py_DECREF(t);
      throw Raised{};
    }
    PyTuple_SET_ITEM(t, i++, o);
  }
  return t;
}

// append(addr, cache_k, k, v, table, lengths, counts, weights) -> lengths
PyObject *append(PyObject *const *a, Py_ssize_t n) {
  const char *where = "attn_cache_append";
  need_args(where, n, 8);
  const Cache c(a[0], a[1]);
  const at::Tensor &k = tensor(where, "k", a[2]), &v = tensor(where, "v", a[3]);
  attn_cache_append_args g = {};
  g.dtype = rows(where, "k", k, c);
  if (rows(where, "v", v, c) != g.dtype) raise(PyExc_TypeError, "%s: k and v must share a dtype", where);
  if (v.sizes() != k.sizes()) raise(PyExc_ValueError, "%s: v must be %s, got %s", where, shape_of(k).c_str(), shape_of(v).c_str());
  if (k.size(2) != c.c->Hkv)
    raise(PyExc_ValueError, "%s: k and v must have the cache's %d heads, got %lld", where, c.c->Hkv, (long long)k.size(2));
  const int64_t B = k.size(0);
  const at::Tensor &table = tensor(where, "table", a[4]), &lengths = tensor(where, "lengths", a[5]);
  const attn_cache_seqs s = sequences(where, c, B, table, lengths);
  g.S = (int)k.size(1);
  g.k = k.data_ptr();
  g.v = v.data_ptr();
  g.k_stride_b = stride(k, 0); g.k_stride_s = stride(k, 1); g.k_stride_h = stride(k, 2);
  g.v_stride_b = stride(v, 0); g.v_stride_s = stride(v, 1); g.v_stride_h = stride(v, 2);
  if (a[6] != Py_None) {
    const at::Tensor &t = tensor(where, "counts", a[6]);
    ints(where, "counts", t, B, c);
    g.counts = static_cast<const int32_t *>(t.data_ptr());
  }
  if (a[7] != Py_None) {
    const at::Tensor &t = tensor(where, "weights", a[7]);
    written_rows(where, "weights", t, B, (int64_t)s.max_pages * c.c->page_size, c);
    g.weights = static_cast<float *>(t.data_ptr());
    g.weights_stride_b = t.stride(0);
    g.weights_stride_h = t.stride(1);
  }
  const On on(c);
  const at::Tensor out = at::empty_like(lengths);
  g.lengths_out = static_cast<int32_t *>(out.data_ptr());
  check_status(attn_cache_append(c.c, &s, &g, on.stream), where);
  return THPVariable_Wrap(out);
}

// q, table, lengths, causal, window, softcap, sink, off_by_one, scale, weights, weights_out from a[2] on
void fwd_args(const char *where, const Cache &c, PyObject *const *a, attn_cache_seqs *s, attn_cache_fwd_args *g) {
  const at::Tensor &q = tensor(where, "q", a[2]);
  g->dtype = rows(where, "q", q, c);
  const int64_t B = q.size(0), Hq = q.size(2);
  if (Hq % c.c->Hkv) raise(PyExc_ValueError, "%s: q's %lld heads must be a multiple of the cache's %d", where, (long long)Hq, c.c->Hkv);
  *s = sequences(where, c, B, tensor(where, "table", a[3]), tensor(where, "lengths", a[4]));
  g->Sq = (int)q.size(1);
  g->Hq = (int)Hq;
  g->q = q.data_ptr();
  g->q_stride_b = stride(q, 0); g->q_stride_s = stride(q, 1); g->q_stride_h = stride(q, 2);
  g->causal = truth(a[5]);
  g->window = whole32(where, "window", a[6]);
  g->softcap = (float)real(a[7]);
  if (a[8] != Py_None) {
    const at::Tensor &t = tensor(where, "sink", a[8]);
    if (t.numel() != Hq || t.scalar_type() != at::kFloat || !t.is_contiguous())
      raise(PyExc_ValueError, "%s: sink must hold one float32 logit per query head [%lld]", where, (long long)Hq);
    same_device(where, c, t);
    g->sink = static_cast<const float *>(t.data_ptr());
  }
  g->softmax_type = truth(a[9]) ? ATTN_SOFTMAX_OFF_BY_ONE : ATTN_SOFTMAX_DEFAULT;
  g->scale = a[10] == Py_None ? (float)(1.0 / std::sqrt((double)c.c->D)) : (float)real(a[10]);
  if (a[11] != Py_None) {
    const int64_t room = (int64_t)s->max_pages * c.c->page_size;
    const at::Tensor &w = tensor(where, "weights", a[11]);
    weight_rows(where, "weights", w, B, room, c);
    const at::Tensor &o = a[12] == Py_None ? w : tensor(where, "weights_out", a[12]);
    written_rows(where, "weights_out", o, B, room, c);
    for (int d = 0; d < 2; ++d)
      if (stride(w, d) != stride(o, d)) raise(PyExc_ValueError, "%s: weights and weights_out must have the same strides", where);
    g->weights = static_cast<const float *>(w.data_ptr());
    g->weights_out = static_cast<float *>(o.data_ptr());
    g->weights_stride_b = stride(w, 0);
    g->weights_stride_h = stride(w, 1);
  } else if (a[12] != Py_None) {
    raise(PyExc_ValueError, "%s: weights_out needs weights", where);
  }
}

// fwd(addr, cache_k, <fwd_args>, out, lse) -> (O, LSE)
PyObject *fwd(PyObject *const *a, Py_ssize_t n) {
  const char *where = "attn_cache_fwd";
  need_args(where, n, 15);
  const Cache c(a[0], a[1]);
  attn_cache_seqs s;
  attn_cache_fwd_args g = {};
  fwd_args(where, c, a, &s, &g);
  const at::Tensor &q = THPVariable_Unpack(a[2]);
  const at::Tensor O = output(where, "out", a[13], q.sizes(), q.scalar_type(), c);
  const at::Tensor LSE = output(where, "lse", a[14], {q.size(0), q.size(2), q.size(1)}, at::kFloat, c);
  const On on(c);
  const size_t need = attn_cache_fwd_workspace_size(c.c, &s, &g);
  if (need == 0) {  // refused: the call itself says why
    check_status(attn_cache_fwd(c.c, &s, &g, O.data_ptr(), static_cast<float *>(LSE.data_ptr()), nullptr, 0, on.stream), where);
    check_status(ATTN_ERR_INVALID, where);
  }
  // Scratch of this call alone: the caching allocator hands it on in stream order, and inside a graph
  // capture it belongs to that graph.
  const at::Tensor ws = at::empty({(int64_t)need}, at::TensorOptions().dtype(at::kByte).device(c.device()));
  check_status(attn_cache_fwd(c.c, &s, &g, O.data_ptr(), static_cast<float *>(LSE.data_ptr()), ws.data_ptr(), need, on.stream), where);
  return wrap({O, LSE});
}

// path(addr, cache_k, <fwd_args>) -> str
PyObject *path(PyObject *const *a, Py_ssize_t n) {
  const char *where = "attn_cache_path_name";
  need_args(where, n, 13);
  const Cache c(a[0], a[1]);
  attn_cache_seqs s;
  attn_cache_fwd_args g = {};
  fwd_args(where, c, a, &s, &g);
  return PyUnicode_FromString(attn_cache_path_name(c.c, &s, &g));
}

// evict(addr, cache_k, table, lengths, weights, table_out, keep, recent, first, kept, weights_out)
//   -> (kept, lengths, weights)
PyObject *evict(PyObject *const *a, Py_ssize_t n) {
  const char *where = "attn_cache_evict";
  need_args(where, n, 11);
  const Cache c(a[0], a[1]);
  const at::Tensor &table = tensor(where, "table", a[2]), &lengths = tensor(where, "lengths", a[3]);
  const int64_t B = lengths.numel();
  const attn_cache_seqs s = sequences(where, c, B, table, lengths);
  attn_cache_evict_args g = {};
  g.keep = whole32(where, "keep", a[6]);
  g.recent = whole32(where, "recent", a[7]);
  g.first = whole32(where, "first", a[8]);
  if (g.keep < 1 || g.recent < 0 || g.first < 0 || (int64_t)g.first + g.recent > g.keep)
    raise(PyExc_ValueError, "%s: keep must be at least 1 and at least first + recent", where);
  const at::Tensor &w = tensor(where, "weights", a[4]);
  weight_rows(where, "weights", w, B, (int64_t)s.max_pages * c.c->page_size, c);
  const at::Tensor &to = tensor(where, "table_out", a[5]);
  page_table(where, "table_out", to, B, ((int64_t)g.keep + c.c->page_size - 1) / c.c->page_size, c);
  const int64_t shape[3] = {B, c.c->Hkv, g.keep};
  const at::Tensor kept = output(where, "kept", a[9], shape, at::kInt, c);
  // A given one may have wider rows: those that the sequences' next calls take.
  const at::Tensor w_out = a[10] == Py_None ? output(where, "weights_out", a[10], shape, at::kFloat, c) : tensor(where, "weights_out", a[10]);
  written_rows(where, "weights_out", w_out, B, g.keep, c);
  const On on(c);
  const at::Tensor n_out = at::empty_like(lengths);
  g.weights = static_cast<const float *>(w.data_ptr());
  g.weights_stride_b = w.stride(0);
  g.weights_stride_h = w.stride(1);
  g.table_out = static_cast<const int32_t *>(to.data_ptr());
  g.table_out_stride = to.stride(0);
  g.kept = static_cast<int32_t *>(kept.data_ptr());
  g.lengths_out = static_cast<int32_t *>(n_out.data_ptr());
  g.weights_out = static_cast<float *>(w_out.data_ptr());
  g.weights_out_stride_b = w_out.stride(0);
  g.weights_out_stride_h = w_out.stride(1);
  check_status(attn_cache_evict(c.c, &s, &g, on.stream), where);
  return wrap({kept, n_out, w_out});
}

template <PyObject *(*F)(PyObject *const *, Py_ssize_t)> PyObject *entry(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    return F(a, n);
  } catch (const Raised &) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject *(*F)(PyObject *const *, Py_ssize_t)> PyMethodDef method(const char *name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(entry<F>)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method<append>("append"), method<fwd>("fwd"), method<path>("path"), method<evict>("evict"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
