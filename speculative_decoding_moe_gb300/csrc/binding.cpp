// binding.cpp -- the hot calls of the tree-verify binding as a CPython extension:
// argument checks, result allocation and the C ABI call in one step.
//
// A decode step makes dozens of these calls, and checking and marshalling one in
// Python took longer than its kernels: 18 us for an attention call whose kernels
// take 10, and 5.5 here, of which two launches and two tensor maps are 4.0 and the
// result's allocation 1.4 (a rotary call 3.6, of which the result's 1.3 and the
// stream's look-up 0.2).  Tensors are read through ATen, results allocated by torch's allocator; everything else
// goes through include/dfv.h as for any other caller.  Refusals are the binding's
// own TypeError and ValueError, a status of the library is its DfvError.
#include <Python.h>

#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <exception>
#include <optional>
#include <string>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/dfv.h"

namespace {

// The Python side's handles: the C descriptors, and what the checks need.
struct Cache {
  dfv_kv_cache c;
  int index;  // device
};
struct Tree {
  dfv_tree_batch c;
  int index;
};
struct Rules {
  dfv_logit_rules c;
  int n_seqs, index;                               // -1 / -2: none given
  int bias_rows, allowed_rows;                     // 0: none
  int64_t bias_cols, allowed_cols;
};

struct Refused {};  // a Python exception is set

std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + (s.size() == 1 ? ",)" : ")");
}

[[noreturn]] void value_error(const char *fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  PyErr_SetString(PyExc_ValueError, buf);
  throw Refused();
}

const at::Tensor &tensor(PyObject *o, const char *what) {
  if (!THPVariable_Check(o)) {
    if (o == Py_None) value_error("%s is missing", what);
    PyErr_Format(PyExc_TypeError, "%s must be a tensor, got %s", what, Py_TYPE(o)->tp_name);
    throw Refused();
  }
  return THPVariable_Unpack(o);
}

void check(const at::Tensor &t, const char *what, at::ScalarType dt, at::IntArrayRef shape, int index) {
  if (t.scalar_type() != dt) {
    PyErr_Format(PyExc_TypeError, "%s must be %s, got %s", what, at::toString(dt), at::toString(t.scalar_type()));
    throw Refused();
  }
  if (t.sizes() != shape)
    value_error("%s must have shape %s, got %s", what, shape_text(shape).c_str(), shape_text(t.sizes()).c_str());
  if (t.get_device() != index) value_error("%s is on %s, not with the other tensors of the call", what, t.device().str().c_str());
}

// Address of a contiguous tensor of this type, shape and device.
void *need(PyObject *o, const char *what, at::ScalarType dt, at::IntArrayRef shape, int index) {
  const at::Tensor &t = tensor(o, what);
  check(t, what, dt, shape, index);
  if (!t.is_contiguous()) value_error("%s must be contiguous", what);
  return t.data_ptr();
}
void *given(PyObject *o, const char *what, at::ScalarType dt, at::IntArrayRef shape, int index) {
  return o == Py_None ? nullptr : need(o, what, dt, shape, index);
}

// A [rows, heads, dim] tensor whose last dimension is contiguous.
struct Rows3 {
  void *p;
  int64_t row, head;
};
Rows3 rows3(const at::Tensor &t, const char *what, int64_t rows, int64_t heads, int64_t dim, at::ScalarType dt, int index) {
  check(t, what, dt, {rows, heads, dim}, index);
  if (t.stride(2) != 1) value_error("%s must be contiguous in its last dimension", what);
  // a dimension of size 1 has no stride of its own
  return {t.data_ptr(), rows > 1 ? t.stride(0) : 0, heads > 1 ? t.stride(1) : 0};
}

// The last check before a launch: host tensors pass the ones of type and shape.
void on_gpu(int index) {
  if (index < 0) value_error("the tensors of the call must be CUDA tensors");
}
// A result, from torch's allocator without its dispatcher (1.3 us instead of 1.8), in
// the memory of the call's stream: a block of another stream's may still be in use
// there, and would be handed out there again before this call ends.
at::Tensor empty(at::IntArrayRef shape, at::ScalarType dt, const at::Tensor &like, void *stream) {
  const int index = (int)like.get_device();
  on_gpu(index);
  std::optional<c10::cuda::CUDAStreamGuard> there;
  if (c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream() != stream)
    there.emplace(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(stream), (c10::DeviceIndex)index));
  return at::Tensor(at::detail::empty_cuda(shape, dt, like.device(), std::nullopt));
}

template <class T>
const T &handle(PyObject *o) {
  void *p = PyLong_AsVoidPtr(o);
  if (!p) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "handle is NULL");
    throw Refused();
  }
  return *static_cast<const T *>(p);
}
long long whole(PyObject *o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}
int number(PyObject *o) {
  const long long v = whole(o);
  if (v < INT32_MIN || v > INT32_MAX) value_error("%lld does not fit 32 bits", v);
  return (int)v;
}
double real(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return v;
}
void *stream(PyObject *o) {
  void *p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw Refused();
  return p;
}
at::ScalarType type_of(const Cache &c) { return c.c.dtype == DFV_F16 ? at::kHalf : at::kBFloat16; }

// A workspace of this device (its size and alignment are the library's checks).
struct Space {
  void *p;
  size_t n;
};
Space space(PyObject *o, int index) {
  const at::Tensor &t = tensor(o, "ws");
  if (t.get_device() != index || !t.is_contiguous()) value_error("ws must be contiguous, on the device of the other tensors");
  return {t.data_ptr(), t.nbytes()};
}
void together(const Cache &c, const Tree &t) {
  if (c.index != t.index) value_error("cache and tree are not on one device");
}

// Raises DfvError(status, where) of the Python module unless the status is 0.
void done(int status, const char *where) {
  if (status == DFV_OK) return;
  PyObject *m = PyImport_ImportModule("speculative_decoding_moe_gb300.dfv");
  PyObject *cls = m ? PyObject_GetAttrString(m, "DfvError") : nullptr;
  PyObject *e = cls ? PyObject_CallFunction(cls, "is", status, where) : nullptr;
  if (e) PyErr_SetObject(cls, e);
  Py_XDECREF(e);
  Py_XDECREF(cls);
  Py_XDECREF(m);
  throw Refused();
}

PyObject *same(PyObject *o) {
  Py_INCREF(o);
  return o;
}

// (cache, layer, tree, plan's head_dim, rot_dim, interleaved, scale, turns, q, k, v, positions, out, stream, plan's
// device)
PyObject *rope_append(PyObject *const *a) {
  const Cache &c = handle<Cache>(a[0]);
  const int layer = number(a[1]);
  const Tree &t = handle<Tree>(a[2]);
  together(c, t);
  const at::Tensor &q = tensor(a[8], "q"), &k = tensor(a[9], "k"), &v = tensor(a[10], "v");
  const int64_t rows = t.c.n_rows, H = q.dim() == 3 ? q.size(1) : 0, K = c.c.n_kv_heads, D = c.c.head_dim;
  const at::ScalarType dt = type_of(c);
  const Rows3 rq = rows3(q, "q", rows, H, D, dt, c.index), rk = rows3(k, "k", rows, K, D, dt, c.index),
              rv = rows3(v, "v", rows, K, D, dt, c.index);
  const void *pos = need(a[11], "positions", at::kInt, {rows}, c.index);
  if (number(a[3]) != D) value_error("the rotary plan is for head_dim %d, the cache has %d", number(a[3]), (int)D);
  if (number(a[14]) != c.index) value_error("the rotary plan and the cache are not on one device");
  at::Tensor made;
  if (a[12] == Py_None) made = empty({rows, H, D}, dt, q, stream(a[13]));
  const Rows3 ro = rows3(made.defined() ? made : tensor(a[12], "out"), "out", rows, H, D, dt, c.index);
  on_gpu(c.index);
  done(dfv_rope_append(&c.c, layer, &t.c, (int)H, number(a[4]), number(a[5]), (float)real(a[6]),
                       static_cast<const uint64_t *>(stream(a[7])), rq.p, rq.row, rq.head, rk.p, rk.row, rk.head, rv.p,
                       rv.row, rv.head, static_cast<const int32_t *>(pos), ro.p, ro.row, ro.head, stream(a[13])),
       "dfv_rope_append");
  return made.defined() ? THPVariable_Wrap(made) : same(a[12]);
}

// (cache, layer, tree, q, ws, scale or None, out, lse, stream)
PyObject *tree_attention(PyObject *const *a) {
  const Cache &c = handle<Cache>(a[0]);
  const int layer = number(a[1]);
  const Tree &t = handle<Tree>(a[2]);
  together(c, t);
  const at::Tensor &q = tensor(a[3], "q");
  const int64_t rows = t.c.n_rows, H = q.dim() == 3 ? q.size(1) : 0, D = c.c.head_dim;
  const at::ScalarType dt = type_of(c);
  const Rows3 rq = rows3(q, "q", rows, H, D, dt, c.index);
  const Space ws = space(a[4], c.index);
  void *lse = given(a[7], "lse", at::kFloat, {rows, H}, c.index);
  const double scale = a[5] == Py_None ? 1.0 / std::sqrt((double)D) : real(a[5]);
  at::Tensor made;
  if (a[6] == Py_None) made = empty({rows, H, D}, dt, q, stream(a[8]));
  const Rows3 ro = rows3(made.defined() ? made : tensor(a[6], "out"), "out", rows, H, D, dt, c.index);
  on_gpu(c.index);
  done(dfv_tree_attention(&c.c, layer, &t.c, (int)H, (float)scale, rq.p, rq.row, rq.head, ro.p, ro.row, ro.head,
                          static_cast<float *>(lse), ws.p, ws.n, stream(a[8])),
       "dfv_tree_attention");
  return made.defined() ? THPVariable_Wrap(made) : same(a[6]);
}

// (logits, tree, tokens, rules, ws, out, argmax, store, stream)
PyObject *logits_process(PyObject *const *a) {
  const at::Tensor &x = tensor(a[0], "logits");
  const Tree &t = handle<Tree>(a[1]);
  const Rules &r = handle<Rules>(a[3]);
  const int64_t rows = t.c.n_rows;
  if (x.dim() != 2 || x.size(0) != rows || x.stride(1) != 1)
    value_error("logits must be [%d, V] with contiguous rows", (int)rows);
  const int64_t V = x.size(1);
  const at::ScalarType dt = x.scalar_type();
  if (dt != at::kBFloat16 && dt != at::kFloat) {
    PyErr_Format(PyExc_TypeError, "logits must be bf16 or fp32, got %s", at::toString(dt));
    throw Refused();
  }
  if (x.get_device() != t.index || (r.index != -2 && r.index != t.index))
    value_error("logits, tree and rules are not on one device");
  if (r.n_seqs >= 0 && r.n_seqs != t.c.n_seqs)
    value_error("the rules are for %d sequences, the call has %d", r.n_seqs, t.c.n_seqs);
  if (r.bias_rows && (r.bias_cols != V || (r.bias_rows != 1 && r.bias_rows != t.c.n_seqs)))
    value_error("bias must be [1 or %d, %lld]", t.c.n_seqs, (long long)V);
  if (r.allowed_rows && (r.allowed_cols != (V + 31) / 32 || (r.allowed_rows != 1 && r.allowed_rows != rows)))
    value_error("allowed must be [1 or %d, %lld]", (int)rows, (long long)((V + 31) / 32));
  if (V > INT32_MAX) value_error("V does not fit 32 bits");
  const Space ws = space(a[4], t.index);
  const void *tok = given(a[2], "tokens", at::kInt, {rows}, t.index);
  const int store = PyObject_IsTrue(a[7]);
  if (store < 0) throw Refused();
  at::Tensor made, best;
  void *arg = given(a[6], "argmax", at::kInt, {rows}, t.index), *out = nullptr;
  int64_t out_row = 0;
  if (!store) {
    if (a[5] != Py_None) value_error("store=False takes no out");
  } else {
    if (a[5] == Py_None) made = empty({rows, V}, dt, x, stream(a[8]));
    const at::Tensor &o = made.defined() ? made : tensor(a[5], "out");
    if (o.sizes() != x.sizes() || o.scalar_type() != dt || o.stride(1) != 1 || o.get_device() != t.index)
      value_error("out must be like logits");
    out = o.data_ptr();
    out_row = rows > 1 ? o.stride(0) : V;
  }
  if (!arg) {
    best = empty({rows}, at::kInt, x, stream(a[8]));
    arg = best.data_ptr();
  }
  on_gpu(t.index);
  done(dfv_logits_process(x.data_ptr(), rows > 1 ? x.stride(0) : V, dt == at::kFloat ? DFV_F32 : DFV_BF16, (int)V, &t.c,
                          static_cast<const int32_t *>(tok), &r.c, out, out_row, static_cast<int32_t *>(arg),
                          ws.p, ws.n, stream(a[8])),
       "dfv_logits_process");
  PyObject *o = !store ? same(Py_None) : made.defined() ? THPVariable_Wrap(made) : same(a[5]);
  PyObject *b = best.defined() ? THPVariable_Wrap(best) : same(a[6]);
  PyObject *both = o && b ? PyTuple_Pack(2, o, b) : nullptr;
  Py_XDECREF(o);
  Py_XDECREF(b);
  return both;
}

// (tree, tokens, target, path, tau, stream)
PyObject *accept_tree(PyObject *const *a) {
  const Tree &t = handle<Tree>(a[0]);
  const int64_t rows = t.c.n_rows, S = t.c.n_seqs;
  const void *tok = need(a[1], "tokens", at::kInt, {rows}, t.index), *target = need(a[2], "target", at::kInt, {rows}, t.index);
  const at::Tensor &like = tensor(a[1], "tokens");
  int64_t width = t.c.max_nodes;
  if (a[3] != Py_None) {
    const at::Tensor &g = tensor(a[3], "path");
    width = g.dim() == 2 ? g.size(1) : -1;
  }
  void *pp = given(a[3], "path", at::kInt, {S, width}, t.index), *tp = given(a[4], "tau", at::kInt, {S}, t.index);
  at::Tensor path, tau;
  if (!pp) {
    path = empty({S, width}, at::kInt, like, stream(a[5]));
    pp = path.data_ptr();
  }
  if (!tp) {
    tau = empty({S}, at::kInt, like, stream(a[5]));
    tp = tau.data_ptr();
  }
  on_gpu(t.index);
  done(dfv_accept_tree(&t.c, static_cast<const int32_t *>(tok), static_cast<const int32_t *>(target),
                       static_cast<int32_t *>(pp), width, static_cast<int32_t *>(tp), stream(a[5])),
       "dfv_accept_tree");
  PyObject *p = path.defined() ? THPVariable_Wrap(path) : same(a[3]);
  PyObject *n = tau.defined() ? THPVariable_Wrap(tau) : same(a[4]);
  PyObject *both = p && n ? PyTuple_Pack(2, p, n) : nullptr;
  Py_XDECREF(p);
  Py_XDECREF(n);
  return both;
}

// (cache, tree, path, tau, ws, new_lens, stream)
PyObject *cache_commit(PyObject *const *a) {
  const Cache &c = handle<Cache>(a[0]);
  const Tree &t = handle<Tree>(a[1]);
  together(c, t);
  const at::Tensor &path = tensor(a[2], "path");
  const Space ws = space(a[4], c.index);
  const int64_t S = t.c.n_seqs, width = path.dim() == 2 ? path.size(1) : -1;
  const void *pp = need(a[2], "path", at::kInt, {S, width}, c.index), *tp = need(a[3], "tau", at::kInt, {S}, c.index);
  void *lens = need(a[5], "new_lens", at::kInt, {c.c.max_seqs}, c.index);
  on_gpu(c.index);
  done(dfv_cache_commit(&c.c, &t.c, static_cast<const int32_t *>(pp), width, static_cast<const int32_t *>(tp),
                        static_cast<int32_t *>(lens), ws.p, ws.n, stream(a[6])),
       "dfv_cache_commit");
  return same(a[5]);
}

// index lists of one length
struct Lists {
  const int32_t *a, *b;
  int n;
};
Lists lists(const Cache &c, PyObject *a, const char *an, PyObject *b, const char *bn) {
  const int64_t n = tensor(a, an).numel();
  Lists l = {static_cast<const int32_t *>(need(a, an, at::kInt, {n}, c.index)), nullptr, (int)n};
  if (b) l.b = static_cast<const int32_t *>(need(b, bn, at::kInt, {n}, c.index));
  return l;
}

// (cache, src, dst, stream)
PyObject *cache_copy_pages(PyObject *const *a) {
  const Cache &c = handle<Cache>(a[0]);
  const Lists l = lists(c, a[1], "src", a[2], "dst");
  on_gpu(c.index);
  done(dfv_cache_copy_pages(&c.c, l.a, l.b, l.n, stream(a[3])), "dfv_cache_copy_pages");
  return same(Py_None);
}
// (cache, seqs, n_new, ws, stream)
PyObject *pages_reserve(PyObject *const *a) {
  const Cache &c = handle<Cache>(a[0]);
  const Lists l = lists(c, a[1], "seqs", a[2], "n_new");
  const Space ws = space(a[3], c.index);
  on_gpu(c.index);
  done(dfv_pages_reserve(&c.c, l.a, l.b, l.n, ws.p, ws.n, stream(a[4])), "dfv_pages_reserve");
  return same(Py_None);
}
// (cache, src, dst, ws, stream)
PyObject *pages_fork(PyObject *const *a) {
  const Cache &c = handle<Cache>(a[0]);
  const Lists l = lists(c, a[1], "src", a[2], "dst");
  const Space ws = space(a[3], c.index);
  on_gpu(c.index);
  done(dfv_pages_fork(&c.c, l.a, l.b, l.n, ws.p, ws.n, stream(a[4])), "dfv_pages_fork");
  return same(Py_None);
}
// (cache, seqs, stream)
PyObject *pages_free(PyObject *const *a) {
  const Cache &c = handle<Cache>(a[0]);
  const Lists l = lists(c, a[1], "seqs", nullptr, nullptr);
  on_gpu(c.index);
  done(dfv_pages_free(&c.c, l.a, l.n, stream(a[2])), "dfv_pages_free");
  return same(Py_None);
}

// No C++ exception leaves the extension.
template <PyObject *(*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != N) return PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
  try {
    return F(args);
  } catch (const Refused &) {
    return nullptr;
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    return nullptr;
  }
}
#define DFV_ENTRY(name, n) \
  { #name, (PyCFunction)(void (*)(void))entry<name, n>, METH_FASTCALL, nullptr }

PyMethodDef kMethods[] = {DFV_ENTRY(rope_append, 15),   DFV_ENTRY(tree_attention, 9), DFV_ENTRY(logits_process, 9),
                          DFV_ENTRY(accept_tree, 6),    DFV_ENTRY(cache_commit, 7),   DFV_ENTRY(cache_copy_pages, 4),
                          DFV_ENTRY(pages_reserve, 5),  DFV_ENTRY(pages_fork, 5),     DFV_ENTRY(pages_free, 3),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_dfvbind", "hot calls of the tree-verify binding", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__dfvbind(void) { return PyModule_Create(&kModule); }
