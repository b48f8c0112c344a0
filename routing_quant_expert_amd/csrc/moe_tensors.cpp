// The calls of the operators beside the layer on torch tensors (Python module
// `_tensors`): every tensor is held against the call's description (moe_join,
// moe_grouped, moe_adapters), then the entry point of include/moe.h is called.
// Native because the host's part of a small call is all of it: a join_forward
// of one row takes 3.6 us so, 4.6 through ctypes without the checks of its seven
// tensors and 5.4 with them in Python.
//
// A tensor has to be where the device can read it, of the described type (one
// of integers is taken for the bits of any type), with its rows where the
// strides say, and inside its memory. Objects that are no tensors give their
// address by data_ptr() and are not looked at further.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdio>
#include <cstring>
#include <exception>

#include "../../include/moe.h"

namespace {

PyObject* moe_error = nullptr;   // the binding's exception type

struct {
  decltype(&::moe_join_forward) join_forward;
  decltype(&::moe_join_backward) join_backward;
  decltype(&::moe_grouped_forward) grouped_forward;
  decltype(&::moe_grouped_backward_x) grouped_backward_x;
  decltype(&::moe_grouped_backward_w) grouped_backward_w;
  decltype(&::moe_adapter_project) adapter_project;
  decltype(&::moe_last_error) last_error;
} entry;

// Every failure is an exception here and a MoeError (or the Python error that is set) at the module's functions.
struct PythonError {};

[[noreturn]] void fail(int code, const char* text) {
  if (PyObject* args = Py_BuildValue("(is)", code, text)) {
    PyErr_SetObject(moe_error, args);   // (a tuple: the exception's arguments)
    Py_DECREF(args);
  }
  throw PythonError();
}
[[noreturn]] void fail(const char* what, const char* text) {
  char buf[160];
  snprintf(buf, sizeof(buf), "%s: %s", what, text);
  fail(MOE_EINVAL, buf);
}

// The value of a new reference as an address or a number.
unsigned long long number(PyObject* o) {
  if (!o) throw PythonError();
  const unsigned long long v = PyLong_AsUnsignedLongLong(o);
  Py_DECREF(o);
  if (PyErr_Occurred()) throw PythonError();
  return v;
}
unsigned long long call(PyObject* o, const char* method) { return number(PyObject_CallMethod(o, method, nullptr)); }

// What a call reads or writes: `outer` times `rows` rows of `width` elements, strides in elements.
struct Extent {
  int64_t outer, outer_stride, rows, stride, width;
  bool empty() const { return outer <= 0 || rows <= 0 || width <= 0; }
  // From its first element to its last one; as much as fits where an invalid description asks for more.
  int64_t span() const {
    const __int128 v = (__int128)(outer - 1) * outer_stride + (__int128)(rows - 1) * stride + width;
    return v > kMost ? kMost : v < 0 ? 0 : (int64_t)v;
  }
  static constexpr int64_t kMost = INT64_MAX / 8;
};
Extent vector(int64_t n) { return {1, 0, 1, 0, n}; }
Extent matrix(int64_t rows, int64_t stride, int64_t width) { return {1, 0, rows, stride, width}; }

constexpr int kIndex = 16;   // 32-bit integers; otherwise MOE_TYPE_*

// Elements of a tensor in the units of the description (bytes of `e`): sizes and strides of integers that stand for others' bits scale.
struct View {
  const at::Tensor& t;
  int64_t item, e;
  int first;   // dimensions of size 1 in front are left out
  int dims() const { return (int)t.dim() - first; }
  int64_t size(int d) const { return t.sizes()[first + d]; }
  bool is_stride(int d, int64_t elements) const { return t.strides()[first + d] * item == elements * e; }
  // The dimensions from d on lie one after another and have at least `n` elements.
  bool packed(int d, int64_t n) const {
    int64_t expect = 1;
    for (int i = dims() - 1; i >= d; --i) {
      if (size(i) != 1 && t.strides()[first + i] != expect) return false;
      expect *= size(i);
    }
    return expect * item >= n * e;
  }
};

bool rows_fit(const View& v, const Extent& x) {
  const int n = v.dims();
  if (x.outer == 1 && x.rows == 1)
    return v.packed(0, x.width) || (n == 2 && v.packed(1, x.width));
  if (x.outer == 1) {
    if (n >= 1 && v.size(0) == x.rows && (n > 1 || x.width == 1))
      return v.is_stride(0, x.stride) && v.packed(1, x.width);
    return v.packed(0, x.span()) || (n == 2 && v.size(0) > x.rows && v.is_stride(0, x.stride) && v.packed(1, x.width));
  }
  if (n == 3 && v.size(0) == x.outer && v.size(1) == x.rows)
    return v.is_stride(0, x.outer_stride) && (x.rows == 1 || v.is_stride(1, x.stride)) && v.packed(2, x.width);
  if (v.packed(0, x.span())) return true;
  return n == 2 && v.size(0) == x.outer * x.rows && v.packed(1, x.width) &&
         (x.rows == 1 ? v.is_stride(0, x.outer_stride)
                      : v.is_stride(0, x.stride) && x.outer_stride == x.rows * x.stride);
}

void on_device(const at::Tensor& t, const char* what) {
  if (!t.is_cuda() && !(t.is_cpu() && t.is_pinned())) fail(what, "not on the device");
}

void* address(PyObject* o, const char* what, int type, const Extent& x) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) return (void*)call(o, "data_ptr");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.layout() != at::kStrided || !t.has_storage()) fail(what, "not a strided tensor with memory of its own");
  const at::ScalarType s = t.scalar_type();
  if (type == kIndex) {
    if (s != at::kInt && s != at::kUInt32) fail(what, "must be int32");
  } else {
    const at::ScalarType want = type == MOE_TYPE_BF16 ? at::kBFloat16 : type == MOE_TYPE_FP16 ? at::kHalf : at::kFloat;
    if (s != want && !at::isIntegralType(s, true)) fail(what, "not of the described element type");
  }
  const int64_t item = t.element_size(), e = type == MOE_TYPE_BF16 || type == MOE_TYPE_FP16 ? 2 : 4;
  if (!x.empty()) {
    if (x.span() * e > (int64_t)t.storage().nbytes() - t.storage_offset() * item)
      fail(what, "smaller than what the call reads or writes there");
    int first = 0;
    while (t.dim() - first > 2 && t.sizes()[first] == 1 && (x.outer == 1 || t.dim() - first > 3)) ++first;
    if (!rows_fit({t, item, e, first}, x)) fail(what, "its rows do not lie as the description says");
  }
  on_device(t, what);
  return t.data_ptr();
}

int64_t rows_of(PyObject* o, const char* what) {
  if (o == Py_None) fail(what, "must not be None");
  if (THPVariable_Check(o)) {
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.dim() < 1) fail(what, "has no rows");
    return t.sizes()[0];
  }
  PyObject* shape = PyObject_GetAttrString(o, "shape");
  if (!shape) throw PythonError();
  PyObject* rows = PySequence_GetItem(shape, 0);
  Py_DECREF(shape);
  if (!rows) throw PythonError();
  const long long v = PyLong_AsLongLong(rows);
  Py_DECREF(rows);
  if (v == -1 && PyErr_Occurred()) throw PythonError();
  return v;
}

struct Workspace {
  void* at;
  size_t bytes;
};
Workspace workspace(PyObject* o) {
  if (o == Py_None) return {nullptr, 0};
  if (!THPVariable_Check(o)) return {(void*)call(o, "data_ptr"), (size_t)(call(o, "numel") * call(o, "element_size"))};
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.layout() != at::kStrided || !t.has_storage() || !t.is_contiguous()) fail("workspace", "not contiguous");
  on_device(t, "workspace");
  return {t.data_ptr(), (size_t)(t.numel() * t.element_size())};
}

// The description's memory (a ctypes structure).
template <typename P>
class Plan {
  Py_buffer view_;

 public:
  Plan(PyObject* o, const char* what) {
    if (PyObject_GetBuffer(o, &view_, PyBUF_SIMPLE)) throw PythonError();
    if (view_.len != (Py_ssize_t)sizeof(P)) {
      PyBuffer_Release(&view_);
      fail(what, "not the description of this call");
    }
  }
  ~Plan() { PyBuffer_Release(&view_); }
  Plan(const Plan&) = delete;
  Plan& operator=(const Plan&) = delete;
  const P* operator->() const { return (const P*)view_.buf; }
  const P* get() const { return (const P*)view_.buf; }
};

void* stream_of(PyObject* o) {
  void* s = PyLong_AsVoidPtr(o);
  if (PyErr_Occurred()) throw PythonError();
  return s;
}

// A module function of `n` arguments around `body`, which calls the entry point and gives its code.
template <int N, int (*Body)(PyObject* const*)>
PyObject* function(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, %zd given", N, n);
    return nullptr;
  }
  try {
    const int code = Body(args);
    if (code) fail(code, entry.last_error());
    Py_RETURN_NONE;
  } catch (const PythonError&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unexpected error");
  }
  return nullptr;
}

template <typename F>
int without_gil(F&& f) {
  PyThreadState* state = PyEval_SaveThread();
  const int code = f();
  PyEval_RestoreThread(state);
  return code;
}

int join_forward(PyObject* const* a) {
  const Plan<moe_join> j(a[0], "join");
  const int64_t m = rows_of(a[1], "x"), dim = j->dim;
  const Extent each = vector(dim);
  const void* x = address(a[1], "x", j->residual_type, matrix(m, j->x_stride, dim));
  const void* b = address(a[2], "block", j->type, matrix(m, j->b_stride, dim));
  const void* w_post = address(a[3], "w_post", j->type, each);
  const void* gate = address(a[4], "gate", j->type, j->gate_rows ? matrix(m, j->gate_stride, dim) : each);
  const void* w_pre = address(a[5], "w_pre", j->type, each);
  void* x_out = address(a[6], "x_out", j->residual_type, matrix(m, j->x_out_stride, dim));
  void* y = address(a[7], "y", j->type, matrix(m, j->y_stride, dim));
  void* stream = stream_of(a[8]);
  return without_gil([&] { return entry.join_forward(j.get(), x, b, w_post, gate, w_pre, m, x_out, y, stream); });
}

int join_backward(PyObject* const* a) {
  const Plan<moe_join> j(a[0], "join");
  const int64_t m = rows_of(a[8], "dx"), dim = j->dim;
  const Extent each = vector(dim), stream_rows = matrix(m, j->x_out_stride, dim), block_rows = matrix(m, j->b_stride, dim);
  const Extent gates = j->gate_rows ? matrix(m, j->gate_stride, dim) : each;
  const void* dy = address(a[1], "dy", j->type, matrix(m, j->y_stride, dim));
  const void* dx_out = address(a[2], "dx_out", j->residual_type, stream_rows);
  const void* x_out = address(a[3], "x_out", j->residual_type, stream_rows);
  const void* b = address(a[4], "block", j->type, block_rows);
  const void* w_post = address(a[5], "w_post", j->type, each);
  const void* gate = address(a[6], "gate", j->type, gates);
  const void* w_pre = address(a[7], "w_pre", j->type, each);
  void* dx = address(a[8], "dx", j->residual_type, matrix(m, j->x_stride, dim));
  void* db = address(a[9], "dblock", j->type, block_rows);
  float* dw_post = (float*)address(a[10], "dw_post", MOE_TYPE_F32, each);
  void* dgate = address(a[11], "dgate", j->gate_rows ? j->type : MOE_TYPE_F32, gates);
  float* dw_pre = (float*)address(a[12], "dw_pre", MOE_TYPE_F32, each);
  const Workspace ws = workspace(a[13]);
  void* stream = stream_of(a[14]);
  return without_gil([&] {
    return entry.join_backward(j.get(), dy, dx_out, x_out, b, w_post, gate, w_pre, m, dx, db, dw_post, dgate, dw_pre,
                               ws.at, ws.bytes, stream);
  });
}

enum Way { kForward, kInput, kWeight };
template <Way W>
int grouped(PyObject* const* a) {
  const Plan<moe_grouped> g(a[0], "grouped");
  const int64_t rows = rows_of(a[1], W == kForward ? "x" : "dy");
  const Extent x = matrix(rows, g->x_stride, g->k), y = matrix(rows, g->y_stride, g->n);
  const Extent w = {g->n_groups, g->w_group_stride, g->n, g->w_stride, g->k};
  const void* in = address(a[1], W == kForward ? "x" : "dy", g->type, W == kForward ? x : y);
  const void* other = address(a[2], W == kWeight ? "x" : "w", g->type, W == kWeight ? x : w);
  const int32_t* offsets = (const int32_t*)address(a[3], "offsets", kIndex, vector((int64_t)g->n_groups + 1));
  void* out = address(a[4], W == kForward ? "y" : W == kInput ? "dx" : "dw", g->out_type,
                      W == kForward ? y : W == kInput ? x : w);
  int32_t* status = (int32_t*)address(a[5], "status", kIndex, vector(1));
  void* stream = stream_of(a[6]);
  const auto f = W == kForward ? entry.grouped_forward : W == kInput ? entry.grouped_backward_x : entry.grouped_backward_w;
  return without_gil([&] { return f(g.get(), in, other, offsets, rows, out, status, stream); });
}

// The adapters' own tensors, which the description keeps beside their addresses.
void kept_on_device(PyObject* plan) {
  PyObject* kept = PyObject_GetAttrString(plan, "_kept");
  if (!kept) {   // (a description that was copied or filled in by hand)
    PyErr_Clear();
    return;
  }
  const Py_ssize_t n = PyTuple_Check(kept) ? PyTuple_GET_SIZE(kept) : 0;
  bool there = true;
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject* o = PyTuple_GET_ITEM(kept, i);
    if (!THPVariable_Check(o)) continue;
    const at::Tensor& t = THPVariable_Unpack(o);
    there = there && (t.is_cuda() || (t.is_cpu() && t.is_pinned()));
  }
  Py_DECREF(kept);
  if (!there) fail("adapters", "a, b or factor is not on the device");
}

int adapter_project(PyObject* const* a) {
  const Plan<moe_adapters> p(a[0], "adapters");
  const int64_t m = rows_of(a[1], "x");
  const void* x = address(a[1], "x", p->type, matrix(m, p->x_stride, p->k));
  const void* w = address(a[2], "w", p->type, matrix(p->n, p->w_stride, p->k));
  const int32_t* index = (const int32_t*)address(a[3], "index", kIndex, vector(m));
  void* out = address(a[4], "out", p->out_type, matrix(m, p->out_stride, p->n));
  const Workspace ws = workspace(a[5]);
  int32_t* status = (int32_t*)address(a[6], "status", kIndex, vector(1));
  void* stream = stream_of(a[7]);
  if (THPVariable_Check(a[1])) kept_on_device(a[0]);
  return without_gil([&] {
    return entry.adapter_project(p.get(), x, w, index, m, out, ws.at, ws.bytes, status, stream);
  });
}

// bind(MoeError, addresses of the entry points in the order of `entry`)
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  constexpr int kEntries = sizeof(entry) / sizeof(void*);
  if (n != 1 + kEntries) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, %zd given", 1 + kEntries, n);
    return nullptr;
  }
  void* at[kEntries];
  for (int i = 0; i < kEntries; ++i) {
    at[i] = PyLong_AsVoidPtr(args[1 + i]);
    if (PyErr_Occurred()) return nullptr;
  }
  memcpy(&entry, at, sizeof(entry));
  Py_INCREF(args[0]);
  Py_XDECREF(moe_error);
  moe_error = args[0];
  Py_RETURN_NONE;
}

#define MOE_METHOD(name, f) {name, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {MOE_METHOD("bind", bind),
                         MOE_METHOD("join_forward", (function<9, join_forward>)),
                         MOE_METHOD("join_backward", (function<15, join_backward>)),
                         MOE_METHOD("grouped_forward", (function<7, grouped<kForward>>)),
                         MOE_METHOD("grouped_backward_x", (function<7, grouped<kInput>>)),
                         MOE_METHOD("grouped_backward_w", (function<7, grouped<kWeight>>)),
                         MOE_METHOD("adapter_project", (function<8, adapter_project>)),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() { return PyModule_Create(&module); }
