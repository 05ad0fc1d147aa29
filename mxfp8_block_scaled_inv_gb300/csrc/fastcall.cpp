// The common calls of the norm, the routing and the 4-bit products from Python
// without the interpreter's share: checks of the tensors, allocation of the outputs
// on the current stream and the call of libmxq's entry point in one C++ function
// (an eager decode step makes a hundred such calls of a few microseconds each).
//
// Each function answers None for whatever is not the common case (a tensor of
// another type, shape, layout or device, a device that is not the current one, a
// library error): the binding's Python code then does the call, and words the
// error.  The library itself is reached through the addresses that `bind` gets.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

#include "mxq.h"

namespace {

struct Entry {
  decltype(&mxq_add_rms_norm) norm;
  decltype(&mxq_route) route;
  decltype(&mxq_w4_bytes) w4_bytes;
  decltype(&mxq_linear_a8w4) linear;
  decltype(&mxq_experts_workspace_bytes) experts_ws;
  decltype(&mxq_experts_a8w4) experts;
} lib = {};

// The current device if that is where the tensor is, or -1.
int device_of(PyObject* o) {
  if (!THPVariable_CheckExact(o)) return -1;
  const at::Tensor& t = THPVariable_Unpack(o);
  return t.is_cuda() && t.get_device() == c10::cuda::current_device() ? (int)t.get_device() : -1;
}
// A contiguous CUDA tensor of this type on that device, or null.
const at::Tensor* tensor(PyObject* o, at::ScalarType type, int device) {
  if (!THPVariable_CheckExact(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.scalar_type() != type || t.get_device() != device || !t.is_contiguous())
    return nullptr;
  return &t;
}
bool has_shape(const at::Tensor& t, std::initializer_list<int64_t> shape) {
  return t.sizes() == at::IntArrayRef(shape);
}

bool number(PyObject* o, int64_t* v) {
  if (!PyLong_Check(o)) return false;
  int over = 0;
  const long long n = PyLong_AsLongLongAndOverflow(o, &over);
  if (over || (n == -1 && PyErr_Occurred())) {
    PyErr_Clear();
    return false;
  }
  *v = n;
  return true;
}
bool small_number(PyObject* o, int32_t* v) {
  int64_t n;
  if (!number(o, &n) || n < INT32_MIN || n > INT32_MAX) return false;
  *v = (int32_t)n;
  return true;
}
bool real(PyObject* o, float* v) {
  if (!PyFloat_Check(o) && !PyLong_Check(o)) return false;
  const double d = PyFloat_AsDouble(o);
  if (d == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  *v = (float)d;
  return true;
}

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(like.device()));
}
void* current_stream(int device) {
  return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
}

void* address(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
uint8_t* bytes(const at::Tensor& t) { return static_cast<uint8_t*>(address(t)); }

// An entry point without the interpreter's lock.  Its arguments are values by then:
// what can throw has been evaluated under the lock.
template <typename F, typename... A>
int call(F f, A... args) {
  int st;
  Py_BEGIN_ALLOW_THREADS
  st = f(args...);
  Py_END_ALLOW_THREADS
  return st;
}

// norm(x, weight, eps, residual, want_y, want_codes) -> (s, y, q, sc)
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 6) Py_RETURN_NONE;
  const int dev = device_of(a[0]);
  if (dev < 0) Py_RETURN_NONE;
  const at::Tensor* x = tensor(a[0], at::kBFloat16, dev);
  float eps;
  if (!x || x->dim() < 1 || x->size(-1) < 16 || !real(a[2], &eps)) Py_RETURN_NONE;
  const int64_t D = x->size(-1), T = x->numel() / D;
  if (D > 65536) Py_RETURN_NONE;
  const at::Tensor *w = nullptr, *r = nullptr;
  if (a[1] != Py_None && (!(w = tensor(a[1], at::kBFloat16, dev)) || !has_shape(*w, {D}))) Py_RETURN_NONE;
  if (a[3] != Py_None && (!(r = tensor(a[3], at::kBFloat16, dev)) || r->sizes() != x->sizes()))
    Py_RETURN_NONE;
  at::Tensor s, y, q, sc;
  if (r) s = empty(x->sizes(), at::kBFloat16, *x);
  if (a[4] == Py_True) y = empty(x->sizes(), at::kBFloat16, *x);
  if (a[5] == Py_True) {
    q = empty(x->sizes(), at::kByte, *x);
    auto shape = x->sizes().vec();
    shape.back() = (D + 127) / 128;
    sc = empty(shape, at::kByte, *x);
  }
  if (call(lib.norm, address(*x), r ? address(*r) : nullptr, address(s), w ? address(*w) : nullptr, T,
           (int32_t)D, eps, address(y), bytes(q), bytes(sc), current_stream(dev)))
    Py_RETURN_NONE;
  PyObject* out = PyTuple_New(4);
  if (!out) return nullptr;
  const at::Tensor* all[4] = {&s, &y, &q, &sc};
  for (int i = 0; i < 4; ++i) {
    PyObject* o = all[i]->defined() ? THPVariable_Wrap(*all[i]) : Py_NewRef(Py_None);
    if (!o) {
      Py_DECREF(out);
      return nullptr;
    }
    PyTuple_SET_ITEM(out, i, o);
  }
  return out;
  END_HANDLE_TH_ERRORS
}

// route(logits, k, scoring, bias, groups, topk_groups, group_top, renormalise, scale)
// -> (ids, weights)
PyObject* route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 9) Py_RETURN_NONE;
  const int dev = device_of(a[0]);
  if (dev < 0) Py_RETURN_NONE;
  int32_t dtype = MXQ_LOGITS_F32;
  const at::Tensor* l = tensor(a[0], at::kFloat, dev);
  if (!l) {
    l = tensor(a[0], at::kBFloat16, dev);
    dtype = MXQ_LOGITS_BF16;
  }
  int32_t k, scoring, groups, keep, top;
  float scale;
  if (!l || l->dim() != 2 || !small_number(a[1], &k) || !small_number(a[2], &scoring) ||
      !small_number(a[4], &groups) || !small_number(a[5], &keep) || !small_number(a[6], &top) ||
      !real(a[8], &scale) || k < 1 || k > 32 || l->size(1) > 1024)
    Py_RETURN_NONE;
  const int64_t T = l->size(0), E = l->size(1);
  const at::Tensor* b = nullptr;
  if (a[3] != Py_None && (!(b = tensor(a[3], at::kFloat, dev)) || !has_shape(*b, {E}))) Py_RETURN_NONE;
  at::Tensor ids = empty({T, k}, at::kInt, *l), w = empty({T, k}, at::kFloat, *l);
  if (call(lib.route, address(*l), dtype, T, (int32_t)E, b ? b->data_ptr<float>() : nullptr, k, scoring,
           groups, keep, top, (int32_t)(a[7] == Py_True), scale, ids.data_ptr<int32_t>(),
           w.data_ptr<float>(), current_stream(dev)))
    Py_RETURN_NONE;
  return Py_BuildValue("(NN)", THPVariable_Wrap(ids), THPVariable_Wrap(w));
  END_HANDLE_TH_ERRORS
}

// linear(a, a_sf, w4, N) -> out
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 4) Py_RETURN_NONE;
  const int dev = device_of(a[0]);
  if (dev < 0) Py_RETURN_NONE;
  const at::Tensor *x = tensor(a[0], at::kByte, dev), *s = tensor(a[1], at::kByte, dev),
                   *w = tensor(a[2], at::kByte, dev);
  int32_t N;
  if (!x || !s || !w || x->dim() != 2 || !small_number(a[3], &N) || x->size(1) > 65536) Py_RETURN_NONE;
  const int64_t T = x->size(0), K = x->size(1);
  const size_t size = lib.w4_bytes(1, N, (int32_t)K);
  if (!size || !has_shape(*s, {T, (K + 127) / 128}) || !has_shape(*w, {(int64_t)size})) Py_RETURN_NONE;
  at::Tensor out = empty({T, N}, at::kBFloat16, *x);
  if (call(lib.linear, bytes(*x), bytes(*s), bytes(*w), address(out), T, N, (int32_t)K, current_stream(dev)))
    Py_RETURN_NONE;
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// experts(a, a_sf, ids, weights, w13, w2, I, N) -> out
PyObject* experts(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 8) Py_RETURN_NONE;
  const int dev = device_of(a[0]);
  if (dev < 0) Py_RETURN_NONE;
  const at::Tensor *x = tensor(a[0], at::kByte, dev), *s = tensor(a[1], at::kByte, dev),
                   *ids = tensor(a[2], at::kInt, dev), *wt = tensor(a[3], at::kFloat, dev),
                   *w13 = tensor(a[4], at::kByte, dev), *w2 = tensor(a[5], at::kByte, dev);
  int32_t I, N;
  if (!x || !s || !ids || !wt || !w13 || !w2 || x->dim() != 2 || ids->dim() != 2 ||
      !small_number(a[6], &I) || !small_number(a[7], &N) || x->size(1) > 65536 || ids->size(1) > 32)
    Py_RETURN_NONE;
  const int64_t T = x->size(0), K = x->size(1), k = ids->size(1);
  const size_t one13 = lib.w4_bytes(2, I, (int32_t)K), one2 = lib.w4_bytes(1, N, I);
  if (!one13 || !one2) Py_RETURN_NONE;
  const int64_t E = w2->numel() / (int64_t)one2;
  if (E < 1 || E > 1024 || !has_shape(*s, {T, (K + 127) / 128}) || !has_shape(*ids, {T, k}) ||
      !has_shape(*wt, {T, k}) || !has_shape(*w13, {E * (int64_t)one13}) ||
      !has_shape(*w2, {E * (int64_t)one2}))
    Py_RETURN_NONE;
  const size_t need = lib.experts_ws(T, (int32_t)k, (int32_t)E, (int32_t)K, I, N);
  if (!need) Py_RETURN_NONE;
  at::Tensor out = empty({T, N}, at::kBFloat16, *x), ws = empty({(int64_t)need}, at::kByte, *x);
  if (call(lib.experts, bytes(*x), bytes(*s), ids->data_ptr<int32_t>(), wt->data_ptr<float>(), bytes(*w13),
           bytes(*w2), address(out), T, (int32_t)k, (int32_t)E, (int32_t)K, I, N, nullptr, address(ws), need,
           current_stream(dev)))
    Py_RETURN_NONE;
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// bind(addresses of the six entry points, in Entry's order)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* p[6];
  if (n != 6) {
    PyErr_SetString(PyExc_TypeError, "bind takes six addresses");
    return nullptr;
  }
  for (int i = 0; i < 6; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind got a null address");
      return nullptr;
    }
  }
  lib.norm = reinterpret_cast<decltype(lib.norm)>(p[0]);
  lib.route = reinterpret_cast<decltype(lib.route)>(p[1]);
  lib.w4_bytes = reinterpret_cast<decltype(lib.w4_bytes)>(p[2]);
  lib.linear = reinterpret_cast<decltype(lib.linear)>(p[3]);
  lib.experts_ws = reinterpret_cast<decltype(lib.experts_ws)>(p[4]);
  lib.experts = reinterpret_cast<decltype(lib.experts)>(p[5]);
  Py_RETURN_NONE;
}

#define METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(bind), METHOD(norm), METHOD(route), METHOD(linear), METHOD(experts),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "mxq_fastcall", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit_mxq_fastcall(void) { return PyModule_Create(&module); }
