// paged_ext.cpp — the short way from Python into the paged-cache calls.
//
// A decode step makes these calls for a few microseconds of GPU work each, and
// marshalling 20 to 30 arguments through ctypes takes longer than that.  The
// functions here take the tensors themselves, check what _paged.py checks,
// allocate the outputs and call the C ABI of the loaded library (`bind` gets
// the addresses): 4 to 10 us a call instead of 11 to 21.  They decide nothing: where
// any check fails, or a call is not plain (a stream or outputs of the caller's,
// another device, an empty batch), they return None, and _paged.py goes its
// own way, which names the fault.  An int is the library's status.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/core/grad_mode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "dsa_paged.h"

namespace {

decltype(&dsa_page_plan_workspace_size) plan_size;
decltype(&dsa_page_plan) plan;
decltype(&dsa_page_append) append;
decltype(&dsa_attend_paged_workspace_size) paged_size;
decltype(&dsa_attend_paged) paged;
decltype(&dsa_attend_selected_workspace_size) selected_size;
decltype(&dsa_attend_selected) selected;

PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  void* p[7];
  if (n != 7) {
    PyErr_SetString(PyExc_TypeError, "bind takes seven addresses");
    return nullptr;
  }
  for (int i = 0; i < 7; ++i)
    if (!(p[i] = PyLong_AsVoidPtr(args[i]))) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an address is null");
      return nullptr;
    }
  plan_size = reinterpret_cast<decltype(plan_size)>(p[0]);
  plan = reinterpret_cast<decltype(plan)>(p[1]);
  append = reinterpret_cast<decltype(append)>(p[2]);
  paged_size = reinterpret_cast<decltype(paged_size)>(p[3]);
  paged = reinterpret_cast<decltype(paged)>(p[4]);
  selected_size = reinterpret_cast<decltype(selected_size)>(p[5]);
  selected = reinterpret_cast<decltype(selected)>(p[6]);
  Py_RETURN_NONE;
}

// A tensor argument; nullptr and true for None.
bool take(PyObject* o, const at::Tensor*& t, bool may_be_none = false) {
  t = nullptr;
  if (o == Py_None) return may_be_none;
  if (!THPVariable_Check(o)) return false;
  t = &THPVariable_Unpack(o);
  return true;
}

bool take_int(PyObject* o, int& x) {
  if (!PyLong_Check(o)) return false;
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  x = (int)v;
  return x == v;
}

bool is(const at::Tensor& t, at::ScalarType type, const c10::Device& dev, at::IntArrayRef shape) {
  return t.scalar_type() == type && t.device() == dev && t.sizes() == shape && t.is_contiguous();
}

bool small(const at::Tensor& t) {  // every extent is an int
  for (const int64_t n : t.sizes())
    if (n > 0x7fffffff) return false;
  return true;
}

// Whether one of the tensors wants a gradient, which the calls would lose.
template <size_t N>
bool wants_gradient(const at::Tensor* (&t)[N]) {
  if (!at::GradMode::is_enabled()) return false;
  for (const at::Tensor* x : t)
    if (x && x->requires_grad()) return true;
  return false;
}

bool on_current_device(const at::Tensor& t) {
  return t.is_cuda() && t.device().index() == c10::cuda::current_device();
}

// The pages of a cache: their element type and how far apart they lie.
bool pool(const at::Tensor& K, const at::Tensor* V, const at::Tensor* Ks, const at::Tensor* Vs, const c10::Device& dev,
          int64_t Hkv, int64_t d, int& type, int64_t& stride) {
  if (K.dim() != 4 || K.device() != dev || K.size(0) < 1 || K.size(2) != Hkv || K.size(3) != d || !small(K)) return false;
  const int64_t n = K.size(0), page = K.size(1);
  switch (K.scalar_type()) {
    case at::kBFloat16: type = DSA_DTYPE_BF16; break;
    case at::kFloat: type = DSA_DTYPE_FP32; break;
    case at::kByte:
    case at::kFloat8_e4m3fn: type = DSA_DTYPE_FP8_E4M3; break;
    default: return false;
  }
  stride = n > 1 ? K.stride(0) : page * Hkv * d;
  for (const at::Tensor* t : {&K, V}) {
    if (!t) continue;
    if (t->device() != dev || t->sizes() != K.sizes() || t->scalar_type() != K.scalar_type() || t->stride(3) != 1 ||
        t->stride(2) != d || t->stride(1) != Hkv * d || (n > 1 && t->stride(0) != stride) || stride < page * Hkv * d)
      return false;
  }
  const bool fp8 = type == DSA_DTYPE_FP8_E4M3;
  if (fp8 != (Ks != nullptr) || (fp8 && V) != (Vs != nullptr)) return false;
  const int64_t shape[3] = {n, page, Hkv};
  return (!Ks || is(*Ks, at::kFloat, dev, shape)) && (!Vs || is(*Vs, at::kFloat, dev, shape));
}

bool query_type(const at::Tensor& t, int& type) {
  if (t.scalar_type() != at::kBFloat16 && t.scalar_type() != at::kFloat) return false;
  type = t.scalar_type() == at::kFloat ? DSA_DTYPE_FP32 : DSA_DTYPE_BF16;
  return true;
}

template <typename T>
T* ptr(const at::Tensor* t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}

void* stream(const c10::Device& dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

// lens, new_lens, block_table, free_pages, used, page, n_pages, max_tokens, workspace -> the five outputs
PyObject* page_plan(const at::Tensor* (&t)[6], int page, int n_pages, int max_tokens) {
  const at::Tensor &lens = *t[0], &table = *t[2], &free = *t[3], &ws = *t[5];
  if (lens.dim() != 1 || table.dim() != 2 || free.dim() != 1 || !on_current_device(lens) || !small(table) || !small(free))
    Py_RETURN_NONE;
  const c10::Device dev = lens.device();
  const int64_t B = lens.size(0), width = table.size(1);
  const auto i32 = at::kInt;
  if (B < 1 || max_tokens < 0 || !is(lens, i32, dev, {B}) || !is(*t[1], i32, dev, {B}) || !is(table, i32, dev, {B, width}) ||
      !is(free, i32, dev, {free.size(0)}) || !is(*t[4], i32, dev, {1}) || ws.device() != dev || !ws.is_contiguous())
    Py_RETURN_NONE;
  size_t need = 0;
  if (plan_size((int)B, max_tokens, &need) != DSA_OK || ws.nbytes() < need) Py_RETURN_NONE;
  const auto options = lens.options();
  const at::Tensor out[5] = {at::empty({B + 1}, options), at::empty({max_tokens}, options.dtype(at::kLong)),
                             at::empty({max_tokens}, options), at::empty({B}, options), at::empty({1}, options)};
  const int r = plan(ptr<int32_t>(t[0]), ptr<int32_t>(t[1]), ptr<int32_t>(t[3]), (int)free.size(0), ptr<int32_t>(t[4]),
                     (int)B, page, n_pages, (int)width, max_tokens, ptr<int32_t>(t[2]), ptr<int32_t>(&out[0]),
                     ptr<int64_t>(&out[1]), ptr<int32_t>(&out[2]), ptr<int32_t>(&out[3]), ptr<int32_t>(&out[4]),
                     ws.data_ptr(), ws.nbytes(), stream(dev));
  if (r != DSA_OK) return PyLong_FromLong(r);
  PyObject* tuple = PyTuple_New(5);
  for (int i = 0; tuple && i < 5; ++i) PyTuple_SET_ITEM(tuple, i, THPVariable_Wrap(out[i]));
  return tuple;
}

// k, K, slots, v, V, K_scale, V_scale, workspace -> status
PyObject* page_append(const at::Tensor* (&t)[8]) {
  const at::Tensor &k = *t[0], &K = *t[1], &slots = *t[2], &ws = *t[7];
  int src = 0, type = 0;
  int64_t stride = 0;
  if (wants_gradient(t) || k.dim() != 3 || !on_current_device(k) || !query_type(k, src) || !small(k) || (t[3] == nullptr) != (t[4] == nullptr))
    Py_RETURN_NONE;
  const c10::Device dev = k.device();
  if (k.size(0) < 1 || !k.is_contiguous() || (t[3] && !is(*t[3], k.scalar_type(), dev, k.sizes())) ||
      !is(slots, at::kLong, dev, {k.size(0)}) || !pool(K, t[4], t[5], t[6], dev, k.size(1), k.size(2), type, stride) ||
      ws.device() != dev || !ws.is_contiguous() || ws.nbytes() < 256)
    Py_RETURN_NONE;
  return PyLong_FromLong(append(k.data_ptr(), ptr<void>(t[3]), ptr<int64_t>(t[2]), (int)k.size(0), (int)k.size(1),
                                (int)k.size(2), src, type, K.data_ptr(), ptr<void>(t[4]), ptr<float>(t[5]),
                                ptr<float>(t[6]), (int)K.size(0), (int)K.size(1), stride, ws.data_ptr(), ws.nbytes(),
                                stream(dev)));
}

// Q, K, V, block_table, lens, q_offsets, idx, K_scale, V_scale, workspace, max_q, scale, whether lse -> out (, lse)
PyObject* attend(const at::Tensor* (&t)[10], int max_q, const float* scale, bool with_lse) {
  const at::Tensor &Q = *t[0], &K = *t[1], &table = *t[3], &lens = *t[4], &ws = *t[9];
  const at::Tensor* idx = t[6];
  int qt = 0, type = 0;
  int64_t stride = 0;
  if (wants_gradient(t) || Q.dim() != 3 || lens.dim() != 1 || table.dim() != 2 || (idx && idx->dim() != 2) || !on_current_device(Q) ||
      !query_type(Q, qt) || !small(Q) || !small(table) || K.dim() != 4)
    Py_RETURN_NONE;
  const c10::Device dev = Q.device();
  const int64_t rows = Q.size(0), Hq = Q.size(1), d = Q.size(2), B = lens.size(0), width = table.size(1), Hkv = K.size(2);
  if (rows < 1 || B < 1 || !Q.is_contiguous() || !pool(K, t[2], t[7], t[8], dev, Hkv, d, type, stride) ||
      !is(lens, at::kInt, dev, {B}) || !is(*t[5], at::kInt, dev, {B + 1}) || !is(table, at::kInt, dev, {B, width}) ||
      (idx && (!small(*idx) || !is(*idx, at::kInt, dev, {rows, idx->size(1)}))) || ws.device() != dev || !ws.is_contiguous())
    Py_RETURN_NONE;
  const int mid = idx ? (int)idx->size(1) : max_q;
  size_t need = 0;
  if ((idx ? selected_size : paged_size)((int)B, (int)rows, mid, (int)Hq, (int)Hkv, (int)d, qt, type, &need) != DSA_OK ||
      ws.nbytes() < need)
    Py_RETURN_NONE;
  const at::Tensor out = at::empty({rows, Hq, d}, Q.options());
  at::Tensor lse;
  if (with_lse) lse = at::empty({rows, Hq}, Q.options().dtype(at::kFloat));
  float* l = with_lse ? static_cast<float*>(lse.data_ptr()) : nullptr;
  const int n_pages = (int)K.size(0), page = (int)K.size(1);
  const int r =
      idx ? selected(Q.data_ptr(), K.data_ptr(), t[2]->data_ptr(), ptr<float>(t[7]), ptr<float>(t[8]), ptr<int32_t>(t[3]),
                     ptr<int32_t>(t[4]), ptr<int32_t>(t[5]), ptr<int32_t>(idx), mid, (int)B, (int)rows, n_pages, page,
                     stride, (int)width, (int)Hq, (int)Hkv, (int)d, scale, qt, type, out.data_ptr(), l, ws.data_ptr(),
                     ws.nbytes(), stream(dev))
          : paged(Q.data_ptr(), K.data_ptr(), t[2]->data_ptr(), ptr<float>(t[7]), ptr<float>(t[8]), ptr<int32_t>(t[3]),
                  ptr<int32_t>(t[4]), ptr<int32_t>(t[5]), (int)B, (int)rows, max_q, n_pages, page, stride, (int)width,
                  (int)Hq, (int)Hkv, (int)d, scale, qt, type, out.data_ptr(), l, ws.data_ptr(), ws.nbytes(), stream(dev));
  if (r != DSA_OK) return PyLong_FromLong(r);
  if (!with_lse) return THPVariable_Wrap(out);
  PyObject* tuple = PyTuple_New(2);
  if (tuple) {
    PyTuple_SET_ITEM(tuple, 0, THPVariable_Wrap(out));
    PyTuple_SET_ITEM(tuple, 1, THPVariable_Wrap(lse));
  }
  return tuple;
}

// A C++ exception (an allocation that fails, say) becomes Python's.
template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_Clear();  // the caller's own allocation fails with torch's own error
    Py_RETURN_NONE;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

PyObject* py_page_plan(PyObject*, PyObject* const* args, Py_ssize_t n) {
  const at::Tensor* t[6];
  int x[3];
  if (n != 9 || !plan || !take(args[8], t[5])) Py_RETURN_NONE;
  for (int i = 0; i < 5; ++i)
    if (!take(args[i], t[i])) Py_RETURN_NONE;
  for (int i = 0; i < 3; ++i)
    if (!take_int(args[5 + i], x[i])) Py_RETURN_NONE;
  return guarded([&] { return page_plan(t, x[0], x[1], x[2]); });
}

PyObject* py_page_append(PyObject*, PyObject* const* args, Py_ssize_t n) {
  const at::Tensor* t[8];
  if (n != 8 || !append) Py_RETURN_NONE;
  for (int i = 0; i < 8; ++i)
    if (!take(args[i], t[i], i >= 3 && i < 7)) Py_RETURN_NONE;
  return guarded([&] { return page_append(t); });
}

PyObject* py_attend(PyObject*, PyObject* const* args, Py_ssize_t n) {
  const at::Tensor* t[10];
  int max_q = 0;
  float scale = 0.f;
  if (n != 13 || !paged || !take_int(args[10], max_q)) Py_RETURN_NONE;
  for (int i = 0; i < 10; ++i)
    if (!take(args[i], t[i], i >= 6 && i < 9)) Py_RETURN_NONE;
  const bool own_scale = args[11] != Py_None;
  if (own_scale) {
    if (!PyFloat_Check(args[11])) Py_RETURN_NONE;
    scale = (float)PyFloat_AS_DOUBLE(args[11]);
  }
  const bool with_lse = args[12] == Py_True;
  return guarded([&] { return attend(t, max_q, own_scale ? &scale : nullptr, with_lse); });
}

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(bind)), METH_FASTCALL, nullptr},
    {"page_plan", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_page_plan)), METH_FASTCALL, nullptr},
    {"page_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_page_append)), METH_FASTCALL, nullptr},
    {"attend", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_attend)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

// DSA_BUILT_FOR: the torch and Python of the build, by which the next one tells whether the binary fits
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_ext", DSA_BUILT_FOR, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged_ext() { return PyModule_Create(&module); }
