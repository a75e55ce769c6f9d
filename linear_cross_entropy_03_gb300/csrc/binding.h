// What the extension's sources share: checks of tensors, and errors.
#pragma once

#include <Python.h>

#include <cstdarg>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/flce.h"

namespace flce_binding {

extern PyObject* g_error;  // FlceError(status, where)

// Raises FlceError; to be returned.
inline PyObject* fail(int status, const char* format, ...) {
  va_list args;
  va_start(args, format);
  PyObject* where = PyUnicode_FromFormatV(format, args);
  va_end(args);
  if (where == nullptr) return nullptr;
  PyObject* e = PyObject_CallFunction(g_error, "iO", status, where);
  Py_DECREF(where);
  if (e != nullptr) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  return nullptr;
}

constexpr int kUnknown = -1;

inline int code_of(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return FLCE_DTYPE_BF16;
    case at::kFloat: return FLCE_DTYPE_FP32;
    case at::kHalf: return FLCE_DTYPE_FP16;
    default: return kUnknown;
  }
}

// An argument that is a tensor on the current GPU, or None where that is allowed.
// `device`: the current GPU, looked up with the first tensor (-1 before).
inline bool tensor_of(PyObject* o, const char* where, bool optional, const at::Tensor** t, int* device) {
  *t = nullptr;
  if (o == Py_None && optional) return true;
  if (!THPVariable_Check(o)) return fail(FLCE_ERR_INVALID_ARG, "%s: a tensor is wanted", where), false;
  *t = &THPVariable_Unpack(o);
  if ((*t)->is_cuda()) {
    if (*device < 0) *device = c10::cuda::current_device();
    if ((*t)->get_device() == *device) return true;
  }
  return fail(FLCE_ERR_INVALID_ARG, "%s: not on the current GPU", where), false;
}

// A matrix: rows of contiguous elements at one distance.
struct Rows {
  int64_t n = 0, h = 0, ld = 0;
};

inline bool rows_of(const at::Tensor& t, const char* where, Rows* r) {
  r->h = t.dim() > 0 ? t.size(-1) : 0;
  if (r->h < 1) return fail(FLCE_ERR_INVALID_ARG, "%s: no columns", where), false;
  r->ld = r->h;
  if (t.is_contiguous()) {
    r->n = t.numel() / r->h;
    return true;
  }
  if (r->h > 1 && t.stride(-1) != 1)
    return fail(FLCE_ERR_UNSUPPORTED, "%s: its last dimension is not contiguous", where), false;
  r->n = 1;
  for (int64_t d = t.dim() - 2; d >= 0; --d) {
    if (t.size(d) == 1) continue;
    if (r->n > 1 && t.stride(d) != r->ld * r->n)
      return fail(FLCE_ERR_UNSUPPORTED, "%s: its rows have no one distance", where), false;
    if (r->n == 1) r->ld = t.stride(d);
    r->n *= t.size(d);
  }
  return true;
}

// A second matrix of the first's shape and type.
inline bool like(const at::Tensor& t, const at::Tensor& x, const char* where, int64_t* ld, const char* first = "x") {
  if (t.scalar_type() != x.scalar_type() || t.sizes() != x.sizes())
    return fail(FLCE_ERR_INVALID_ARG, "%s: of another shape or type than %s", where, first), false;
  Rows r;
  if (!rows_of(t, where, &r)) return false;
  *ld = r.ld;
  return true;
}

inline bool vector_of(const at::Tensor& t, int64_t h, const char* where) {
  if (t.dim() != 1 || t.size(0) != h || !t.is_contiguous())
    return fail(FLCE_ERR_INVALID_ARG, "%s: a contiguous vector of %lld elements is wanted", where, (long long)h), false;
  if (code_of(t) == kUnknown) return fail(FLCE_ERR_UNSUPPORTED, "%s: its type", where), false;
  return true;
}

inline bool floats_of(const at::Tensor& t, int64_t n, const char* where) {
  if (t.scalar_type() != at::kFloat || t.numel() != n || !t.is_contiguous())
    return fail(FLCE_ERR_INVALID_ARG, "%s: a contiguous fp32 tensor of %lld elements is wanted", where, (long long)n),
           false;
  return true;
}

inline flce_stream_t stream() { return reinterpret_cast<flce_stream_t>(c10::cuda::getCurrentCUDAStream().stream()); }

inline const void* data(const at::Tensor* t) { return t == nullptr ? nullptr : t->data_ptr(); }

inline at::Tensor floats(at::IntArrayRef shape, const at::Tensor& by) {
  return at::empty(shape, by.options().dtype(at::kFloat));
}

// A tuple of tensors, undefined ones as None.
inline PyObject* tuple_of(std::initializer_list<const at::Tensor*> tensors) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(tensors.size()));
  if (r == nullptr) return nullptr;
  Py_ssize_t i = 0;
  for (const at::Tensor* t : tensors) {
    PyObject* o = t->defined() ? THPVariable_Wrap(*t) : Py_NewRef(Py_None);
    if (o == nullptr) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// Tells autograd that tensors were written, as torch's own operations in place do: a
// backward pass that saved what they held is then refused, and not run on other numbers.
inline void written(std::initializer_list<const at::Tensor*> tensors) {
  for (const at::Tensor* t : tensors)
    if (t != nullptr && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

inline bool flag(PyObject* o) { return o != Py_None && PyObject_IsTrue(o) == 1; }

// The functions of binding_losses.cpp.
PyObject* policy_loss(PyObject*, PyObject* const* a, Py_ssize_t count);
PyObject* preference_loss(PyObject*, PyObject* const* a, Py_ssize_t count);
PyObject* distillation_loss(PyObject*, PyObject* const* a, Py_ssize_t count);
PyObject* embedding(PyObject*, PyObject* const* a, Py_ssize_t count);
PyObject* embedding_backward(PyObject*, PyObject* const* a, Py_ssize_t count);

}  // namespace flce_binding
