// The tensor side of layer_norm, layer_norm_backward, grad_norm and AdamW.step:
// checks tensors, allocates outputs and calls the C entry points, on the current
// stream.  A call of these costs the host more than the GPU when the tensors are
// small or many, so this is a Python extension in C++ and not ctypes: with that, the
// norm of 300 gradients took 365 us a call (here 18) and the norm of one row 25 us (7.5).
#include "binding.h"

#include <algorithm>
#include <vector>

PyObject* flce_binding::g_error = nullptr;

namespace {

using namespace flce_binding;

// layer_norm(x, weight, bias, kind, eps, residual, out, sum_out, row_stats) -> (y, sum, mean, rstd)
PyObject* layer_norm(PyObject*, PyObject* const* a, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  if (count != 9) return fail(FLCE_ERR_INVALID_ARG, "layer_norm: arguments");
  int device = -1;
  const at::Tensor *x, *w, *b, *r, *out, *sum_out;
  if (!tensor_of(a[0], "layer_norm: x", false, &x, &device) ||
      !tensor_of(a[1], "layer_norm: weight", true, &w, &device) ||
      !tensor_of(a[2], "layer_norm: bias", true, &b, &device) ||
      !tensor_of(a[5], "layer_norm: residual", true, &r, &device) ||
      !tensor_of(a[6], "layer_norm: out", true, &out, &device) ||
      !tensor_of(a[7], "layer_norm: sum_out", true, &sum_out, &device))
    return nullptr;
  const long kind = PyLong_AsLong(a[3]);
  const double eps = PyFloat_AsDouble(a[4]);
  if (PyErr_Occurred()) return nullptr;
  const int dtype = code_of(*x);
  if (dtype == kUnknown) return fail(FLCE_ERR_UNSUPPORTED, "layer_norm: x: its type");
  Rows m;
  int64_t ld_r = 0, ld_y, ld_s;
  if (!rows_of(*x, "layer_norm: x", &m)) return nullptr;
  ld_y = ld_s = m.h;
  if ((r != nullptr && !like(*r, *x, "layer_norm: residual", &ld_r)) ||
      (w != nullptr && !vector_of(*w, m.h, "layer_norm: weight")) ||
      (b != nullptr && !vector_of(*b, m.h, "layer_norm: bias")) ||
      (out != nullptr && !like(*out, *x, "layer_norm: out", &ld_y)) ||
      (sum_out != nullptr && !like(*sum_out, *x, "layer_norm: sum_out", &ld_s)))
    return nullptr;
  if (w != nullptr && b != nullptr && w->scalar_type() != b->scalar_type())
    return fail(FLCE_ERR_UNSUPPORTED, "layer_norm: weight and bias have different types");
  if (sum_out != nullptr && r == nullptr) return fail(FLCE_ERR_INVALID_ARG, "layer_norm: sum_out without residual");
  const bool stats = flag(a[8]);
  const at::IntArrayRef rows = x->sizes().slice(0, x->dim() - 1);
  const at::Tensor y = out != nullptr ? *out : at::empty(x->sizes(), x->options());
  const at::Tensor sum = sum_out != nullptr ? *sum_out
                         : r != nullptr     ? at::empty(x->sizes(), x->options())
                                            : at::Tensor();
  const at::Tensor mean = stats && kind == FLCE_NORM_LAYER ? floats(rows, *x) : at::Tensor();
  const at::Tensor rstd = stats ? floats(rows, *x) : at::Tensor();
  const at::Tensor* param = w != nullptr ? w : b;
  const flce_status_t st = ln_fwd(
      static_cast<int>(kind), dtype, data(x), m.ld, data(r), ld_r, data(w), data(b),
      param != nullptr ? code_of(*param) : dtype, m.n, m.h, static_cast<float>(eps), y.data_ptr(), ld_y,
      sum.defined() ? sum.data_ptr() : nullptr, ld_s, mean.defined() ? mean.data_ptr<float>() : nullptr,
      rstd.defined() ? rstd.data_ptr<float>() : nullptr, stream());
  if (st != FLCE_OK) return fail(st, "ln_fwd");
  written({out, sum_out});
  return tuple_of({&y, &sum, &mean, &rstd});
  END_HANDLE_TH_ERRORS
}

// layer_norm_backward(grad_y, x, weight, mean, rstd, kind, grad_sum, grad_x, grad_weight, grad_bias, out,
//                     grad_weight_out, grad_bias_out, accumulate, workspace) -> (grad_x, grad_weight, grad_bias)
PyObject* layer_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  if (count != 15) return fail(FLCE_ERR_INVALID_ARG, "layer_norm_backward: arguments");
  int device = -1;
  const at::Tensor *gy, *x, *w, *mean, *rstd, *gs, *out, *gw_out, *gb_out, *ws;
  if (!tensor_of(a[0], "layer_norm_backward: grad_y", false, &gy, &device) ||
      !tensor_of(a[1], "layer_norm_backward: x", false, &x, &device) ||
      !tensor_of(a[2], "layer_norm_backward: weight", true, &w, &device) ||
      !tensor_of(a[3], "layer_norm_backward: mean", true, &mean, &device) ||
      !tensor_of(a[4], "layer_norm_backward: rstd", false, &rstd, &device) ||
      !tensor_of(a[6], "layer_norm_backward: grad_sum", true, &gs, &device) ||
      !tensor_of(a[10], "layer_norm_backward: out", true, &out, &device) ||
      !tensor_of(a[11], "layer_norm_backward: grad_weight_out", true, &gw_out, &device) ||
      !tensor_of(a[12], "layer_norm_backward: grad_bias_out", true, &gb_out, &device) ||
      !tensor_of(a[14], "layer_norm_backward: workspace", true, &ws, &device))
    return nullptr;
  const long kind = PyLong_AsLong(a[5]);
  if (PyErr_Occurred()) return nullptr;
  const int dtype = code_of(*x);
  if (dtype == kUnknown) return fail(FLCE_ERR_UNSUPPORTED, "layer_norm_backward: x: its type");
  Rows m;
  int64_t ld_g, ld_s = 0, ld_x;
  if (!rows_of(*x, "layer_norm_backward: x", &m)) return nullptr;
  ld_x = m.h;
  if (!like(*gy, *x, "layer_norm_backward: grad_y", &ld_g) ||
      (w != nullptr && !vector_of(*w, m.h, "layer_norm_backward: weight")) ||
      (mean != nullptr && !floats_of(*mean, m.n, "layer_norm_backward: mean")) ||
      !floats_of(*rstd, m.n, "layer_norm_backward: rstd") ||
      (gs != nullptr && !like(*gs, *x, "layer_norm_backward: grad_sum", &ld_s)) ||
      (out != nullptr && !like(*out, *x, "layer_norm_backward: out", &ld_x)) ||
      (gw_out != nullptr && !floats_of(*gw_out, m.h, "layer_norm_backward: grad_weight_out")) ||
      (gb_out != nullptr && !floats_of(*gb_out, m.h, "layer_norm_backward: grad_bias_out")))
    return nullptr;
  const bool want_x = flag(a[7]) || out != nullptr, accumulate = flag(a[13]);
  const bool want_w = flag(a[8]) || gw_out != nullptr, want_b = flag(a[9]) || gb_out != nullptr;
  if (accumulate && ((want_w && gw_out == nullptr) || (want_b && gb_out == nullptr)))
    return fail(FLCE_ERR_INVALID_ARG, "layer_norm_backward: accumulate adds to grad_weight_out and grad_bias_out");
  const int64_t size = static_cast<int64_t>(ln_workspace_size(m.n, m.h));
  if (size == 0) return fail(FLCE_ERR_INVALID_ARG, "ln_workspace_size");
  const at::Tensor gx = out != nullptr ? *out : want_x ? at::empty(x->sizes(), x->options()) : at::Tensor();
  const at::Tensor gw = gw_out != nullptr ? *gw_out : want_w ? floats({m.h}, *x) : at::Tensor();
  const at::Tensor gb = gb_out != nullptr ? *gb_out : want_b ? floats({m.h}, *x) : at::Tensor();
  const bool given = ws != nullptr && ws->is_contiguous() && static_cast<int64_t>(ws->nbytes()) >= size;
  const at::Tensor scratch = given ? *ws : at::empty({size}, x->options().dtype(at::kByte));
  const flce_status_t st = ln_bwd(
      static_cast<int>(kind), dtype, data(gy), ld_g, data(x), m.ld, data(w), w ? code_of(*w) : dtype,
      static_cast<const float*>(data(mean)), static_cast<const float*>(data(rstd)), data(gs), ld_s, m.n, m.h,
      gx.defined() ? gx.data_ptr() : nullptr, ld_x, gw.defined() ? gw.data_ptr<float>() : nullptr,
      gb.defined() ? gb.data_ptr<float>() : nullptr, accumulate, scratch.data_ptr(), scratch.nbytes(), stream());
  if (st != FLCE_OK) return fail(st, "ln_bwd");
  written({out, gw_out, gb_out});
  return tuple_of({&gx, &gw, &gb});
  END_HANDLE_TH_ERRORS
}

// The members of a sequence, or what an iterator yields: held as long as this is, and
// so the memory of tensors that nobody else holds.
class Members {
 public:
  explicit Members(PyObject* sequence) : fast_(PySequence_Fast(sequence, "a sequence of tensors is wanted")) {}
  Members(const Members&) = delete;
  Members& operator=(const Members&) = delete;
  ~Members() { Py_XDECREF(fast_); }
  bool ok() const { return fast_ != nullptr; }  // else an error is set
  Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(fast_); }
  // Calls f(i, tensor or null) for each; false once f does.
  template <typename F>
  bool for_each(const char* where, F f) const {
    int device = -1;
    for (Py_ssize_t i = 0; i < size(); ++i) {
      const at::Tensor* t;
      if (!tensor_of(PySequence_Fast_GET_ITEM(fast_, i), where, true, &t, &device) || !f(i, t)) return false;
    }
    return true;
  }

 private:
  PyObject* fast_;
};

// grad_norm(grads, grad_scale, max_norm, eps, out, workspace) -> (norm, scale)
PyObject* grad_norm_of(PyObject*, PyObject* const* a, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  if (count != 6) return fail(FLCE_ERR_INVALID_ARG, "grad_norm: arguments");
  const Members grads(a[0]);
  if (!grads.ok()) return nullptr;
  std::vector<flce_tensor_t> table;
  table.reserve(static_cast<size_t>(grads.size()));
  const bool ok = grads.for_each("grad_norm", [&](Py_ssize_t, const at::Tensor* t) {
    if (t == nullptr) return true;
    const int dtype = code_of(*t);
    if (dtype == kUnknown) return fail(FLCE_ERR_UNSUPPORTED, "grad_norm: a tensor's type"), false;
    if (!t->is_contiguous()) return fail(FLCE_ERR_UNSUPPORTED, "grad_norm: a tensor that is not contiguous"), false;
    table.push_back({t->data_ptr(), t->numel(), dtype, 0});
    return true;
  });
  if (!ok) return nullptr;
  const double scale = PyFloat_AsDouble(a[1]), most = PyFloat_AsDouble(a[2]), eps = PyFloat_AsDouble(a[3]);
  if (PyErr_Occurred()) return nullptr;
  int device = -1;
  const at::Tensor *out, *ws;
  if (!tensor_of(a[4], "grad_norm: out", true, &out, &device) ||
      !tensor_of(a[5], "grad_norm: workspace", true, &ws, &device) ||
      (out != nullptr && !floats_of(*out, 2, "grad_norm: out")))
    return nullptr;
  const auto options = at::TensorOptions().device(at::kCUDA, c10::cuda::current_device());
  const int64_t size = static_cast<int64_t>(grad_norm_workspace_size(static_cast<int64_t>(table.size())));
  const at::Tensor result = out != nullptr ? *out : at::empty({2}, options.dtype(at::kFloat));
  const bool given = ws != nullptr && ws->is_contiguous() && static_cast<int64_t>(ws->nbytes()) >= size;
  const at::Tensor scratch = given ? *ws : at::empty({size}, options.dtype(at::kByte));
  const flce_status_t st =
      grad_norm(table.data(), static_cast<int64_t>(table.size()), static_cast<float>(scale), static_cast<float>(most),
                static_cast<float>(eps), result.data_ptr<float>(), scratch.data_ptr(), scratch.nbytes(), stream());
  if (st != FLCE_OK) return fail(st, "grad_norm");
  written({out});
  const at::Tensor flat = result.dim() == 1 ? result : result.view({2});
  const at::Tensor norm = flat.select(0, 0), factor = flat.select(0, 1);
  return tuple_of({&norm, &factor});
  END_HANDLE_TH_ERRORS
}

// The tensors of an optimiser: lists of parameters, moments, the moments' scales and
// copies, one entry for each parameter.
constexpr int kLists = 6;

bool lists_ok(PyObject* const* lists, Py_ssize_t count) {
  for (int k = 0; k < kLists; ++k)
    if (!PyList_Check(lists[k]) || PyList_GET_SIZE(lists[k]) != count)
      return fail(FLCE_ERR_INVALID_ARG, "AdamW: lists of %zd tensors are wanted", count), false;
  return true;
}

// Checks the tensors and fills the table and the element counts with them; on an error
// both stay as they were.
bool fill_table(PyObject* const* lists, Py_ssize_t count, flce_adamw_tensor_t* table, int64_t* sizes) {
  if (!lists_ok(lists, count)) return false;
  struct Span {
    uintptr_t from, to;
    Py_ssize_t tensor;
  };
  std::vector<Span> spans;
  std::vector<flce_adamw_tensor_t> filled(table, table + count);
  int device = -1;
  for (Py_ssize_t i = 0; i < count; ++i) {
    const at::Tensor* t[kLists];
    for (int k = 0; k < kLists; ++k) {
      if (!tensor_of(PyList_GET_ITEM(lists[k], i), "AdamW: a tensor", k > 2, &t[k], &device)) return false;
      if (t[k] != nullptr && !t[k]->is_contiguous())
        return fail(FLCE_ERR_UNSUPPORTED, "AdamW: tensor %zd: not contiguous", i), false;
    }
    const int64_t n = t[0]->numel(), blocks = (n + FLCE_ADAMW_BLOCK - 1) / FLCE_ADAMW_BLOCK;
    flce_adamw_tensor_t& e = filled[static_cast<size_t>(i)];
    e.param_dtype = code_of(*t[0]);
    e.copy_dtype = t[5] != nullptr ? code_of(*t[5]) : FLCE_DTYPE_BF16;
    if (e.param_dtype == kUnknown || e.copy_dtype == kUnknown)
      return fail(FLCE_ERR_UNSUPPORTED, "AdamW: tensor %zd: its type, or its copy's", i), false;
    const bool scaled = t[1]->scalar_type() == at::kFloat8_e4m3fn;
    if (t[1]->scalar_type() != t[2]->scalar_type() || (!scaled && t[1]->scalar_type() != at::kFloat))
      return fail(FLCE_ERR_UNSUPPORTED, "AdamW: tensor %zd: moments are both fp32 or both float8_e4m3fn", i), false;
    if (t[1]->numel() != n || t[2]->numel() != n || (t[5] != nullptr && t[5]->numel() != n))
      return fail(FLCE_ERR_INVALID_ARG, "AdamW: tensor %zd: moments or copy of another size", i), false;
    for (int k = 3; k < 5; ++k) {
      if (scaled != (t[k] != nullptr))
        return fail(FLCE_ERR_INVALID_ARG, "AdamW: tensor %zd: 8-bit moments come with scales, fp32 ones without", i),
               false;
      if (scaled && !floats_of(*t[k], blocks, "AdamW: scales")) return false;
    }
    void* at[kLists];
    for (int k = 0; k < kLists; ++k) {
      at[k] = t[k] != nullptr ? t[k]->data_ptr() : nullptr;
      const uintptr_t from = reinterpret_cast<uintptr_t>(at[k]);
      if (t[k] != nullptr && t[k]->nbytes() > 0) spans.push_back({from, from + t[k]->nbytes(), i});
    }
    e.param = at[0], e.exp_avg = at[1], e.exp_avg_sq = at[2];
    e.exp_avg_scale = static_cast<float*>(at[3]), e.exp_avg_sq_scale = static_cast<float*>(at[4]), e.copy = at[5];
    e.moment_bits = scaled ? 8 : 32;
    e.n = n;
  }
  std::sort(spans.begin(), spans.end(), [](const Span& x, const Span& y) { return x.from < y.from; });
  for (size_t k = 1; k < spans.size(); ++k)
    if (spans[k].from < spans[k - 1].to)
      return fail(FLCE_ERR_INVALID_ARG, "AdamW: tensors %zd and %zd share memory", spans[k - 1].tensor,
                  spans[k].tensor),
             false;
  std::copy(filled.begin(), filled.end(), table);
  for (Py_ssize_t i = 0; i < count; ++i) sizes[i] = table[i].n;
  return true;
}

// Whether the table still says where the tensors lie and what they are: a parameter may
// have been given other memory (`p.data = ...`, a model that was moved) and a list's
// entry another tensor since it was filled.  A step asks this of every tensor, at 17 ns
// each (with at::Tensor's functions 28), by TensorImpl's inline functions and by the first
// tensor's GPU: an address is one GPU's alone.
bool table_holds(PyObject* const* lists, Py_ssize_t count, const flce_adamw_tensor_t* table, const int64_t* sizes) {
  if (count == 0) return true;
  caffe2::TypeMeta type_of[3];
  type_of[FLCE_DTYPE_BF16] = c10::scalarTypeToTypeMeta(at::kBFloat16);
  type_of[FLCE_DTYPE_FP32] = c10::scalarTypeToTypeMeta(at::kFloat);
  type_of[FLCE_DTYPE_FP16] = c10::scalarTypeToTypeMeta(at::kHalf);
  const caffe2::TypeMeta fp32 = type_of[FLCE_DTYPE_FP32], e4m3 = c10::scalarTypeToTypeMeta(at::kFloat8_e4m3fn);
  const auto impl_of = [](PyObject* o) -> const c10::TensorImpl* {
    return THPVariable_Check(o) ? THPVariable_Unpack(o).unsafeGetTensorImpl() : nullptr;
  };
  const auto same = [&](PyObject* list, Py_ssize_t i, const void* at, caffe2::TypeMeta type, size_t esz, int64_t n) {
    PyObject* const o = PyList_GET_ITEM(list, i);
    if (o == Py_None) return at == nullptr;
    const c10::TensorImpl* const t = impl_of(o);
    if (t == nullptr || t->dtype() != type || t->numel() != n || !t->is_contiguous() || !t->has_storage()) return false;
    const char* const storage = static_cast<const char*>(t->unsafe_storage().unsafeGetStorageImpl()->data());
    return n == 0 || storage + static_cast<size_t>(t->storage_offset()) * esz == at;
  };
  const c10::TensorImpl* const first = impl_of(PyList_GET_ITEM(lists[0], 0));
  if (first == nullptr || first->device() != c10::Device(c10::kCUDA, c10::cuda::current_device())) return false;
  const auto size_of = [](int dtype) { return dtype == FLCE_DTYPE_FP32 ? 4u : 2u; };
  for (Py_ssize_t i = 0; i < count; ++i) {
    const flce_adamw_tensor_t& e = table[i];
    const int64_t n = sizes[i], blocks = (n + FLCE_ADAMW_BLOCK - 1) / FLCE_ADAMW_BLOCK;
    const caffe2::TypeMeta moment = e.moment_bits == 8 ? e4m3 : fp32;
    if (!same(lists[0], i, e.param, type_of[e.param_dtype], size_of(e.param_dtype), n) ||
        !same(lists[1], i, e.exp_avg, moment, e.moment_bits / 8, n) ||
        !same(lists[2], i, e.exp_avg_sq, moment, e.moment_bits / 8, n) ||
        !same(lists[3], i, e.exp_avg_scale, fp32, 4, blocks) ||
        !same(lists[4], i, e.exp_avg_sq_scale, fp32, 4, blocks) ||
        !same(lists[5], i, e.copy, type_of[e.copy_dtype], size_of(e.copy_dtype), n))
      return false;
  }
  return true;
}

// adamw_table(table, sizes, params, exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale, copies, weight_decay,
// lr_scale): checks an optimiser's tensors, lists of one length, and fills the table at address `table` and the
// element counts at `sizes` with them.
PyObject* adamw_table(PyObject*, PyObject* const* a, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  if (count != 10) return fail(FLCE_ERR_INVALID_ARG, "AdamW: arguments");
  auto* table = static_cast<flce_adamw_tensor_t*>(PyLong_AsVoidPtr(a[0]));
  auto* sizes = static_cast<int64_t*>(PyLong_AsVoidPtr(a[1]));
  if (PyErr_Occurred()) return nullptr;
  for (const int k : {2, 8, 9})
    if (!PyList_Check(a[k]) || PyList_GET_SIZE(a[k]) != PyList_GET_SIZE(a[2]))
      return fail(FLCE_ERR_INVALID_ARG, "AdamW: lists of one length are wanted");
  const Py_ssize_t tensors = PyList_GET_SIZE(a[2]);
  for (Py_ssize_t i = 0; i < tensors; ++i) {
    table[i].weight_decay = static_cast<float>(PyFloat_AsDouble(PyList_GET_ITEM(a[8], i)));
    table[i].lr_scale = static_cast<float>(PyFloat_AsDouble(PyList_GET_ITEM(a[9], i)));
    if (PyErr_Occurred()) return nullptr;
  }
  if (!fill_table(a + 2, tensors, table, sizes)) return nullptr;
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// A number, or a device fp32 element whose address goes to *at.
bool number_of(PyObject* o, const char* where, int* device, double* value, const float** at) {
  *at = nullptr;
  if (!THPVariable_Check(o)) {
    *value = PyFloat_AsDouble(o);
    return !PyErr_Occurred();
  }
  const at::Tensor* t;
  if (!tensor_of(o, where, false, &t, device) || !floats_of(*t, 1, where)) return false;
  *value = 0;
  *at = t->data_ptr<float>();
  return true;
}

// adamw(table, sizes, count, numbers, grads, lr, grad_scale, skip_nonfinite, step, params, exp_avg, exp_avg_sq,
// exp_avg_scale, exp_avg_sq_scale, copies): fills the table of flce_adamw_tensor_t at address `table` again if the
// tensors of the lists are no longer those in it, fills in the gradients (an element count of 0 where there is none)
// and the step's numbers (the flce_adamw_t at `numbers`), and takes the step.
PyObject* adamw(PyObject*, PyObject* const* a, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  if (count != 9 + kLists) return fail(FLCE_ERR_INVALID_ARG, "AdamW.step: arguments");
  auto* table = static_cast<flce_adamw_tensor_t*>(PyLong_AsVoidPtr(a[0]));
  auto* sizes = static_cast<int64_t*>(PyLong_AsVoidPtr(a[1]));
  const Py_ssize_t tensors = PyLong_AsSsize_t(a[2]);
  auto* numbers = static_cast<flce_adamw_t*>(PyLong_AsVoidPtr(a[3]));
  if (PyErr_Occurred()) return nullptr;
  const Members grads(a[4]);  // before the rest is looked at: an iterator may move anything
  if (!grads.ok()) return nullptr;
  if (grads.size() != tensors)
    return fail(FLCE_ERR_INVALID_ARG, "AdamW.step: %zd gradients for %zd tensors", grads.size(), tensors);
  int on = -1;
  double factor = 1;
  if (!number_of(a[5], "AdamW.step: lr", &on, &numbers->lr, &numbers->lr_dev)) return nullptr;
  numbers->grad_scale_dev = nullptr;
  if (a[6] != Py_None && !number_of(a[6], "AdamW.step: grad_scale", &on, &factor, &numbers->grad_scale_dev))
    return nullptr;
  numbers->grad_scale = static_cast<float>(factor);
  numbers->skip_nonfinite = flag(a[7]);
  numbers->step = PyLong_AsLongLong(a[8]);
  if (PyErr_Occurred()) return nullptr;
  if (!lists_ok(a + 9, tensors)) return nullptr;
  if (!table_holds(a + 9, tensors, table, sizes) && !fill_table(a + 9, tensors, table, sizes)) return nullptr;
  const bool ok = grads.for_each("AdamW.step", [&](Py_ssize_t i, const at::Tensor* t) {
    flce_adamw_tensor_t& e = table[i];
    e.n = 0;
    if (t == nullptr) return true;
    const int dtype = code_of(*t);
    if (dtype == kUnknown) return fail(FLCE_ERR_UNSUPPORTED, "AdamW.step: a gradient's type"), false;
    if (!t->is_contiguous() || t->numel() != sizes[i])
      return fail(FLCE_ERR_INVALID_ARG, "AdamW.step: gradient %zd is no contiguous tensor of %lld elements", i,
                  (long long)sizes[i]),
             false;
    e.grad = t->data_ptr();
    e.grad_dtype = dtype;
    e.n = sizes[i];
    return true;
  });
  if (!ok) return nullptr;
  const flce_status_t st = adamw_step(table, tensors, numbers, stream());
  if (st != FLCE_OK) return fail(st, "adamw_step");
  // parameters and copies; moments are in no graph
  for (Py_ssize_t i = 0; i < tensors; ++i) {
    if (table[i].n == 0) continue;
    PyObject* const copy = PyList_GET_ITEM(a[9 + 5], i);
    written({&THPVariable_Unpack(PyList_GET_ITEM(a[9], i)), copy != Py_None ? &THPVariable_Unpack(copy) : nullptr});
  }
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// set_error(type): the exception to raise.
PyObject* set_error(PyObject*, PyObject* type) {
  Py_INCREF(type);
  Py_XSETREF(g_error, type);
  Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"layer_norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(layer_norm)), METH_FASTCALL, nullptr},
    {"layer_norm_backward", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(layer_norm_backward)),
     METH_FASTCALL, nullptr},
    {"grad_norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(grad_norm_of)), METH_FASTCALL, nullptr},
    {"adamw", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(adamw)), METH_FASTCALL, nullptr},
    {"adamw_table", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(adamw_table)), METH_FASTCALL, nullptr},
    {"policy_loss", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(policy_loss)), METH_FASTCALL, nullptr},
    {"preference_loss", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(preference_loss)), METH_FASTCALL,
     nullptr},
    {"distillation_loss", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(distillation_loss)),
     METH_FASTCALL, nullptr},
    {"embedding", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(embedding)), METH_FASTCALL, nullptr},
    {"embedding_backward", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(embedding_backward)),
     METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "flce_torch", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_flce_torch(void) { return PyModule_Create(&kModule); }
