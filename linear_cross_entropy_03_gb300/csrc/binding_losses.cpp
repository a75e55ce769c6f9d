// The tensor side of policy_loss, preference_loss, distillation_loss, embedding and
// embedding_backward (binding.cpp says why this is C++).
#include "binding.h"

#include <ATen/cuda/EmptyTensor.h>

namespace flce_binding {
namespace {

// An uninitialised tensor on the GPU of another one.  (at::empty takes twice as long to get
// to the same place, and a call makes up to four.)
at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, const at::Tensor& by) {
  return at::detail::empty_cuda(shape, type, by.device(), std::nullopt);
}

// The first four bytes of a workspace (its status word), as a tensor that shares its memory.
at::Tensor first_word(const at::Tensor& workspace) {
  auto impl = c10::make_intrusive<c10::TensorImpl>(c10::Storage(workspace.storage()),
                                                   c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                   caffe2::TypeMeta::Make<int32_t>());
  impl->set_sizes_contiguous({1});
  impl->set_storage_offset(workspace.storage_offset() * static_cast<int64_t>(workspace.itemsize()) / 4);
  return at::Tensor(std::move(impl));
}

// Whether a tensor of as many elements as `shape` has them in the same order: both are alike
// but for dimensions of one element, or one of them is flat.
bool in_order(at::IntArrayRef sizes, at::IntArrayRef shape) {
  c10::SmallVector<int64_t, 6> a, b;
  for (const int64_t n : sizes)
    if (n != 1) a.push_back(n);
  for (const int64_t n : shape)
    if (n != 1) b.push_back(n);
  return a.size() <= 1 || b.size() <= 1 || a == b;
}

// What the losses on logits take and return alike.
struct Call {
  const char* name;
  int device = -1;
  const at::Tensor *logits = nullptr, *grad_out = nullptr, *buffer = nullptr, *workspace = nullptr, *status = nullptr;
  Rows rows;
  int64_t ld_grad = 0;
  int dtype = 0, reduction = 0;
  float grad_scale = 1;
  bool want_grad = true;
  at::Tensor loss, grad, scratch, word;

  // PyUnicode_FromFormat's arguments: "<name>: <argument>"
  PyObject* bad(int status, const char* what) const { return fail(status, "%s: %s", name, what); }

  bool tensor(PyObject* o, const char* what, bool optional, const at::Tensor** t) {
    *t = nullptr;
    if (o == Py_None && optional) return true;
    if (!THPVariable_Check(o)) return fail(FLCE_ERR_INVALID_ARG, "%s: %s: a tensor is wanted", name, what), false;
    return tensor_of(o, name, optional, t, &device);
  }

  // logits, reduction, grad_scale, grad_out, in_place, want_grad, grad_out_buffer, workspace, status
  bool take(PyObject* const* a) {
    if (!tensor(a[0], "logits", false, &logits) || !tensor(a[3], "grad_out", true, &grad_out) ||
        !tensor(a[6], "grad_out_buffer", true, &buffer) || !tensor(a[7], "workspace", true, &workspace) ||
        !tensor(a[8], "status", true, &status))
      return false;
    reduction = static_cast<int>(PyLong_AsLong(a[1]));
    grad_scale = static_cast<float>(PyFloat_AsDouble(a[2]));
    if (PyErr_Occurred()) return false;
    dtype = code_of(*logits);
    if (dtype == kUnknown) return bad(FLCE_ERR_UNSUPPORTED, "logits: their type"), false;
    if (logits->dim() < 2) return bad(FLCE_ERR_INVALID_ARG, "logits: rows of logits are wanted"), false;
    if (!rows_of(*logits, name, &rows)) return false;
    want_grad = flag(a[5]);
    const bool in_place = flag(a[4]);
    if (in_place && (!want_grad || buffer != nullptr))
      return bad(FLCE_ERR_INVALID_ARG, "in_place with another place for the gradient, or none"), false;
    if (buffer != nullptr && !want_grad) return bad(FLCE_ERR_INVALID_ARG, "grad_out_buffer without a gradient"), false;
    ld_grad = rows.h;
    if (in_place) buffer = logits;
    if (buffer != nullptr && !like(*buffer, *logits, name, &ld_grad, "logits")) return false;
    if (status != nullptr && (status->scalar_type() != at::kInt || status->numel() != 1))
      return bad(FLCE_ERR_INVALID_ARG, "status: one int32 element is wanted"), false;
    if (losses_of_none >= 0) return list_floats(grad_out, {1, losses_of_none}, "grad_out");
    return row_floats(grad_out, "grad_out");
  }

  int64_t losses_of_none = -1;  // where they are not the rows

  // floats of a shape that is not the rows'
  bool list_floats(const at::Tensor* t, at::IntArrayRef shape, const char* what) const {
    if (t == nullptr || (t->scalar_type() == at::kFloat && t->is_contiguous() && t->numel() == c10::multiply_integers(shape) &&
                         in_order(t->sizes(), shape)))
      return true;
    return fail(FLCE_ERR_INVALID_ARG, "%s: %s: a contiguous fp32 vector of %lld elements is wanted", name, what,
                static_cast<long long>(c10::multiply_integers(shape))), false;
  }

  // an element for each row
  bool row_floats(const at::Tensor* t, const char* what) const {
    if (t == nullptr || (t->scalar_type() == at::kFloat && of_rows(*t))) return true;
    return fail(FLCE_ERR_INVALID_ARG, "%s: %s: a contiguous fp32 tensor of the logits' shape without the last "
                "dimension is wanted", name, what), false;
  }
  bool row_targets(const at::Tensor& t) const {
    if (t.scalar_type() != at::kLong) return bad(FLCE_ERR_UNSUPPORTED, "target: int64 is wanted"), false;
    if (of_rows(t)) return true;
    return bad(FLCE_ERR_INVALID_ARG, "target: a contiguous tensor of the logits' shape without the last dimension is "
               "wanted"), false;
  }
  bool of_rows(const at::Tensor& t) const {
    return t.is_contiguous() && t.numel() == rows.n && in_order(t.sizes(), row_shape());
  }

  at::IntArrayRef row_shape() const { return logits->sizes().slice(0, logits->dim() - 1); }

  void allocate(int64_t workspace_bytes, at::IntArrayRef loss_shape) {
    loss = empty(reduction == FLCE_REDUCTION_NONE ? loss_shape : at::IntArrayRef{}, at::kFloat, *logits);
    if (buffer != nullptr)
      grad = *buffer;
    else if (want_grad)
      grad = empty(logits->sizes(), logits->scalar_type(), *logits);
    const bool given = workspace != nullptr && workspace->is_contiguous() &&
                       static_cast<int64_t>(workspace->nbytes()) >= workspace_bytes;
    scratch = given ? *workspace : empty({workspace_bytes}, at::kByte, *logits);
    word = status != nullptr ? *status : first_word(scratch);
  }

  int32_t* status_ptr() const { return status != nullptr ? status->data_ptr<int32_t>() : nullptr; }
  void* grad_ptr() const { return grad.defined() ? grad.data_ptr() : nullptr; }
  const float* grad_out_ptr() const { return static_cast<const float*>(data(grad_out)); }
};

const float* f32(const at::Tensor* t) { return static_cast<const float*>(data(t)); }

int index_type_of(const at::Tensor& t) {
  return t.scalar_type() == at::kLong ? FLCE_INDEX_INT64 : t.scalar_type() == at::kInt ? FLCE_INDEX_INT32 : kUnknown;
}

}  // namespace

// policy_loss(logits, reduction, grad_scale, grad_out, in_place, want_grad, grad_out_buffer, workspace, status,
//             target, advantage, old_logp, ref_logp, row_weight, clip_low, clip_high, kl_weight, temperature,
//             ignore_index) -> (loss, grad_logits, logp, status)
PyObject* policy_loss(PyObject*, PyObject* const* a, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  Call c{"policy_loss"};
  if (count != 19) return c.bad(FLCE_ERR_INVALID_ARG, "arguments");
  const at::Tensor *target, *advantage, *old_logp, *ref_logp, *weight;
  if (!c.take(a) || !c.tensor(a[9], "target", false, &target) || !c.tensor(a[10], "advantage", false, &advantage) ||
      !c.tensor(a[11], "old_logp", true, &old_logp) || !c.tensor(a[12], "ref_logp", true, &ref_logp) ||
      !c.tensor(a[13], "row_weight", true, &weight))
    return nullptr;
  flce_policy_t numbers;
  numbers.clip_low = static_cast<float>(PyFloat_AsDouble(a[14]));
  numbers.clip_high = static_cast<float>(PyFloat_AsDouble(a[15]));
  numbers.kl_weight = static_cast<float>(PyFloat_AsDouble(a[16]));
  numbers.temperature = static_cast<float>(PyFloat_AsDouble(a[17]));
  const int64_t ignore_index = PyLong_AsLongLong(a[18]);
  if (PyErr_Occurred()) return nullptr;
  if (!c.row_targets(*target) || !c.row_floats(advantage, "advantage") || !c.row_floats(old_logp, "old_logp") ||
      !c.row_floats(ref_logp, "ref_logp") || !c.row_floats(weight, "row_weight"))
    return nullptr;
  if (numbers.kl_weight != 0.f && ref_logp == nullptr && c.rows.n > 0)
    return c.bad(FLCE_ERR_INVALID_ARG, "ref_logp: wanted where kl_weight is not 0");
  const size_t size = row_loss_workspace_size(c.rows.n);
  if (size == 0) return c.bad(FLCE_ERR_INVALID_ARG, "too many rows");
  c.allocate(static_cast<int64_t>(size), c.row_shape());
  const at::Tensor logp = empty(c.row_shape(), at::kFloat, *c.logits);
  const flce_status_t st = policy_fwd_bwd(
      data(c.logits), c.dtype, c.rows.ld, c.grad_ptr(), c.ld_grad, target->data_ptr<int64_t>(), f32(advantage),
      f32(old_logp), f32(ref_logp), f32(weight), c.rows.n, c.rows.h, &numbers, ignore_index, c.reduction, c.grad_scale,
      c.grad_out_ptr(), c.loss.data_ptr<float>(), logp.data_ptr<float>(), c.scratch.data_ptr(), c.scratch.nbytes(),
      c.status_ptr(), stream());
  if (st != FLCE_OK) return fail(st, "policy_fwd_bwd");
  written({c.buffer, c.status});
  return tuple_of({&c.loss, &c.grad, &logp, &c.word});
  END_HANDLE_TH_ERRORS
}

// distillation_loss(logits, reduction, grad_scale, grad_out, in_place, want_grad, grad_out_buffer, workspace, status,
//                   ids, values, row_weight, temperature) -> (loss, grad_logits, status)
PyObject* distillation_loss(PyObject*, PyObject* const* a, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  Call c{"distillation_loss"};
  if (count != 13) return c.bad(FLCE_ERR_INVALID_ARG, "arguments");
  const at::Tensor *ids, *values, *weight;
  if (!c.take(a) || !c.tensor(a[9], "teacher_ids", false, &ids) ||
      !c.tensor(a[10], "teacher_logits", false, &values) || !c.tensor(a[11], "row_weight", true, &weight))
    return nullptr;
  const float temperature = static_cast<float>(PyFloat_AsDouble(a[12]));
  if (PyErr_Occurred()) return nullptr;
  const int index_type = index_type_of(*ids), value_type = code_of(*values);
  if (index_type == kUnknown || value_type == kUnknown)
    return c.bad(FLCE_ERR_UNSUPPORTED, "the type of the teacher's ids or logits");
  const int64_t top = ids->dim() > 0 ? ids->size(-1) : 0;
  if (top < 1 || ids->sizes() != values->sizes() || ids->dim() != c.logits->dim() ||
      ids->sizes().slice(0, ids->dim() - 1) != c.row_shape() || !ids->is_contiguous() || !values->is_contiguous())
    return c.bad(FLCE_ERR_INVALID_ARG, "teacher: contiguous ids and logits, a list for each row, are wanted");
  if (!c.row_floats(weight, "row_weight")) return nullptr;
  const size_t size = row_loss_workspace_size(c.rows.n);
  if (size == 0) return c.bad(FLCE_ERR_INVALID_ARG, "too many rows");
  c.allocate(static_cast<int64_t>(size), c.row_shape());
  const flce_status_t st = distill_fwd_bwd(
      data(c.logits), c.dtype, c.rows.ld, c.grad_ptr(), c.ld_grad, data(ids), index_type, data(values), value_type, top,
      f32(weight), c.rows.n, c.rows.h, temperature, c.reduction, c.grad_scale, c.grad_out_ptr(),
      c.loss.data_ptr<float>(), c.scratch.data_ptr(), c.scratch.nbytes(), c.status_ptr(), stream());
  if (st != FLCE_OK) return fail(st, "distill_fwd_bwd");
  written({c.buffer, c.status});
  return tuple_of({&c.loss, &c.grad, &c.word});
  END_HANDLE_TH_ERRORS
}

// preference_loss(logits, reduction, grad_scale, grad_out, in_place, want_grad, grad_out_buffer, workspace, status,
//                 target, offsets, ref_logp, kind, beta, label_smoothing, margin, average, ignore_index)
//     -> (loss, grad_logits, logp, status)
PyObject* preference_loss(PyObject*, PyObject* const* a, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  Call c{"preference_loss"};
  if (count != 18) return c.bad(FLCE_ERR_INVALID_ARG, "arguments");
  const at::Tensor *offsets, *target, *ref_logp, *logits;
  if (!c.tensor(a[0], "logits", false, &logits) || !c.tensor(a[10], "offsets", true, &offsets)) return nullptr;
  int64_t sequences;
  if (offsets != nullptr) {
    if (offsets->scalar_type() != at::kLong || offsets->dim() != 1 || !offsets->is_contiguous() ||
        offsets->numel() % 2 != 1)
      return c.bad(FLCE_ERR_INVALID_ARG, "offsets: a contiguous int64 vector of 2 * pairs + 1 elements is wanted");
    sequences = offsets->numel() - 1;
  } else {
    if (logits->dim() < 3 || logits->size(0) % 2 != 0)
      return c.bad(FLCE_ERR_INVALID_ARG, "logits: [2 * pairs, tokens, V] is wanted where offsets are not given");
    sequences = logits->size(0);
  }
  c.losses_of_none = sequences / 2;
  if (!c.take(a) || !c.tensor(a[9], "target", false, &target) || !c.tensor(a[11], "ref_logp", true, &ref_logp))
    return nullptr;
  flce_preference_t numbers;
  numbers.kind = static_cast<int32_t>(PyLong_AsLong(a[12]));
  numbers.beta = static_cast<float>(PyFloat_AsDouble(a[13]));
  numbers.label_smoothing = static_cast<float>(PyFloat_AsDouble(a[14]));
  numbers.margin = static_cast<float>(PyFloat_AsDouble(a[15]));
  numbers.average = flag(a[16]) ? 1 : 0;
  const int64_t ignore_index = PyLong_AsLongLong(a[17]);
  if (PyErr_Occurred()) return nullptr;
  if (!c.row_targets(*target) || !c.list_floats(ref_logp, {2, sequences / 2}, "ref_logp")) return nullptr;
  const size_t size = preference_workspace_size(c.rows.n, sequences / 2);
  if (size == 0) return c.bad(FLCE_ERR_INVALID_ARG, "too many rows");
  c.allocate(static_cast<int64_t>(size), {sequences / 2});
  const at::Tensor logp = empty({sequences}, at::kFloat, *c.logits);
  const flce_status_t st = preference_fwd_bwd(
      data(c.logits), c.dtype, c.rows.ld, c.grad_ptr(), c.ld_grad, target->data_ptr<int64_t>(),
      offsets != nullptr ? offsets->data_ptr<int64_t>() : nullptr, f32(ref_logp), sequences / 2, c.rows.n, c.rows.h,
      &numbers, ignore_index, c.reduction, c.grad_scale, c.grad_out_ptr(), c.loss.data_ptr<float>(),
      logp.data_ptr<float>(), c.scratch.data_ptr(), c.scratch.nbytes(), c.status_ptr(), stream());
  if (st != FLCE_OK) return fail(st, "preference_fwd_bwd");
  written({c.buffer, c.status});
  return tuple_of({&c.loss, &c.grad, &logp, &c.word});
  END_HANDLE_TH_ERRORS
}

namespace {

bool status_of(PyObject* o, const char* where, int* device, int32_t** at, const at::Tensor** t) {
  *at = nullptr;
  if (!tensor_of(o, where, true, t, device)) return false;
  if (*t == nullptr) return true;
  if ((*t)->scalar_type() != at::kInt || (*t)->numel() != 1)
    return fail(FLCE_ERR_INVALID_ARG, "%s: one int32 element is wanted", where), false;
  *at = (*t)->data_ptr<int32_t>();
  return true;
}

}  // namespace

// embedding(weight, ids, scale, out, status) -> y
PyObject* embedding(PyObject*, PyObject* const* a, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  if (count != 5) return fail(FLCE_ERR_INVALID_ARG, "embedding: arguments");
  int device = -1;
  const at::Tensor *weight, *ids, *out, *word;
  int32_t* status;
  if (!tensor_of(a[0], "embedding: weight", false, &weight, &device) ||
      !tensor_of(a[1], "embedding: ids", false, &ids, &device) ||
      !tensor_of(a[3], "embedding: out", true, &out, &device) ||
      !status_of(a[4], "embedding: status", &device, &status, &word))
    return nullptr;
  const double scale = PyFloat_AsDouble(a[2]);
  if (PyErr_Occurred()) return nullptr;
  const int dtype = code_of(*weight), index_type = index_type_of(*ids);
  if (dtype == kUnknown) return fail(FLCE_ERR_UNSUPPORTED, "embedding: weight: its type");
  if (index_type == kUnknown) return fail(FLCE_ERR_UNSUPPORTED, "embedding: ids: int64 or int32 is wanted");
  if (weight->dim() != 2) return fail(FLCE_ERR_INVALID_ARG, "embedding: weight: a matrix is wanted");
  if (!ids->is_contiguous()) return fail(FLCE_ERR_UNSUPPORTED, "embedding: ids: not contiguous");
  Rows table, y_rows;
  if (!rows_of(*weight, "embedding: weight", &table)) return nullptr;
  c10::SmallVector<int64_t, 6> shape(ids->sizes().begin(), ids->sizes().end());
  shape.push_back(table.h);
  y_rows.ld = table.h;
  if (out != nullptr) {
    if (out->scalar_type() != weight->scalar_type() || out->sizes() != at::IntArrayRef(shape))
      return fail(FLCE_ERR_INVALID_ARG, "embedding: out: of another shape or type than the rows looked up");
    if (!rows_of(*out, "embedding: out", &y_rows)) return nullptr;
  }
  const at::Tensor y = out != nullptr ? *out : empty(shape, weight->scalar_type(), *weight);
  const flce_status_t st =
      embedding_fwd(dtype, data(weight), table.ld, data(ids), index_type, ids->numel(), table.n, table.h,
                    static_cast<float>(scale), y.data_ptr(), y_rows.ld, status, stream());
  if (st != FLCE_OK) return fail(st, "embedding_fwd");
  written({out, word});
  return THPVariable_Wrap(y);
  END_HANDLE_TH_ERRORS
}

// embedding_backward(grad_y, ids, vocabulary, scale, padding_index, grad_weight_out, accumulate, workspace, status)
//     -> grad_weight; vocabulary -1: that of grad_weight_out; padding_index -1: none
PyObject* embedding_backward(PyObject*, PyObject* const* a, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  if (count != 9) return fail(FLCE_ERR_INVALID_ARG, "embedding_backward: arguments");
  int device = -1;
  const at::Tensor *gy, *ids, *out, *ws, *word;
  int32_t* status;
  if (!tensor_of(a[0], "embedding_backward: grad_y", false, &gy, &device) ||
      !tensor_of(a[1], "embedding_backward: ids", false, &ids, &device) ||
      !tensor_of(a[5], "embedding_backward: grad_weight_out", true, &out, &device) ||
      !tensor_of(a[7], "embedding_backward: workspace", true, &ws, &device) ||
      !status_of(a[8], "embedding_backward: status", &device, &status, &word))
    return nullptr;
  int64_t v = PyLong_AsLongLong(a[2]);
  const double scale = PyFloat_AsDouble(a[3]);
  const int64_t padding = PyLong_AsLongLong(a[4]);
  if (PyErr_Occurred()) return nullptr;
  const bool accumulate = flag(a[6]);
  const int dtype = code_of(*gy), index_type = index_type_of(*ids);
  if (dtype == kUnknown) return fail(FLCE_ERR_UNSUPPORTED, "embedding_backward: grad_y: its type");
  if (index_type == kUnknown) return fail(FLCE_ERR_UNSUPPORTED, "embedding_backward: ids: int64 or int32 is wanted");
  if (!ids->is_contiguous()) return fail(FLCE_ERR_UNSUPPORTED, "embedding_backward: ids: not contiguous");
  Rows rows;
  if (!rows_of(*gy, "embedding_backward: grad_y", &rows)) return nullptr;
  if (gy->dim() != ids->dim() + 1 || gy->sizes().slice(0, ids->dim()) != ids->sizes())
    return fail(FLCE_ERR_INVALID_ARG, "embedding_backward: ids: one for each row of grad_y is wanted");
  if (out != nullptr) {
    if (out->scalar_type() != at::kFloat || out->dim() != 2 || out->size(1) != rows.h || !out->is_contiguous())
      return fail(FLCE_ERR_INVALID_ARG, "embedding_backward: grad_weight_out: a contiguous fp32 matrix of %lld columns "
                  "is wanted", (long long)rows.h);
    if (v >= 0 && v != out->size(0))
      return fail(FLCE_ERR_INVALID_ARG, "embedding_backward: grad_weight_out: another number of rows than vocabulary");
    v = out->size(0);
  } else if (v < 0 || accumulate) {
    return fail(FLCE_ERR_INVALID_ARG, "embedding_backward: %s", accumulate ? "accumulate adds to grad_weight_out"
                                                                           : "vocabulary is wanted");
  }
  const size_t size = embedding_workspace_size(rows.n, v, rows.h);
  if (size == 0) return fail(FLCE_ERR_INVALID_ARG, "embedding_backward: no rows, or more rows or columns than it takes");
  const at::Tensor grad = out != nullptr ? *out : empty({v, rows.h}, at::kFloat, *gy);
  const bool given = ws != nullptr && ws->is_contiguous() && ws->nbytes() >= size;
  const at::Tensor scratch =
      given ? *ws : empty({static_cast<int64_t>(size)}, at::kByte, *gy);
  const flce_status_t st = embedding_bwd(
      dtype, data(gy), rows.ld, data(ids), index_type, rows.n, v, rows.h, static_cast<float>(scale), padding,
      grad.data_ptr<float>(), accumulate, scratch.data_ptr(), scratch.nbytes(), status, stream());
  if (st != FLCE_OK) return fail(st, "embedding_bwd");
  written({out, word});
  return THPVariable_Wrap(grad);
  END_HANDLE_TH_ERRORS
}

}  // namespace flce_binding
