// The distance from a teacher of which each row has the largest logits, and its gradient
// on the student's logits (row_loss.cuh).
#include "row_loss.cuh"

namespace flce {
cudaError_t launch_distill_long(const RowLossParams& p, int dtype, cudaStream_t s);  // distill_long.cu
}

using namespace flce;

extern "C" {

flce_status_t distill_fwd_bwd(const void* logits, int dtype, int64_t ld, void* grad_logits, int64_t ld_grad,
                              const void* ids, int index_type, const void* values, int value_dtype, int64_t top,
                              const float* row_weight, int64_t N, int64_t V, float temperature, int reduction,
                              float grad_scale, const float* grad_out_none, float* loss, void* workspace,
                              size_t workspace_bytes, int32_t* status_dev, flce_stream_t stream) {
  static_assert(FLCE_DISTILL_MAX_TOP == kMaxTeacher, "the header states the limit");
  if (!float_dtype(value_dtype)) return FLCE_ERR_UNSUPPORTED;
  const flce_status_t st = check_rows(logits, dtype, ld, grad_logits, ld_grad, N, V, N, reduction, grad_out_none,
                                      loss, workspace, workspace_bytes, kRowLossFixed, status_dev);
  if (st != FLCE_OK) return st;
  if (index_type != FLCE_INDEX_INT64 && index_type != FLCE_INDEX_INT32) return FLCE_ERR_INVALID_ARG;
  if (top < 1 || !temperature_ok(temperature) || (N > 0 && (ids == nullptr || values == nullptr)))
    return FLCE_ERR_INVALID_ARG;
  if (top > kMaxTeacher) return FLCE_ERR_UNSUPPORTED;
  if (!aligned_to(ids, index_type == FLCE_INDEX_INT64 ? 8 : 4) || !aligned_to(values, elem_size(value_dtype)) ||
      !aligned_to(row_weight, 4))
    return FLCE_ERR_MISALIGNED;
  RowLossParams p = row_params(logits, ld, grad_logits, ld_grad, N, V, reduction, grad_scale, grad_out_none, loss,
                               temperature);
  p.ids = ids, p.ids32 = index_type == FLCE_INDEX_INT32, p.values = values, p.value_dtype = value_dtype;
  p.K = static_cast<int>(top);
  p.row_weight = row_weight;
  use_workspace(&p, workspace, status_dev);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = top <= 32 * kListAhead ? launch_rows<kDistill>(p, dtype, s) : launch_distill_long(p, dtype, s);
  return e == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}

}  // extern "C"
