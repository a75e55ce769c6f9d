// The clipped policy loss with a KL term on the tokens that a policy sampled, and its
// gradient on their logits (row_loss.cuh).
#include "row_loss.cuh"

using namespace flce;

extern "C" {

size_t row_loss_workspace_size(int64_t N) { return N < 0 || N >= (int64_t(1) << 31) ? 0 : kRowLossFixed; }

flce_status_t policy_fwd_bwd(const void* logits, int dtype, int64_t ld, void* grad_logits, int64_t ld_grad,
                             const int64_t* target, const float* advantage, const float* old_logp,
                             const float* ref_logp, const float* row_weight, int64_t N, int64_t V,
                             const flce_policy_t* numbers, int64_t ignore_index, int reduction, float grad_scale,
                             const float* grad_out_none, float* loss, float* logp, void* workspace,
                             size_t workspace_bytes, int32_t* status_dev, flce_stream_t stream) {
  const flce_status_t st = check_rows(logits, dtype, ld, grad_logits, ld_grad, N, V, N, reduction, grad_out_none,
                                      loss, workspace, workspace_bytes, kRowLossFixed, status_dev);
  if (st != FLCE_OK) return st;
  if (numbers == nullptr || (N > 0 && (target == nullptr || advantage == nullptr))) return FLCE_ERR_INVALID_ARG;
  if (!(numbers->clip_low >= 0.f) || !(numbers->clip_high >= 0.f) || !temperature_ok(numbers->temperature) ||
      !(numbers->kl_weight == 0.f || positive(numbers->kl_weight)))
    return FLCE_ERR_INVALID_ARG;
  if (numbers->kl_weight != 0.f && ref_logp == nullptr && N > 0) return FLCE_ERR_INVALID_ARG;
  if (!aligned_to(target, 8) || !aligned_to(advantage, 4) || !aligned_to(old_logp, 4) || !aligned_to(ref_logp, 4) ||
      !aligned_to(row_weight, 4) || !aligned_to(logp, 4))
    return FLCE_ERR_MISALIGNED;
  RowLossParams p = row_params(logits, ld, grad_logits, ld_grad, N, V, reduction, grad_scale, grad_out_none, loss,
                               numbers->temperature);
  p.ignore_index = ignore_index, p.target = target;
  p.advantage = advantage, p.old_logp = old_logp, p.ref_logp = ref_logp, p.row_weight = row_weight;
  p.ratio_low = 1.f - numbers->clip_low, p.ratio_high = 1.f + numbers->clip_high, p.kl_weight = numbers->kl_weight;
  p.logp = logp;
  use_workspace(&p, workspace, status_dev);
  return launch_rows<kPolicy>(p, dtype, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? FLCE_OK
                                                                                                : FLCE_ERR_CUDA;
}

}  // extern "C"
