// distill_fwd_bwd's kernels for lists that a warp does not hold in its registers.
#include "row_loss.cuh"

namespace flce {

cudaError_t launch_distill_long(const RowLossParams& p, int dtype, cudaStream_t s) {
  return launch_rows<kDistillLong>(p, dtype, s);
}

}  // namespace flce
