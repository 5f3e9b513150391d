// branch_grad_mixed.cu -- the gradient of branch_leave for an FP32 stream and a BF16 branch.
#include "branch_grad.cuh"

namespace bsmma {
namespace branch {
bsmma_status grad_leave_mixed(const GradParams& p, cudaStream_t stream) {
  return launch_leave_grad<true, false>(p, stream);
}
}  // namespace branch
}  // namespace bsmma
