// branch_grad_bf16.cu -- the gradient of branch_leave for a BF16 stream and branch.
#include "branch_grad.cuh"

namespace bsmma {
namespace branch {
bsmma_status grad_leave_bf16(const GradParams& p, cudaStream_t stream) {
  return launch_leave_grad<false, false>(p, stream);
}
}  // namespace branch
}  // namespace bsmma
