// branch_grad_f32.cu -- the gradient of branch_leave for an FP32 stream and branch.
#include "branch_grad.cuh"

namespace bsmma {
namespace branch {
bsmma_status grad_leave_f32(const GradParams& p, cudaStream_t stream) {
  return launch_leave_grad<true, true>(p, stream);
}
}  // namespace branch
}  // namespace bsmma
