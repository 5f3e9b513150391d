// branch_grad.cu -- the gradients of the residual branch: the host's choices, the launch that
// adds the workers' sums, and branch_enter's kernels (branch_grad.cuh has the kernel).
#include <algorithm>

#include "branch_grad.cuh"

namespace bsmma {
namespace branch {
namespace {

// Workers: runs of rows, as many as fill the GPU's 152 SMs with the blocks that fit one (by
// registers; at most two of them, 46479 rows of 1136 in BF16 took 181 us for 96).  A number of T and
// H alone, so that the sums' order, and with it every bit, is the same wherever the call runs.
int workers_of(int64_t T, int64_t H) {
  const int64_t vecs = H / 8;
  const int64_t warps = (vecs + 63) / 64;   // of a block; 16 with 128 registers a thread fit an SM
  const int64_t most = 152 * (vecs <= 128 ? 16 : std::max<int64_t>(16 / warps, 1));
  return static_cast<int>(std::min(T, most));
}

// The worker that has a row: the last one whose first row is not after it.
__device__ __forceinline__ int worker_of(int64_t T, int workers, int64_t row) {
  return static_cast<int>(((row + 1) * workers - 1) / T);
}
struct SumParams {
  const float *part_w, *part_b, *part_g;
  float *dweight, *dbias, *dgate;
  int64_t T, H, gate_rows;
  int workers, fixed;   // fixed: blockIdx.y below it are dweight and dbias
  bool by_worker;
};
// The workers' sums of 32 columns, added by LANES threads a column, each a run of workers.
template <int LANES>
__global__ void __launch_bounds__(32 * LANES) sum_kernel(const SumParams p) {
  __shared__ float part[LANES][32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  const float* from;
  float* to;
  int w0 = 0, w1 = p.workers;
  int64_t step = p.H, first = 0;   // worker w's sum is at from + w * step (the first's + first)
  int y = static_cast<int>(blockIdx.y);
  if (y < p.fixed) {
    const bool weight = y == 0 && p.part_w;
    from = weight ? p.part_w : p.part_b;
    to = weight ? p.dweight : p.dbias;
  } else {
    // a gate whose rows are several workers': gate y, or the one that worker y + 1's first row
    // continues where worker y + 1 is the first to continue it
    y -= p.fixed;
    int64_t g = y;
    if (p.by_worker) {
      const int64_t row = first_row(p.T, p.workers, y + 1);
      g = row / p.gate_rows;
      if (g * p.gate_rows == row || first_row(p.T, p.workers, y) > g * p.gate_rows) return;
    }
    const int64_t begin = g * p.gate_rows;
    const int64_t end = begin + p.gate_rows < p.T ? begin + p.gate_rows : p.T;
    w0 = worker_of(p.T, p.workers, begin);
    w1 = worker_of(p.T, p.workers, end - 1) + 1;
    if (w1 - w0 < 2) return;
    // its last gate is in a worker's second place, unless it begins with it
    first = first_row(p.T, p.workers, w0) < begin ? p.H : 0;
    from = p.part_g;
    to = p.dgate + g * p.H;
    step = 2 * p.H;
  }
  float s = 0.f;
  if (c < p.H) {
    const int n = w1 - w0, a = w0 + n * run / LANES, e = w0 + n * (run + 1) / LANES;
#pragma unroll 8
    for (int w = a; w < e; ++w) s += from[w * step + (w == w0 ? first : 0) + c];
  }
  part[run][lane] = s;
  __syncthreads();
  if (run == 0 && c < p.H) {
#pragma unroll
    for (int i = 1; i < LANES; ++i) s += part[i][lane];
    to[c] = s;
  }
}

template <bool DF, bool VF>
bsmma_status launch_enter_grad(const GradParams& p, cudaStream_t stream) {
  return p.part_b ? launch_grad_kernel<false, DF, VF, true, true, false>(p, stream)
                  : launch_grad_kernel<false, DF, VF, true, false, false>(p, stream);
}

}  // namespace

bsmma_status grad_enter(const GradParams& p, cudaStream_t stream) {
  if (!p.a.v_f32) return launch_enter_grad<false, false>(p, stream);
  return p.a.d_f32 ? launch_enter_grad<true, true>(p, stream) : launch_enter_grad<false, true>(p, stream);
}

}  // namespace branch

int64_t branch_grad_workspace_bytes(int64_t T, int64_t H) {
  return 4 * H * 4 * branch::workers_of(T, H);   // dweight, dbias and two gates a worker
}

bsmma_status launch_branch_grad(const BranchGradArgs& a, bool leave, void* workspace,
                                cudaStream_t stream) {
  using namespace branch;
  GradParams p = {};
  p.a = a;
  p.workers = workers_of(a.T, a.H);
  float* ws = static_cast<float*>(workspace);
  const int64_t plane = a.H * p.workers;
  if (a.dweight) p.part_w = ws;
  if (a.dbias) p.part_b = ws + plane;
  if (a.dgate && a.gate_rows > 1) p.part_g = ws + 2 * plane;
  bsmma_status st;
  if (!leave) st = grad_enter(p, stream);
  else if (!a.d_f32) st = grad_leave_bf16(p, stream);
  else st = a.v_f32 ? grad_leave_f32(p, stream) : grad_leave_mixed(p, stream);
  if (st != BSMMA_OK) return st;
  count_launches(1);
  SumParams s = {};
  s.part_w = p.part_w;
  s.part_b = p.part_b;
  s.part_g = p.part_g;
  s.dweight = a.dweight;
  s.dbias = a.dbias;
  s.dgate = a.dgate;
  s.T = a.T;
  s.H = a.H;
  s.gate_rows = a.gate_rows;
  s.workers = p.workers;
  s.fixed = (a.dweight != nullptr) + (a.dbias != nullptr);
  // with a gate for each row no gate is shared by two workers
  const int64_t gates = a.dgate && a.gate_rows > 1 ? (a.T + a.gate_rows - 1) / a.gate_rows : 0;
  const int shared = static_cast<int>(std::min<int64_t>(gates, p.workers - 1));
  s.by_worker = gates > p.workers - 1;
  if (s.fixed + shared == 0) return BSMMA_OK;
  // Eight threads a column where the blocks fill the GPU, else 32: few columns have as many workers as
  // many have (5499 rows of 128, both directions 58 and 43 us; 16383 of
  // 4096, 242 and 237)
  const dim3 grid(static_cast<unsigned>((a.H + 31) / 32), s.fixed + shared);
  const cudaError_t e = grid.x * grid.y < 4 * 152 ? launch_dependent(sum_kernel<32>, grid, dim3(1024), 0, stream, s)
                                                  : launch_dependent(sum_kernel<8>, grid, dim3(256), 0, stream, s);
  count_launches(1);
  return cuda_ok(e);
}

}  // namespace bsmma
