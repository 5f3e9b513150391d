// branch.h -- host-side interface of the residual branch's operators (branch.cu,
// branch_grad*.cu).
#pragma once
#include "internal.h"

namespace bsmma {

struct NormArgs {
  int kind = 0;                  // bsmma_norm
  float eps = 0.f;
  const float* weight = nullptr;
  const float* bias = nullptr;
};

// A row to write as the next product's input: BF16, FP32, INT8 or MX codes with their scales.
struct OperandArgs {
  int form = 0;                  // bsmma_operand
  void* out = nullptr;
  void* scales = nullptr;
};

// Keep the values whose 16 random bits are at least `threshold`, times `scale`.
struct DropArgs {
  uint32_t threshold = 0;        // 0: no dropout
  float scale = 1.f;
  const int64_t* rng = nullptr;  // {seed, offset} in device memory
};

struct EnterArgs {
  const void* x;
  bool x_f32;
  int64_t T, H;
  float inv_h;                   // 1 / H
  NormArgs norm;
  OperandArgs to;
};

struct LeaveArgs {
  const void* x;
  bool x_f32;
  const void* y;
  bool y_f32;
  int64_t T, H;
  float inv_h;
  NormArgs norm;
  const void* gate;              // of y's type, or nullptr
  int64_t gate_rows;
  float x_scale, y_scale;
  DropArgs drop;
  void* out;
  NormArgs next;                 // kind 0: none
  OperandArgs to;
};

// Both gradients: the gradient d of what the branch's step gave, the rows v that were normed.
struct BranchGradArgs {
  const void* d;
  bool d_f32;
  const void* v;
  bool v_f32;
  int64_t T, H;
  float inv_h;
  NormArgs norm;
  const void* dres;              // entering: added to dv (of v's type), or nullptr
  const void* gate;              // leaving: as forward
  int64_t gate_rows;
  float x_scale, y_scale;
  DropArgs drop;
  void* dv;
  void* dx;                      // leaving: x_scale * d, or nullptr
  float *dweight, *dbias, *dgate;
};

bsmma_status launch_branch_enter(const EnterArgs& a, cudaStream_t stream);
bsmma_status launch_branch_leave(const LeaveArgs& a, cudaStream_t stream);
bsmma_status launch_dropout(const void* x, bool f32, int64_t n, const DropArgs& drop, void* y,
                            cudaStream_t stream);
// Bytes of workspace of a gradient over T rows (sums of pieces of the rows).
int64_t branch_grad_workspace_bytes(int64_t T, int64_t H);
bsmma_status launch_branch_grad(const BranchGradArgs& a, bool leave, void* workspace,
                                cudaStream_t stream);

}  // namespace bsmma
