// moe_step.h -- host-side interface of the decoding step's expert layer.
#pragma once
#include <cuda_bf16.h>

#include "internal.h"

namespace bsmma {

struct StepArgs {
  const void* x;                 // [T][H] BF16
  int64_t T, H;
  const int32_t* ids;            // [T][k]
  const float* weights;
  int k, E;
  int64_t F;
  const void *w_in, *s_in, *w_out, *s_out;
  int act;
  __nv_bfloat16* out;            // [T][H]
  uint64_t limit_ns;             // of a wait on the device, and where one that ran out is latched
  int* status;
  // in the workspace
  float* x_power;                // [T], and the tokens in FP16 over it
  uint16_t* x16;                 // [T][H]
  float* inner_power;            // [T * k][F / 32, in fours], and the inner rows in FP16 over it, or
  uint16_t* inner;               // [T * k][F]             in BF16
};

int64_t step_workspace_bytes(int64_t T, int k, int64_t H, int64_t F);
bsmma_status launch_moe_step(StepArgs a, int form, void* workspace, cudaStream_t stream);

}  // namespace bsmma
