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
  __nv_bfloat16* inner;          // workspace [T * k][F]
  __nv_bfloat16* out;            // [T][H]
};

bsmma_status launch_moe_step(const StepArgs& a, int form, cudaStream_t stream);

}  // namespace bsmma
