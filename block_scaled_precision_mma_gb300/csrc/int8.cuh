// int8.cuh -- what the INT8 product kernels share: their arguments, the widening of INT8
// values to FP16 and the output store.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"

namespace bsmma {
namespace int8 {

constexpr int kMaxG = 1024;   // groups per launch

struct Int8Params {
  const int8_t* A;
  const float* sA;
  const int8_t* B;
  const float* sB;
  const __nv_bfloat16* bias;
  void* D;
  const int64_t* m_sizes;   // nullptr: one group of total_M rows
  int64_t total_M, N, K;
  int G;
  int* status;
};

// Four INT8 values as two FP16 pairs, exact: with u = x + 128 the FP16 bits 0x6400 | u are
// the number 1024 + u.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  const __half2 bias = __half2half2(__ushort_as_half(0x6480));   // 1024 + 128
  uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
  const __half2 x = __hsub2(*reinterpret_cast<__half2*>(&a), bias);
  const __half2 y = __hsub2(*reinterpret_cast<__half2*>(&b), bias);
  lo = *reinterpret_cast<const uint32_t*>(&x);
  hi = *reinterpret_cast<const uint32_t*>(&y);
}

template <bool F32>
__device__ __forceinline__ void store_out(void* D, int64_t i, float v) {
  if constexpr (F32)
    static_cast<float*>(D)[i] = v;
  else
    static_cast<__nv_bfloat16*>(D)[i] = __float2bfloat16_rn(v);
}

// SM-pair kernel (int8_pair.cu).
bsmma_status launch_pair(const Int8Params& p, bool f32, const DeviceInfo* dev, cudaStream_t stream);

}  // namespace int8
}  // namespace bsmma
