// int8.cuh -- what the INT8 product kernels share: their arguments, the widening of INT8
// values to FP16, the output store and the table of the groups' rows.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

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

// sum * sa * sb + bias.  With the product of the scales first an element costs one multiplication
// and one fused step, but a subnormal product has lost bits that the result may have, and an
// infinite one makes a sum of 0 NaN.  There the smaller scale meets the sum first: a sum is an
// integer, so a subnormal product with it is exact, and one that overflows does so beside a
// scale at least as large, where the result does too.
__device__ __forceinline__ bool normal_product(float lo, float hi, float s) {
  return lo * s >= FLT_MIN && hi * s <= FLT_MAX;
}
__device__ __forceinline__ float scale_sum(float sum, float sa, float sb, float bias) {
  const float p = sa * sb;
  if (normal_product(fabsf(p), fabsf(p), 1.f)) return fmaf(sum, p, bias);
  const bool a_first = fabsf(sa) < fabsf(sb);
  return fmaf(sum * (a_first ? sa : sb), a_first ? sb : sa, bias);
}

template <bool F32>
__device__ __forceinline__ void store_out(void* D, int64_t i, float v) {
  if constexpr (F32)
    static_cast<float*>(D)[i] = v;
  else
    static_cast<__nv_bfloat16*>(D)[i] = __float2bfloat16_rn(v);
}

// Where each group's rows and blocks of rows begin, for blocks of THREADS threads.
template <int THREADS>
struct GroupTable {
  int32_t start[kMaxG + 1];    // first row of each group
  int32_t tile0[kMaxG + 1];    // its first row block
  int32_t warp_sum[2][THREADS / 32];
  int bad;
};

// Fills the table (every thread of the block); blocks of tn rows.  Sizes that are negative or
// sum to more than total_M set `bad` and latch the status once.
template <int THREADS>
__device__ __forceinline__ void build_table(GroupTable<THREADS>& t, const Int8Params& p, int tn) {
  constexpr uint32_t kFull = 0xFFFFFFFFu, kThreads = THREADS;
  const int G = p.G, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (!p.m_sizes) {
    if (tid == 0) {
      t.start[0] = 0;
      t.tile0[0] = 0;
      t.start[1] = static_cast<int32_t>(p.total_M);
      t.tile0[1] = static_cast<int32_t>((p.total_M + tn - 1) / tn);
      t.bad = 0;
    }
    __syncthreads();
    return;
  }
  constexpr int kPer = kMaxG / kThreads;
  int64_t rows = 0;
  int32_t m[kPer], blocks = 0;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int g = tid * kPer + i;
    const int64_t v = g < G ? p.m_sizes[g] : 0;
    const bool out = v < 0 || v > p.total_M;
    bad |= out;
    m[i] = out ? 0 : static_cast<int32_t>(v);
    rows += m[i];
    blocks += (m[i] + tn - 1) / tn;
  }
  // sums of up to 1024 sizes below 2^31 each can pass 32 bits: checked in 64 first
  int64_t all = rows;
#pragma unroll
  for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(kFull, all, o);
  bad |= all > p.total_M;
  bad = __syncthreads_or(bad);
  int32_t ir = static_cast<int32_t>(bad ? 0 : rows), ib = bad ? 0 : blocks;
  const int32_t r_own = ir, b_own = ib;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t a = __shfl_up_sync(kFull, ir, o), b = __shfl_up_sync(kFull, ib, o);
    if (lane >= o) {
      ir += a;
      ib += b;
    }
  }
  if (lane == 31) {
    t.warp_sum[0][warp] = ir;
    t.warp_sum[1][warp] = ib;
  }
  __syncthreads();
  int32_t r0 = ir - r_own, b0 = ib - b_own;
  int64_t total = 0;
  for (int w = 0; w < static_cast<int>(kThreads) / 32; ++w) {
    if (w < warp) {
      r0 += t.warp_sum[0][w];
      b0 += t.warp_sum[1][w];
    }
    total += t.warp_sum[0][w];
  }
  bad |= total > p.total_M;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int g = tid * kPer + i;
    if (g <= G) {
      t.start[g] = r0;
      t.tile0[g] = b0;
    }
    r0 += m[i];
    b0 += (m[i] + tn - 1) / tn;
    if (g == G - 1) {
      t.start[G] = r0;
      t.tile0[G] = b0;
    }
  }
  if (tid == 0) {
    t.bad = bad;
    if (bad && blockIdx.x == 0) report_status(p.status, kDevBadMSizes);
  }
  __syncthreads();
}

// The group of row block mt: the last one whose first block is not after it.
template <int THREADS>
__device__ __forceinline__ int find_group(const GroupTable<THREADS>& t, int G, int mt) {
  int lo = 0, hi = G - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.tile0[mid] <= mt) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Blocks of `tn` rows that a group's rows make on the host's estimate: of one group exactly, of
// several on average over groups 0.6 to 1.4 times as large as their mean.
inline double blocks_per_group(const Int8Params& a, double rows, int tn) {
  double blocks = std::ceil(rows / tn);
  if (a.G > 1) {
    blocks = 0;
    for (const double f : {0.6, 0.8, 1.0, 1.2, 1.4}) blocks += std::ceil(f * rows / tn) / 5;
  }
  return blocks < 1 ? 1 : blocks;
}
inline double groups_with_rows(const Int8Params& a) {
  return a.total_M < a.G ? static_cast<double>(a.total_M) : a.G;
}

// SM-pair kernel (int8_pair.cu), and the SM cycles it is expected to take.
double pair_cycles(const Int8Params& p, const DeviceInfo* dev);
bsmma_status launch_pair(const Int8Params& p, bool f32, const DeviceInfo* dev, cudaStream_t stream);

}  // namespace int8
}  // namespace bsmma
