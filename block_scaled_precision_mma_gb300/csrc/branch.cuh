// branch.cuh -- device code shared by the residual branch's operators: rows in registers, their
// sums, and the dropout generator.
//
// A row of H values (H % 8 == 0) is held by TPR threads, a warp (TPR 32) or a block, V pieces
// of eight consecutive values each: piece i of thread `tid` is number tid + i * TPR of the row,
// so a warp reads and writes whole 512-byte (BF16) or 1-KB (FP32) runs.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "bsmma.h"
#include "ptx.cuh"

namespace bsmma {
namespace branch {

constexpr uint32_t kFull = 0xFFFFFFFFu;

// Eight consecutive values as they are stored.
template <bool F32>
struct Raw {
  uint4 r[F32 ? 2 : 1];
};

template <bool F32>
__device__ __forceinline__ Raw<F32> load_raw(const void* base, int64_t i) {
  Raw<F32> v;
  if constexpr (F32) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + i);
    v.r[0] = p[0];
    v.r[1] = p[1];
  } else {
    v.r[0] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + i);
  }
  return v;
}
template <bool F32>
__device__ __forceinline__ Raw<F32> zero_raw() {
  Raw<F32> v;
#pragma unroll
  for (int j = 0; j < (F32 ? 2 : 1); ++j) v.r[j] = make_uint4(0, 0, 0, 0);
  return v;
}
template <bool F32>
__device__ __forceinline__ void widen(const Raw<F32>& v, float (&f)[8]) {
  if constexpr (F32) {
    const uint32_t w[8] = {v.r[0].x, v.r[0].y, v.r[0].z, v.r[0].w,
                           v.r[1].x, v.r[1].y, v.r[1].z, v.r[1].w};
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(w[j]);
  } else {
    const uint32_t w[4] = {v.r[0].x, v.r[0].y, v.r[0].z, v.r[0].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = __uint_as_float(w[j] << 16);
      f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
}
template <bool F32>
__device__ __forceinline__ Raw<F32> narrow(const float (&f)[8]) {
  Raw<F32> v;
  if constexpr (F32) {
    v.r[0] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                        __float_as_uint(f[3]));
    v.r[1] = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]),
                        __float_as_uint(f[7]));
  } else {
    v.r[0] = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                        pack_bf16x2(f[6], f[7]));
  }
  return v;
}
template <bool F32>
__device__ __forceinline__ void store_raw(void* base, int64_t i, const Raw<F32>& v) {
  if constexpr (F32) {
    uint4* p = reinterpret_cast<uint4*>(static_cast<float*>(base) + i);
    p[0] = v.r[0];
    p[1] = v.r[1];
  } else {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + i) = v.r[0];
  }
}

// Eight FP32 parameters of columns c .. c + 7.  (Plain loads here and below: the kernels may start
// before the one ahead of them has finished, and a read-only load could move above that wait.)
__device__ __forceinline__ void load_columns(const float* p, int c, float (&f)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p + c);
  const float4 b = *reinterpret_cast<const float4*>(p + c + 4);
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
  f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

// The sums of N values over the row's threads, in all of them and in an order that does not
// change.  `part` (N * TPR / 32 floats, unused for a warp) is read until the next barrier.
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* part) {
#pragma unroll
  for (int o = 16; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(kFull, v[i], o);
  if constexpr (TPR > 32) {
    constexpr int kWarps = TPR / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) part[i * kWarps + warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = part[i * kWarps + (lane & (kWarps - 1))];
#pragma unroll
    for (int o = kWarps / 2; o; o >>= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(kFull, v[i], o);
  }
}
template <int TPR>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* part) {
  v = __reduce_max_sync(kFull, v);
  if constexpr (TPR > 32) {
    constexpr int kWarps = TPR / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) part[warp] = v;
    __syncthreads();
    v = __reduce_max_sync(kFull, part[lane & (kWarps - 1)]);
  }
  return v;
}

// Philox4x32-10 (J. Salmon, M. Moraes, R. Dror, D. Shaw, "Parallel random numbers: as easy as
// 1, 2, 3", SC 2011), counter (low and high word of `block`, low and high word of the offset),
// key the seed's words: 128 bits for the eight values of number 8 * block and up, 16 bits each,
// low half of a word first.  Bit j of the result: value j is kept, its bits at least
// `threshold`.  16 bits a value make one call serve eight values: about 9 integer instructions
// a value, which stay below the time its bytes take (dropout_kernel).
struct Philox {
  uint32_t k0, k1, c2, c3;
};
__device__ __forceinline__ Philox philox_of(const int64_t* rng) {
  const uint64_t seed = static_cast<uint64_t>(rng[0]), offset = static_cast<uint64_t>(rng[1]);
  return Philox{static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32),
                static_cast<uint32_t>(offset), static_cast<uint32_t>(offset >> 32)};
}
__device__ __forceinline__ uint32_t kept8(const Philox& g, uint64_t block, uint32_t threshold) {
  uint32_t a = static_cast<uint32_t>(block), b = static_cast<uint32_t>(block >> 32);
  uint32_t c = g.c2, d = g.c3, k0 = g.k0, k1 = g.k1;
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t u = static_cast<uint64_t>(a) * 0xD2511F53u, v = static_cast<uint64_t>(c) * 0xCD9E8D57u;
    a = static_cast<uint32_t>(v >> 32) ^ b ^ k0;
    b = static_cast<uint32_t>(v);
    c = static_cast<uint32_t>(u >> 32) ^ d ^ k1;
    d = static_cast<uint32_t>(u);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  const uint32_t w[4] = {a, b, c, d};
  uint32_t mask = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if ((w[j] & 0xFFFFu) >= threshold) mask |= 1u << (2 * j);
    if ((w[j] >> 16) >= threshold) mask |= 2u << (2 * j);
  }
  return mask;
}

}  // namespace branch
}  // namespace bsmma
