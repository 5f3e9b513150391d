// branch.cuh -- device code shared by the residual branch's operators: rows in registers, their
// sums, and the dropout generator.
//
// A row of H values (H % 8 == 0) is held by a warp or by all warps of a block (as many as
// make V pieces of eight values a thread: no lane idles at 7168 values).  A warp has 32 * V pieces in a
// row, its lane l those at l + 32 i, so that each access covers 512 bytes (BF16) or 1 KB (FP32) and
// a thread's pieces are constant distances apart.  Values are handled in pairs, by the
// instructions that do two FP32 operations at once: these kernels are bound by DRAM only while
// they issue few enough instructions a value (with the pieces a number of threads apart that is only
// known at run time, the addresses made a step with dropout, gate and two norms 267 us for 203).
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
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
// Eight values as four pairs.
struct Vals {
  float2 v[4];
};
__device__ __forceinline__ float2 both(float f) { return make_float2(f, f); }
// a * b and a + b as the packed FMA (the same results: b + -0 is b).
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __ffma2_rn(a, b, make_float2(-0.f, -0.f)); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __ffma2_rn(a, make_float2(1.f, 1.f), b); }
template <bool F32>
__device__ __forceinline__ Vals widen(const Raw<F32>& r) {
  Vals o;
  if constexpr (F32) {
    const uint32_t w[8] = {r.r[0].x, r.r[0].y, r.r[0].z, r.r[0].w, r.r[1].x, r.r[1].y, r.r[1].z, r.r[1].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) o.v[j] = make_float2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
  } else {
    const uint32_t w[4] = {r.r[0].x, r.r[0].y, r.r[0].z, r.r[0].w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o.v[j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
  }
  return o;
}
template <bool F32>
__device__ __forceinline__ Raw<F32> narrow(const Vals& f) {
  Raw<F32> r;
  if constexpr (F32) {
    r.r[0] = make_uint4(__float_as_uint(f.v[0].x), __float_as_uint(f.v[0].y), __float_as_uint(f.v[1].x),
                        __float_as_uint(f.v[1].y));
    r.r[1] = make_uint4(__float_as_uint(f.v[2].x), __float_as_uint(f.v[2].y), __float_as_uint(f.v[3].x),
                        __float_as_uint(f.v[3].y));
  } else {
    r.r[0] = make_uint4(pack_bf16x2(f.v[0].x, f.v[0].y), pack_bf16x2(f.v[1].x, f.v[1].y),
                        pack_bf16x2(f.v[2].x, f.v[2].y), pack_bf16x2(f.v[3].x, f.v[3].y));
  }
  return r;
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
__device__ __forceinline__ Vals load_columns(const float* p, int c) {
  const float4 a = *reinterpret_cast<const float4*>(p + c);
  const float4 b = *reinterpret_cast<const float4*>(p + c + 4);
  return Vals{{{a.x, a.y}, {a.z, a.w}, {b.x, b.y}, {b.z, b.w}}};
}

// Where a thread's V pieces are: piece i is number at(i) of the row's `vecs`.
template <bool WARP, int V>
struct Place {
  int base, vecs;
  __device__ __forceinline__ explicit Place(int64_t H)
      : base((WARP ? 0 : static_cast<int>(threadIdx.x >> 5) * (32 * V)) + static_cast<int>(threadIdx.x & 31)),
        vecs(static_cast<int>(H / 8)) {}
  __device__ __forceinline__ int at(int i) const { return base + 32 * i; }
  __device__ __forceinline__ bool in(int i) const { return at(i) < vecs; }
};

// 1 / sqrt(v) to the last place or so: the fast root and one step of Newton's, which would make
// infinity times 0 of an infinite v (0).
__device__ __forceinline__ float inv_sqrt(float v) {
  const float r = rsqrtf(v);
  return v <= FLT_MAX ? r * fmaf(-0.5f * (v * r), r, 1.5f) : r;
}

// The sums of N values over the row's threads, in all of them and in an order that does not
// change.  WARP: the row is the warp's.  Else it is the block's, of at most 32 warps; `part`
// (32 * N floats) is read until the next barrier.
template <bool WARP, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* part) {
#pragma unroll
  for (int o = 16; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(kFull, v[i], o);
  if constexpr (!WARP) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) part[32 * i + warp] = v[i];
    __syncthreads();
    const bool in = lane < static_cast<int>(blockDim.x >> 5);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = in ? part[32 * i + lane] : 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(kFull, v[i], o);
  }
}
// Two sums at once, the lower half-warp on the first and the upper on the second: half the
// shuffles.
template <bool WARP>
__device__ __forceinline__ float2 row_sums2(float2 v, float* part) {
  const int lane = threadIdx.x & 31;
  const bool upper = lane & 16;
  float s = (upper ? v.y : v.x) + __shfl_xor_sync(kFull, upper ? v.x : v.y, 16);
#pragma unroll
  for (int o = 8; o; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
  if constexpr (!WARP) {
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    if ((lane & 15) == 0) part[(lane << 1) + warp] = s;   // [sum][32 warps]
    __syncthreads();
    const float* from = part + ((lane & 16) << 1) + (lane & 15);
    s = (lane & 15) < warps ? from[0] : 0.f;
    if ((lane & 15) + 16 < warps) s += from[16];
#pragma unroll
    for (int o = 8; o; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
  }
  return make_float2(__shfl_sync(kFull, s, 0), __shfl_sync(kFull, s, 16));
}
template <bool WARP>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* part) {
  v = __reduce_max_sync(kFull, v);
  if constexpr (!WARP) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) part[warp] = v;
    __syncthreads();
    v = __reduce_max_sync(kFull, lane < static_cast<int>(blockDim.x >> 5) ? part[lane] : 0u);
  }
  return v;
}

// Philox4x32-10 (J. Salmon, M. Moraes, R. Dror, D. Shaw, "Parallel random numbers: as easy as
// 1, 2, 3", SC 2011), counter (low and high word of `block`, low and high word of the offset),
// key the seed's words: 128 bits for the eight values of number 8 * block and up, 16 bits each,
// low half of a word first; a value is kept where its bits are at least the threshold.  16 bits a
// value make one call serve eight of them.
struct Philox {
  uint32_t k0, k1, c2, c3;
};
__device__ __forceinline__ Philox philox_of(const int64_t* rng) {
  const uint64_t seed = static_cast<uint64_t>(rng[0]), offset = static_cast<uint64_t>(rng[1]);
  // the same in every lane; said by a reduction, whose result needs no vector register, so that
  // the ten rounds' keys are scalar work (every lane of the warp is here)
  return Philox{__reduce_or_sync(kFull, static_cast<uint32_t>(seed)),
                __reduce_or_sync(kFull, static_cast<uint32_t>(seed >> 32)), static_cast<uint32_t>(offset),
                static_cast<uint32_t>(offset >> 32)};
}
__device__ __forceinline__ uint4 philox(const Philox& g, uint64_t block) {
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
  return make_uint4(a, b, c, d);
}
// Values whose bits (of `words`) are below the threshold, given in the upper half of `limit`,
// become 0.
__device__ __forceinline__ void drop(Vals& f, const uint4& words, uint32_t limit) {
  const uint32_t w[4] = {words.x, words.y, words.z, words.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f.v[j].x = w[j] << 16 >= limit ? f.v[j].x : 0.f;
    f.v[j].y = w[j] >= limit ? f.v[j].y : 0.f;
  }
}

}  // namespace branch
}  // namespace bsmma
