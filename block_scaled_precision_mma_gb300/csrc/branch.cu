// branch.cu -- the residual branch forward: the norm before a block (branch_enter), the step
// after it (branch_leave) and dropout by itself.
//
// All of them are bound by DRAM, so every row is read once, kept in registers through its
// reductions, and written once.  The norm of the next block is taken from the row while it is
// there, and a product's operand (INT8 rows, MX codes with their scales) is made from the FP32
// values of the norm, so that neither the normed row nor a second reading of the stream costs
// any bytes.
#include <algorithm>

#include "branch.cuh"
#include "branch.h"

namespace bsmma {
namespace {
using namespace branch;

// ------------------------------------------------------------------------- norms
// f (zeros in pieces past the row) -> n(f) * weight + bias.  The variance of a layer norm is
// summed around the mean, in a second pass over the registers: a row far from zero keeps its
// digits.
template <int TPR, int V>
__device__ __forceinline__ void norm_row(float (&f)[V][8], const NormArgs& a, int tid, int vecs,
                                         float inv_h, float* part) {
  float s[1] = {0.f};
  if (a.kind == BSMMA_NORM_LAYER) {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) s[0] += f[i][j];
    row_sums<TPR>(s, part);
    const float mean = s[0] * inv_h;
    s[0] = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (tid + i * TPR < vecs)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          f[i][j] -= mean;
          s[0] = fmaf(f[i][j], f[i][j], s[0]);
        }
    row_sums<TPR>(s, part + 32);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) s[0] = fmaf(f[i][j], f[i][j], s[0]);
    row_sums<TPR>(s, part);
  }
  const float r = __frsqrt_rn(fmaf(s[0], inv_h, a.eps));
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = tid + i * TPR;
    if (v >= vecs) continue;
    float w[8], b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = 1.f, b[j] = 0.f;
    if (a.weight) load_columns(a.weight, 8 * v, w);
    if (a.bias) load_columns(a.bias, 8 * v, b);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[i][j] = fmaf(f[i][j] * r, w[j], b[j]);
  }
}

// ------------------------------------------------------------------------- operands
// The same rules as int8_quantize's and mx_quantize's (rowwise), on the FP32 values.
template <int FMT>
__device__ __forceinline__ uint32_t fp8x2(float lo, float hi) {
  uint16_t r;
  if constexpr (FMT == BSMMA_OPERAND_E4M3)
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t fp4x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u32.u8 %0, t;\n\t}"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r & 0xFFu;
}

template <int FMT, int TPR, int V>
__device__ __forceinline__ void store_mx(const float (&f)[V][8], const OperandArgs& to, int64_t t,
                                         int64_t H, int tid, int vecs) {
  constexpr int kEmax = FMT == BSMMA_OPERAND_E4M3 ? 8 : FMT == BSMMA_OPERAND_E5M2 ? 15 : 2;
  uint8_t* codes = static_cast<uint8_t*>(to.out) + t * (FMT == BSMMA_OPERAND_E2M1 ? H / 2 : H);
  uint8_t* scales = static_cast<uint8_t*>(to.scales) + t * (H / 32);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = tid + i * TPR;
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(f[i][j]));
    // four neighbouring lanes hold a block of 32 (vecs % 4 == 0: all of them in the row or none)
    amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
    if (v >= vecs) continue;
    int e = 0;
    if (amax > 0.f) {
      const uint32_t bits = __float_as_uint(amax);
      const int ef = static_cast<int>(bits >> 23);
      e = (ef ? ef - 127 : 31 - __clz(static_cast<int>(bits)) - 149) - kEmax;
      e = max(-127, min(127, e));
    }
    // 2^-e; 2^-127 is subnormal
    const float inv = e < 127 ? __uint_as_float(static_cast<uint32_t>(127 - e) << 23)
                              : __uint_as_float(0x00400000u);
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = __fmul_rn(f[i][j], inv);
    if constexpr (FMT == BSMMA_OPERAND_E2M1) {
      *reinterpret_cast<uint32_t*>(codes + 4 * static_cast<int64_t>(v)) =
          fp4x2(y[0], y[1]) | fp4x2(y[2], y[3]) << 8 | fp4x2(y[4], y[5]) << 16 | fp4x2(y[6], y[7]) << 24;
    } else {
      *reinterpret_cast<uint2*>(codes + 8 * static_cast<int64_t>(v)) =
          make_uint2(fp8x2<FMT>(y[0], y[1]) | fp8x2<FMT>(y[2], y[3]) << 16,
                     fp8x2<FMT>(y[4], y[5]) | fp8x2<FMT>(y[6], y[7]) << 16);
    }
    if ((v & 3) == 0) scales[v >> 2] = static_cast<uint8_t>(e + 127);
  }
}

template <int TPR, int V>
__device__ __forceinline__ void store_int8(const float (&f)[V][8], const OperandArgs& to, int64_t t,
                                           int64_t H, int tid, int vecs, float* part) {
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = max(amax, __float_as_uint(f[i][j]) & 0x7FFFFFFFu);
  amax = row_max<TPR>(amax, reinterpret_cast<uint32_t*>(part));
  float s = __fmul_rn(__uint_as_float(amax), 1.f / 127.f);
  if (s == 0.f) s = 1.f;
  if (tid == 0) static_cast<float*>(to.scales)[t] = s;
  // the quotient rounded once: two fused corrections on the reciprocal (as int8_quantize takes
  // it), where nothing of them leaves FP32's range
  const bool normal = s >= 0x1p-88f && s <= 0x1p100f;
  const float inv = normal ? __fdiv_rn(1.f, s) : 0.f;
  int8_t* codes = static_cast<int8_t*>(to.out) + t * H;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = tid + i * TPR;
    if (v >= vecs) continue;
    uint32_t c[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = f[i][j];
      float q = x * inv;
      q = fmaf(fmaf(-s, q, x), inv, q);
      q = fmaf(fmaf(-s, q, x), inv, q);
      if (!normal) q = __fdiv_rn(x, s);
      const int n = max(-127, min(127, __float2int_rn(q)));
      c[j >> 2] |= (static_cast<uint32_t>(n) & 0xFFu) << (8 * (j & 3));
    }
    *reinterpret_cast<uint2*>(codes + 8 * static_cast<int64_t>(v)) = make_uint2(c[0], c[1]);
  }
}

template <int TPR, int V>
__device__ __forceinline__ void store_operand(const float (&f)[V][8], const OperandArgs& to, int64_t t,
                                              int64_t H, int tid, int vecs, float* part) {
  switch (to.form) {
    case BSMMA_OPERAND_BF16:
    case BSMMA_OPERAND_F32:
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (tid + i * TPR < vecs) {
          const int64_t at = t * H + 8 * (tid + i * TPR);
          if (to.form == BSMMA_OPERAND_BF16) store_raw<false>(to.out, at, narrow<false>(f[i]));
          else store_raw<true>(to.out, at, narrow<true>(f[i]));
        }
      break;
    case BSMMA_OPERAND_INT8: store_int8<TPR, V>(f, to, t, H, tid, vecs, part); break;
    case BSMMA_OPERAND_E4M3: store_mx<BSMMA_OPERAND_E4M3, TPR, V>(f, to, t, H, tid, vecs); break;
    case BSMMA_OPERAND_E5M2: store_mx<BSMMA_OPERAND_E5M2, TPR, V>(f, to, t, H, tid, vecs); break;
    default: store_mx<BSMMA_OPERAND_E2M1, TPR, V>(f, to, t, H, tid, vecs); break;
  }
}

// ------------------------------------------------------------------------- kernels
template <int TPR>
constexpr int kBlock = TPR < 128 ? 128 : TPR;

template <bool F32, int TPR, int V>
__global__ void __launch_bounds__(kBlock<TPR>) enter_kernel(const EnterArgs p) {
  __shared__ float part[3 * 32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int tid = threadIdx.x % TPR, vecs = static_cast<int>(p.H / 8);
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kBlock<TPR> / TPR) + threadIdx.x / TPR;
  if (t >= p.T) return;   // (whole warps, and no barrier where a row is a warp's)
  Raw<F32> raw[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = tid + i * TPR;
    raw[i] = v < vecs ? load_raw<F32>(p.x, t * p.H + 8 * v) : zero_raw<F32>();
  }
  float f[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) widen<F32>(raw[i], f[i]);
  norm_row<TPR, V>(f, p.norm, tid, vecs, 1.f / static_cast<float>(p.H), part);
  store_operand<TPR, V>(f, p.to, t, p.H, tid, vecs, part + 64);
}

template <bool XF, bool YF, int TPR, int V>
__global__ void __launch_bounds__(kBlock<TPR>) leave_kernel(const LeaveArgs p) {
  __shared__ float part[5 * 32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int tid = threadIdx.x % TPR, vecs = static_cast<int>(p.H / 8);
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kBlock<TPR> / TPR) + threadIdx.x / TPR;
  if (t >= p.T) return;
  const float inv_h = 1.f / static_cast<float>(p.H);
  Raw<YF> ry[V];
  Raw<XF> rx[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = tid + i * TPR;
    ry[i] = v < vecs ? load_raw<YF>(p.y, t * p.H + 8 * v) : zero_raw<YF>();
    rx[i] = v < vecs ? load_raw<XF>(p.x, t * p.H + 8 * v) : zero_raw<XF>();
  }
  float f[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) widen<YF>(ry[i], f[i]);
  if (p.norm.kind != BSMMA_NORM_NONE) norm_row<TPR, V>(f, p.norm, tid, vecs, inv_h, part);
  Philox gen = {};
  if (p.drop.threshold) gen = philox_of(p.drop.rng);
  const int64_t gate_row =
      p.gate ? static_cast<int64_t>(static_cast<uint32_t>(t) / static_cast<uint32_t>(p.gate_rows)) * p.H : 0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = tid + i * TPR;
    if (v >= vecs) continue;
    if (p.drop.threshold) {
      const uint32_t keep = kept8(gen, static_cast<uint64_t>(t) * vecs + v, p.drop.threshold);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[i][j] = keep >> j & 1u ? f[i][j] * p.drop.scale : 0.f;
    }
    if (p.gate) {
      float g[8];
      widen<YF>(load_raw<YF>(p.gate, gate_row + 8 * v), g);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[i][j] *= g[j];
    }
    float x[8];
    widen<XF>(rx[i], x);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[i][j] = fmaf(p.y_scale, f[i][j], p.x_scale * x[j]);
    const Raw<XF> o = narrow<XF>(f[i]);
    store_raw<XF>(p.out, t * p.H + 8 * v, o);
    widen<XF>(o, f[i]);   // the next norm is of what is stored
  }
  if (p.next.kind == BSMMA_NORM_NONE) return;
  norm_row<TPR, V>(f, p.next, tid, vecs, inv_h, part + 64);
  store_operand<TPR, V>(f, p.to, t, p.H, tid, vecs, part + 128);
}

// Eight values a piece (the last one may be short), kPieces in flight a thread.
constexpr int kDropPieces = 4;
template <bool F32>
__global__ void __launch_bounds__(256) dropout_kernel(const void* x, int64_t n, const DropArgs drop,
                                                      void* y) {
  grid_dependency_wait();
  grid_launch_dependents();
  Philox gen = {};
  if (drop.threshold) gen = philox_of(drop.rng);
  const int64_t whole = n / 8;
  const int64_t base = static_cast<int64_t>(blockIdx.x) * (256 * kDropPieces) + threadIdx.x;
  Raw<F32> raw[kDropPieces];
#pragma unroll
  for (int i = 0; i < kDropPieces; ++i)
    if (base + 256 * i < whole) raw[i] = load_raw<F32>(x, 8 * (base + 256 * i));
#pragma unroll
  for (int i = 0; i < kDropPieces; ++i) {
    const int64_t v = base + 256 * i;
    if (v > whole || 8 * v >= n) continue;
    const uint32_t keep = drop.threshold ? kept8(gen, static_cast<uint64_t>(v), drop.threshold) : 0xFFu;
    if (v < whole) {
      float f[8];
      widen<F32>(raw[i], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = keep >> j & 1u ? f[j] * drop.scale : 0.f;
      store_raw<F32>(y, 8 * v, narrow<F32>(f));
    } else {
      for (int j = 0; j < static_cast<int>(n - 8 * v); ++j) {
        float f;
        if constexpr (F32) f = static_cast<const float*>(x)[8 * v + j];
        else f = __bfloat162float(static_cast<const __nv_bfloat16*>(x)[8 * v + j]);
        f = keep >> j & 1u ? f * drop.scale : 0.f;
        if constexpr (F32) static_cast<float*>(y)[8 * v + j] = f;
        else static_cast<__nv_bfloat16*>(y)[8 * v + j] = __float2bfloat16_rn(f);
      }
    }
  }
}

// The threads of a row: enough that a thread has at most four pieces of it (32 values in
// registers); rows of up to 1024 values take a warp, four to a block.
template <typename Launch>
void by_length(int64_t H, const Launch& launch) {
  const int64_t vecs = H / 8;
  if (vecs <= 32 * 4) launch(std::integral_constant<int, 32>{});
  else if (vecs <= 128 * 4) launch(std::integral_constant<int, 128>{});
  else if (vecs <= 256 * 4) launch(std::integral_constant<int, 256>{});
  else launch(std::integral_constant<int, 512>{});
}

}  // namespace

bsmma_status launch_branch_enter(const EnterArgs& a, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  by_length(a.H, [&](auto tpr) {
    constexpr int kTpr = decltype(tpr)::value, kRows = kBlock<kTpr> / kTpr;
    const unsigned blocks = static_cast<unsigned>((a.T + kRows - 1) / kRows);
    e = launch_dependent(a.x_f32 ? enter_kernel<true, kTpr, 4> : enter_kernel<false, kTpr, 4>,
                         dim3(blocks), dim3(kBlock<kTpr>), 0, stream, a);
  });
  count_launches(1);
  return cuda_ok(e);
}

bsmma_status launch_branch_leave(const LeaveArgs& a, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  by_length(a.H, [&](auto tpr) {
    constexpr int kTpr = decltype(tpr)::value, kRows = kBlock<kTpr> / kTpr;
    const unsigned blocks = static_cast<unsigned>((a.T + kRows - 1) / kRows);
    const auto kern = !a.x_f32   ? leave_kernel<false, false, kTpr, 4>
                      : a.y_f32 ? leave_kernel<true, true, kTpr, 4>
                                : leave_kernel<true, false, kTpr, 4>;
    e = launch_dependent(kern, dim3(blocks), dim3(kBlock<kTpr>), 0, stream, a);
  });
  count_launches(1);
  return cuda_ok(e);
}

bsmma_status launch_dropout(const void* x, bool f32, int64_t n, const DropArgs& drop, void* y,
                            cudaStream_t stream) {
  const int64_t pieces = (n + 7) / 8;
  const unsigned blocks = static_cast<unsigned>((pieces + 256 * kDropPieces - 1) / (256 * kDropPieces));
  const cudaError_t e = launch_dependent(f32 ? dropout_kernel<true> : dropout_kernel<false>,
                                         dim3(blocks), dim3(256), 0, stream, x, n, drop, y);
  count_launches(1);
  return cuda_ok(e);
}

}  // namespace bsmma
