// branch.cu -- the residual branch forward: the norm before a block (branch_enter), the step
// after it (branch_leave) and dropout by itself.
//
// DRAM is their floor, so every row is read once, kept in registers through its reductions, and
// written once.  It bounds the others; rows of BF16 that become codes, or pass through two norms and
// dropout, are held up by their instructions and by the chain of a row's reductions (half to two thirds
// of the issue slots).  The norm of the next block is taken from the row while it is there, and a
// product's operand (INT8 rows, MX codes with their scales) is made from the FP32 values of the norm,
// so that neither the normed row nor a second reading of the stream costs any bytes.
#include <algorithm>

#include "branch.cuh"
#include "branch.h"

namespace bsmma {
namespace {
using namespace branch;

// ------------------------------------------------------------------------- norms
constexpr int kPieces = 4;   // a thread's, in registers (rows of up to 256 values: one, up to 512: two)

// f (zeros in pieces past the row) -> n(f) * weight + bias.  The variance of a layer norm is
// summed around the mean, in a second pass over the registers: a row far from zero keeps its
// digits.  part: 64 floats.
template <bool WARP, int V>
__device__ __forceinline__ void norm_row(Vals (&f)[V], const NormArgs& a, const Place<WARP, V>& at, float inv_h,
                                         float* part) {
  float s[1];
  if (a.kind == BSMMA_NORM_LAYER) {
    float2 acc[2] = {both(0.f), both(0.f)};
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j & 1] = add2(acc[j & 1], f[i].v[j]);
    s[0] = (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
    row_sums<WARP>(s, part);
    const float2 minus_mean = both(-s[0] * inv_h);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (at.in(i))
#pragma unroll
        for (int j = 0; j < 4; ++j) f[i].v[j] = add2(f[i].v[j], minus_mean);
    part += 32;
  }
  float2 acc[2] = {both(0.f), both(0.f)};
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j & 1] = __ffma2_rn(f[i].v[j], f[i].v[j], acc[j & 1]);
  s[0] = (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
  row_sums<WARP>(s, part);
  const float2 rs = both(inv_sqrt(fmaf(s[0], inv_h, a.eps)));
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) f[i].v[j] = mul2(f[i].v[j], rs);
  // what a call may leave out stands in loops of its own, which it jumps over
  if (a.weight) {
    const float* w0 = a.weight + 8 * at.base;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (at.in(i)) {
        const Vals w = load_columns(w0, 256 * i);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[i].v[j] = mul2(f[i].v[j], w.v[j]);
      }
  }
  if (a.bias) {
    const float* b0 = a.bias + 8 * at.base;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (at.in(i)) {
        const Vals b = load_columns(b0, 256 * i);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[i].v[j] = add2(f[i].v[j], b.v[j]);
      }
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

// One piece's codes at `codes` and, by one lane of four, its block's scale at `scale`; the four lanes
// that hold a block of 32 are all here (a row has whole blocks).  in: the piece is in the row.
template <int FMT>
__device__ __forceinline__ void store_mx(const Vals& f, uint8_t* codes, uint8_t* scale, bool in, bool first) {
  constexpr int kEmax = FMT == BSMMA_OPERAND_E4M3 ? 8 : FMT == BSMMA_OPERAND_E5M2 ? 15 : 2;
  float amax = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) amax = fmaxf(fmaxf(amax, fabsf(f.v[j].x)), fabsf(f.v[j].y));
  amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
  if (!in) return;
  // floor(log2 amax) - emax + 127, at least 0: the exponent field less emax (a subnormal's
  // field is 0, and what is below it would be cut to 0 as well); 127 for a block of zeros
  const int field = static_cast<int>(__float_as_uint(amax) >> 23);
  const int code = amax == 0.f ? 127 : max(field - kEmax, 0);
  const float2 inv = both(__uint_as_float(static_cast<uint32_t>(254 - code) << 23));   // 2^(127 - code)
  float2 y[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) y[j] = mul2(f.v[j], inv);
  if constexpr (FMT == BSMMA_OPERAND_E2M1) {
    *reinterpret_cast<uint32_t*>(codes) = fp4x2(y[0].x, y[0].y) | fp4x2(y[1].x, y[1].y) << 8 |
                                          fp4x2(y[2].x, y[2].y) << 16 | fp4x2(y[3].x, y[3].y) << 24;
  } else {
    *reinterpret_cast<uint2*>(codes) = make_uint2(fp8x2<FMT>(y[0].x, y[0].y) | fp8x2<FMT>(y[1].x, y[1].y) << 16,
                                                  fp8x2<FMT>(y[2].x, y[2].y) | fp8x2<FMT>(y[3].x, y[3].y) << 16);
  }
  if (first) *scale = static_cast<uint8_t>(code);
}
template <int FMT, bool WARP, int V>
__device__ __forceinline__ void store_mx_row(const Vals (&f)[V], const OperandArgs& to, int64_t t, int64_t H,
                                             const Place<WARP, V>& at) {
  constexpr int kCodes = FMT == BSMMA_OPERAND_E2M1 ? 4 : 8;   // bytes of a piece
  uint8_t* codes = static_cast<uint8_t*>(to.out) + t * (H / 8) * kCodes + at.base * kCodes;
  uint8_t* scales = static_cast<uint8_t*>(to.scales) + t * (H / 32) + (at.base >> 2);
#pragma unroll
  for (int i = 0; i < V; ++i)
    store_mx<FMT>(f[i], codes + 32 * kCodes * i, scales + 8 * i, at.in(i), (at.base & 3) == 0);
}

// The INT8 scale of a row's largest magnitude, and a piece's codes: the quotient rounded once, by
// two fused corrections on the reciprocal (Markstein's, as int8_quantize takes it) where nothing of them
// leaves FP32's range.
struct Int8Scale {
  float s, inv;   // inv 0: outside that range
};
__device__ __forceinline__ Int8Scale int8_scale(uint32_t amax) {
  float s = __fmul_rn(__uint_as_float(amax), 1.f / 127.f);
  if (s == 0.f) s = 1.f;
  return Int8Scale{s, s >= 0x1p-88f && s <= 0x1p100f ? __fdiv_rn(1.f, s) : 0.f};
}
__device__ __forceinline__ uint32_t magnitude(const Vals& f, uint32_t amax) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    amax = max(max(amax, __float_as_uint(f.v[j].x) & 0x7FFFFFFFu), __float_as_uint(f.v[j].y) & 0x7FFFFFFFu);
  return amax;
}
__device__ __forceinline__ uint2 int8_codes(const Vals& f, const Int8Scale& k) {
  const float2 inv = both(k.inv), minus_s = both(-k.s);
  uint32_t c[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x = f.v[j];
    float2 q = mul2(x, inv);
    q = __ffma2_rn(__ffma2_rn(minus_s, q, x), inv, q);
    q = __ffma2_rn(__ffma2_rn(minus_s, q, x), inv, q);
    if (k.inv == 0.f) q = make_float2(__fdiv_rn(x.x, k.s), __fdiv_rn(x.y, k.s));
    const int n0 = max(-127, min(127, __float2int_rn(q.x))), n1 = max(-127, min(127, __float2int_rn(q.y)));
    c[j >> 1] |= ((static_cast<uint32_t>(n0) & 0xFFu) | (static_cast<uint32_t>(n1) & 0xFFu) << 8) << (16 * (j & 1));
  }
  return make_uint2(c[0], c[1]);
}

template <bool WARP, int V>
__device__ __forceinline__ void store_int8(const Vals (&f)[V], const OperandArgs& to, int64_t t, int64_t H,
                                           const Place<WARP, V>& at, float* part) {
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) amax = magnitude(f[i], amax);
  const Int8Scale k = int8_scale(row_max<WARP>(amax, reinterpret_cast<uint32_t*>(part)));
  if (at.base == 0) static_cast<float*>(to.scales)[t] = k.s;
  int8_t* codes = static_cast<int8_t*>(to.out) + t * H + 8 * at.base;
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (at.in(i)) *reinterpret_cast<uint2*>(codes + 256 * i) = int8_codes(f[i], k);
}

template <bool WARP, int V>
__device__ __forceinline__ void store_operand(const Vals (&f)[V], const OperandArgs& to, int64_t t, int64_t H,
                                              const Place<WARP, V>& at, float* part) {
  switch (to.form) {
    case BSMMA_OPERAND_BF16:
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (at.in(i)) store_raw<false>(to.out, t * H + 8 * at.base + 256 * i, narrow<false>(f[i]));
      break;
    case BSMMA_OPERAND_F32:
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (at.in(i)) store_raw<true>(to.out, t * H + 8 * at.base + 256 * i, narrow<true>(f[i]));
      break;
    case BSMMA_OPERAND_INT8: store_int8<WARP>(f, to, t, H, at, part); break;
    case BSMMA_OPERAND_E4M3: store_mx_row<BSMMA_OPERAND_E4M3, WARP>(f, to, t, H, at); break;
    case BSMMA_OPERAND_E5M2: store_mx_row<BSMMA_OPERAND_E5M2, WARP>(f, to, t, H, at); break;
    default: store_mx_row<BSMMA_OPERAND_E2M1, WARP>(f, to, t, H, at); break;
  }
}

// ------------------------------------------------------------------------- kernels
// WARP: a row a warp (rows of up to 1024 values), four warps a block; else a row a block, as many
// warps as give each thread four pieces.
template <bool WARP>
__device__ __forceinline__ int64_t row_of() {
  return WARP ? static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5) : blockIdx.x;
}
// Rows of up to 8192 values: at most 256 threads, registers for three or four blocks an SM.
constexpr int kMaxThreads = 512, kShortThreads = 256;

// A row a block (a warp), in registers.  16384 x 7168 BF16 into E4M3: 75 to 79 us, 356 MB at 4.5 to 4.7 TB/s
// (E2M1 78; INT8, whose maximum is one more reduction of the row, 105).  What holds it up is a row's chain,
// two reductions and a barrier, at 64% of the issue slots (120 instructions for eight values, 40 of them what
// a row costs each of its warps), and the weights' loads (57% of the L1 cache's cycles); FP32 into
// BF16 16384 x 4096 69 us, 403 MB at 5.8 TB/s.  Tried and slower: two pieces a thread (twice the warps, each
// with a row's costs: 104 us, and a step with dropout, gate and two norms 208 for 179), two rows a block
// that share the weights (87 us, 14 warps an SM), and rows in a ring of asynchronous copies, one (78) or
// two (86) at a time, which widen the values anew in each pass.
template <bool F32, bool WARP, bool SHORT, int V>
__global__ void __launch_bounds__(SHORT ? kShortThreads : kMaxThreads, SHORT ? 4 : 2) enter_kernel(const EnterArgs p) {
  __shared__ float part[WARP ? 1 : 3 * 32];
  grid_dependency_wait();
  grid_launch_dependents();
  const Place<WARP, V> at(p.H);
  const int64_t t = row_of<WARP>();
  if (t >= p.T) return;   // (whole warps, and no barrier where a row is a warp's)
  Raw<F32> raw[V];
#pragma unroll
  for (int i = 0; i < V; ++i)
    raw[i] = at.in(i) ? load_raw<F32>(p.x, t * p.H + 8 * at.base + 256 * i) : zero_raw<F32>();
  Vals f[V];
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = widen<F32>(raw[i]);
  norm_row<WARP>(f, p.norm, at, p.inv_h, part);
  store_operand<WARP>(f, p.to, t, p.H, at, part + (WARP ? 0 : 64));
}

template <bool XF, bool YF, bool WARP, bool SHORT, int V>
__global__ void __launch_bounds__(SHORT ? kShortThreads : kMaxThreads, SHORT ? 3 : 1) leave_kernel(const LeaveArgs p) {
  __shared__ float part[WARP ? 1 : 5 * 32];
  grid_dependency_wait();
  grid_launch_dependents();
  const Place<WARP, V> at(p.H);
  const int64_t t = row_of<WARP>();
  if (t >= p.T) return;
  const float inv_h = p.inv_h;
  const int64_t row = t * p.H + 8 * at.base;
  Raw<YF> ry[V];
  Raw<XF> rx[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    ry[i] = at.in(i) ? load_raw<YF>(p.y, row + 256 * i) : zero_raw<YF>();
    rx[i] = at.in(i) ? load_raw<XF>(p.x, row + 256 * i) : zero_raw<XF>();
  }
  Vals f[V];
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = widen<YF>(ry[i]);
  if (p.norm.kind != BSMMA_NORM_NONE) norm_row<WARP>(f, p.norm, at, inv_h, part);
  if (p.drop.threshold != 0) {
    const Philox gen = philox_of(p.drop.rng);
    const uint64_t block = static_cast<uint64_t>(t) * at.vecs + at.base;
#pragma unroll
    for (int i = 0; i < V; ++i) drop(f[i], philox(gen, block + 32 * i), p.drop.threshold << 16);
  }
  if (p.gate) {
    const int64_t from =
        static_cast<int64_t>(static_cast<uint32_t>(t) / static_cast<uint32_t>(p.gate_rows)) * p.H + 8 * at.base;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (at.in(i)) {
        const Vals g = widen<YF>(load_raw<YF>(p.gate, from + 256 * i));
#pragma unroll
        for (int j = 0; j < 4; ++j) f[i].v[j] = mul2(f[i].v[j], g.v[j]);
      }
  }
  const float2 xs = both(p.x_scale), ys = both(p.y_scale * p.drop.scale);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const Vals x = widen<XF>(rx[i]);
#pragma unroll
    for (int j = 0; j < 4; ++j) f[i].v[j] = __ffma2_rn(ys, f[i].v[j], mul2(xs, x.v[j]));
    const Raw<XF> o = narrow<XF>(f[i]);
    if (at.in(i)) store_raw<XF>(p.out, row + 256 * i, o);
    f[i] = widen<XF>(o);   // the next norm is of what is stored
  }
  if (p.next.kind == BSMMA_NORM_NONE) return;
  norm_row<WARP>(f, p.next, at, inv_h, part + (WARP ? 0 : 64));
  store_operand<WARP>(f, p.to, t, p.H, at, part + (WARP ? 0 : 128));
}

// Eight values a piece (the last one may be short), kPieces in flight a thread.
template <bool F32>
__global__ void __launch_bounds__(256) dropout_kernel(const void* x, int64_t n, const DropArgs args, void* y) {
  grid_dependency_wait();
  grid_launch_dependents();
  const bool dropping = args.threshold != 0;
  Philox gen = {};
  if (dropping) gen = philox_of(args.rng);
  const uint32_t limit = args.threshold << 16;
  const float2 scale = both(args.scale);
  const int64_t whole = n / 8;
  const int64_t base = static_cast<int64_t>(blockIdx.x) * (256 * kPieces) + threadIdx.x;
  Raw<F32> raw[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i)
    if (base + 256 * i < whole) raw[i] = load_raw<F32>(x, 8 * (base + 256 * i));
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int64_t v = base + 256 * i;
    if (v < whole) {
      Vals f = widen<F32>(raw[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) f.v[j] = mul2(f.v[j], scale);
      if (dropping) drop(f, philox(gen, static_cast<uint64_t>(v)), limit);
      store_raw<F32>(y, 8 * v, narrow<F32>(f));
    } else if (v == whole && 8 * v < n) {
      uint4 words = make_uint4(0, 0, 0, 0);
      if (dropping) words = philox(gen, static_cast<uint64_t>(v));
      const uint32_t w[4] = {words.x, words.y, words.z, words.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (8 * v + j >= n) break;
        float f;
        if constexpr (F32) f = static_cast<const float*>(x)[8 * v + j];
        else f = __bfloat162float(static_cast<const __nv_bfloat16*>(x)[8 * v + j]);
        f = (j & 1 ? w[j >> 1] : w[j >> 1] << 16) >= limit ? f * args.scale : 0.f;
        if constexpr (F32) static_cast<float*>(y)[8 * v + j] = f;
        else static_cast<__nv_bfloat16*>(y)[8 * v + j] = __float2bfloat16_rn(f);
      }
    }
  }
}

constexpr int kWarpRow = 8 * 32 * kPieces;   // values of a row that a warp holds
unsigned threads_of(int64_t H) {
  return H <= kWarpRow ? 128u : static_cast<unsigned>(32 * ((H + kWarpRow - 1) / kWarpRow));
}

template <bool F32>
bsmma_status launch_enter(const EnterArgs& a, cudaStream_t stream) {
  const bool warp = a.H <= kWarpRow;
  const unsigned threads = threads_of(a.H);
  return cuda_ok(launch_dependent(a.H <= kWarpRow / 4        ? enter_kernel<F32, true, true, 1>
                                  : a.H <= kWarpRow / 2      ? enter_kernel<F32, true, true, 2>
                                  : warp                     ? enter_kernel<F32, true, true, kPieces>
                                  : threads <= kShortThreads ? enter_kernel<F32, false, true, kPieces>
                                                             : enter_kernel<F32, false, false, kPieces>,
                                  dim3(static_cast<unsigned>(warp ? (a.T + 3) / 4 : a.T)), dim3(threads), 0, stream, a));
}
template <bool XF, bool YF>
bsmma_status launch_leave(const LeaveArgs& a, cudaStream_t stream) {
  const unsigned threads = threads_of(a.H);
  const bool warp = a.H <= kWarpRow;
  return cuda_ok(launch_dependent(a.H <= kWarpRow / 4        ? leave_kernel<XF, YF, true, true, 1>
                                  : a.H <= kWarpRow / 2      ? leave_kernel<XF, YF, true, true, 2>
                                  : warp                     ? leave_kernel<XF, YF, true, true, kPieces>
                                  : threads <= kShortThreads ? leave_kernel<XF, YF, false, true, kPieces>
                                                             : leave_kernel<XF, YF, false, false, kPieces>,
                                  dim3(static_cast<unsigned>(warp ? (a.T + 3) / 4 : a.T)), dim3(threads), 0, stream, a));
}

}  // namespace

bsmma_status launch_branch_enter(const EnterArgs& a, cudaStream_t stream) {
  const bsmma_status st = a.x_f32 ? launch_enter<true>(a, stream) : launch_enter<false>(a, stream);
  count_launches(1);
  return st;
}

bsmma_status launch_branch_leave(const LeaveArgs& a, cudaStream_t stream) {
  const bsmma_status st = !a.x_f32   ? launch_leave<false, false>(a, stream)
                          : a.y_f32 ? launch_leave<true, true>(a, stream)
                                    : launch_leave<true, false>(a, stream);
  count_launches(1);
  return st;
}

bsmma_status launch_dropout(const void* x, bool f32, int64_t n, const DropArgs& drop, void* y,
                            cudaStream_t stream) {
  const int64_t pieces = (n + 7) / 8;
  const unsigned blocks = static_cast<unsigned>((pieces + 256 * kPieces - 1) / (256 * kPieces));
  const cudaError_t e = launch_dependent(f32 ? dropout_kernel<true> : dropout_kernel<false>, dim3(blocks),
                                         dim3(256), 0, stream, x, n, drop, y);
  count_launches(1);
  return cuda_ok(e);
}

}  // namespace bsmma
