// int8_gemm.cu -- INT8 products with scales for each token and channel, dense and grouped
// by expert, and the quantiser that makes their operands.
//
//   D[m][n] = sA[m] * sB[n] * sum_k A[m][k] * B[n][k]  (+ bias[n])
//
// sm_103a has no INT8 tcgen05 MMA, and its mma.sync INT8 rate (158 TOP/s measured) is a
// twelfth of the FP16 tensor rate.  An INT8 value is exact in FP16 and a product of two
// (at most 2^14) is exact in the FP32 accumulator, so the kernels widen both operands to
// FP16 on the way to the tensor core.  The sum is exact as long as its partial sums stay
// below 2^24 (any K <= 1024, and larger K unless almost all products have one sign), and
// is rounded as an FP32 sum beyond.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "int8.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace bsmma {
namespace {

using int8::Int8Params;
using int8::kMaxG;
using int8::store_out;
using int8::widen4;

constexpr uint32_t kFull = 0xFFFFFFFFu;

// ---------------------------------------------------------------- quantiser
// One row per TPR threads, kept in registers between the maximum and the codes (V 16-byte
// pieces a thread), or read twice when it is longer than that (V == 0).
// Bound by DRAM: 16384 rows of 7168 BF16 take 54 us, 352 MB at 6.6 TB/s.
//   s = amax * (1 / 127), both steps in FP32 (1 when that is zero), code = rint(x / s) within [-127, 127].
// The code is that of the correctly rounded quotient x / s, which comes from the reciprocal
// without a division a value, by the corrections that the FP8 quantisers use (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor", IBM J. Res.
// Dev. 34(1), 1990): with y = RN(1 / s), q0 = RN(x y) is within 1.5 ulp of x / s, one
// correction q + (x - s q) y by fused steps makes it one of the two neighbours, a second
// RN(x / s).  That needs s well inside the exponent range: 2^-88 to 2^100 here, where only
// quotients below 2^-11 lose anything, whose code is 0 either way; other rows divide.
struct QuantParams {
  const void* x;
  const int32_t* src;    // nullptr: row r is row r of x
  int64_t rows, x_rows;
  int vecs;              // 16-byte pieces of a row of x
  int k;                 // slots of a token: row r is row src[r] / k of x
  int8_t* codes;
  float* scales;
};

template <bool F32>
__device__ __forceinline__ void unpack(const uint4& r, float (&v)[F32 ? 4 : 8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (F32) {
      v[i] = __uint_as_float(w[i]);
    } else {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}

__device__ __forceinline__ uint32_t code_slow(float x, float s) {
  const float q = fminf(fmaxf(rintf(__fdiv_rn(x, s)), -127.f), 127.f);
  return static_cast<uint32_t>(static_cast<int>(q)) & 0xFFu;
}

__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// N (4 or 8) codes of x / s in bytes, two values an instruction.  inv = 1 / s, or 0 where the
// reciprocal does not serve.
template <int N>
__device__ __forceinline__ void codes_of(const float (&x)[N], float s, float inv,
                                         uint32_t (&out)[N / 4]) {
  constexpr float kMagic = 12582912.f;   // 1.5 * 2^23: adding it rounds to an integer
  uint32_t b[N];
  if (inv != 0.f) {
    const uint64_t inv2 = pack2(inv, inv), minus_s = pack2(-s, -s), zero = pack2(0.f, 0.f),
                   one = pack2(1.f, 1.f), magic2 = pack2(kMagic, kMagic);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const uint64_t x2 = pack2(x[i], x[i + 1]);
      const uint64_t q0 = fma2(x2, inv2, zero);
      const uint64_t q1 = fma2(fma2(minus_s, q0, x2), inv2, q0);
      const uint64_t q = fma2(fma2(minus_s, q1, x2), inv2, q1);
      float y0, y1;
      unpack2(fma2(q, one, magic2), y0, y1);
      b[i] = __float_as_uint(y0);
      b[i + 1] = __float_as_uint(y1);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) b[i] = code_slow(x[i], s);
  }
#pragma unroll
  for (int i = 0; i < N / 4; ++i)
    out[i] = __byte_perm(__byte_perm(b[4 * i], b[4 * i + 1], 0x0040),
                         __byte_perm(b[4 * i + 2], b[4 * i + 3], 0x0040), 0x5410);
}

template <bool F32, int TPR, int V>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) int8_quantize_kernel(const QuantParams p) {
  constexpr int kN = F32 ? 4 : 8, kThreads = TPR < 128 ? 128 : TPR;
  __shared__ uint32_t part[kThreads / 32];
  const int64_t r = static_cast<int64_t>(blockIdx.x) * (kThreads / TPR) + threadIdx.x / TPR;
  const int tid = threadIdx.x % TPR;
  if (r >= p.rows) return;   // whole warps only: TPR < 128 is 32, else one row per block
  int64_t xr = r;
  if (p.src) {
    const int32_t slot = p.src[r];
    xr = slot < 0 ? -1 : slot / p.k;
    if (xr >= p.x_rows) xr = -1;
  }
  const uint4* x = static_cast<const uint4*>(p.x) + xr * p.vecs;
  constexpr int kHeld = V > 0 ? V : 1;
  uint4 held[kHeld];
  uint32_t amax = 0;
  // BF16: the maximum of two magnitudes at a time, kept in a pair
  auto fold = [&](const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (F32) {
        amax = max(amax, w[i] & 0x7FFFFFFFu);
      } else {
        __nv_bfloat162 a = *reinterpret_cast<__nv_bfloat162*>(&amax);
        a = __hmax2(a, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[i])));
        amax = *reinterpret_cast<uint32_t*>(&a);
      }
    }
  };
  if constexpr (V > 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = tid + i * TPR;
      held[i] = make_uint4(0, 0, 0, 0);
      if (v < p.vecs && xr >= 0) held[i] = p.src ? x[v] : __ldcs(x + v);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) fold(held[i]);
  } else if (xr >= 0) {
    for (int v = tid; v < p.vecs; v += TPR) fold(x[v]);
  }
  if constexpr (!F32) amax = max(amax << 16, amax & 0xFFFF0000u);
  amax = __reduce_max_sync(kFull, amax);
  if constexpr (TPR > 32) {
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) amax = max(amax, part[i]);
  }
  float s = __fmul_rn(__uint_as_float(amax), 1.f / 127.f);
  if (s == 0.f) s = 1.f;
  if (tid == 0) p.scales[r] = s;
  const float inv = s >= 0x1p-88f && s <= 0x1p100f ? __fdiv_rn(1.f, s) : 0.f;
  uint32_t* out = reinterpret_cast<uint32_t*>(p.codes) + r * p.vecs * (kN / 4);
  auto emit = [&](int v, const uint4& h) {
    float f[kN];
    unpack<F32>(h, f);
    uint32_t c[kN / 4];
    codes_of(f, s, inv, c);
    if constexpr (F32)
      out[v] = c[0];
    else
      reinterpret_cast<uint2*>(out)[v] = make_uint2(c[0], c[1]);
  };
  if constexpr (V > 0) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (tid + i * TPR < p.vecs) emit(tid + i * TPR, held[i]);
  } else {
    for (int v = tid; v < p.vecs; v += TPR) emit(v, xr >= 0 ? x[v] : make_uint4(0, 0, 0, 0));
  }
}

template <bool F32>
bsmma_status launch_quantize_t(const QuantParams& p, cudaStream_t stream) {
  constexpr int V = 8;
  if (p.vecs <= 32 * 4)
    int8_quantize_kernel<F32, 32, 4><<<static_cast<unsigned>((p.rows + 3) / 4), 128, 0, stream>>>(p);
  else if (p.vecs <= 128 * V)
    int8_quantize_kernel<F32, 128, V><<<static_cast<unsigned>(p.rows), 128, 0, stream>>>(p);
  else if (p.vecs <= 512 * V)
    int8_quantize_kernel<F32, 512, V><<<static_cast<unsigned>(p.rows), 512, 0, stream>>>(p);
  else
    int8_quantize_kernel<F32, 512, 0><<<static_cast<unsigned>(p.rows), 512, 0, stream>>>(p);
  count_launches(1);
  return cuda_ok(cudaGetLastError());
}

// ---------------------------------------------------------------- products
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Row block `y` (blocks of R rows of one group, groups in order) -> group, its first row
// and its rows left.  Called by every thread of a 256-thread block; false past the last
// block or when the sizes are negative or exceed total_M.
struct RowBlock {
  int64_t row0;
  int g, rows, state;   // state: 1 found, 0 past the end, -1 bad sizes
};
__device__ __forceinline__ bool find_row_block(const Int8Params& p, int64_t y, int R,
                                               RowBlock& rb) {
  if (!p.m_sizes) {
    rb.g = 0;
    rb.row0 = y * R;
    const int64_t left = p.total_M - rb.row0;
    rb.rows = left < R ? static_cast<int>(left) : R;
    return left > 0;
  }
  constexpr int kPer = kMaxG / 256;
  __shared__ RowBlock found;
  __shared__ int64_t warp_rows[8], warp_blocks[8];
  __syncthreads();
  if (threadIdx.x == 0) found.state = 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t m[kPer], rows = 0, blocks = 0;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int g = threadIdx.x * kPer + i;
    m[i] = g < p.G ? p.m_sizes[g] : 0;
    if (m[i] < 0 || m[i] > p.total_M) {
      bad = true;
      m[i] = 0;
    }
    rows += m[i];
    blocks += (m[i] + R - 1) / R;
  }
  int64_t ir = rows, ib = blocks;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t a = __shfl_up_sync(kFull, ir, o), b = __shfl_up_sync(kFull, ib, o);
    if (lane >= o) {
      ir += a;
      ib += b;
    }
  }
  if (lane == 31) {
    warp_rows[warp] = ir;
    warp_blocks[warp] = ib;
  }
  bad = __syncthreads_or(bad);
  int64_t r0 = ir - rows, b0 = ib - blocks, all = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    if (w < warp) {
      r0 += warp_rows[w];
      b0 += warp_blocks[w];
    }
    all += warp_rows[w];
  }
  bad = bad || all > p.total_M;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int64_t nb = (m[i] + R - 1) / R;
    if (!bad && y >= b0 && y < b0 + nb) {
      found.g = threadIdx.x * kPer + i;
      found.row0 = r0 + (y - b0) * R;
      const int64_t left = m[i] - (y - b0) * R;
      found.rows = left < R ? static_cast<int>(left) : R;
      found.state = 1;
    }
    r0 += m[i];
    b0 += nb;
  }
  if (bad && threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0)
    report_status(p.status, kDevBadMSizes);
  __syncthreads();
  rb = found;
  return rb.state == 1;
}

// Products of few rows: bound by reading B once.  A block of 8 warps takes 32 channels and
// up to 8 * NT rows of A; its warps share out K in pieces of 128 and add their sums through
// shared memory.  A lane reads 16 consecutive K of a channel straight into registers and
// uses the same 16 K of A, so the order of K inside an MMA step (the same for both
// operands) needs no shuffle.
template <int NT, bool F32>
__global__ void __launch_bounds__(256) int8_rows_kernel(const Int8Params p) {
  constexpr int R = 8 * NT;
  __shared__ float sums[8][32 * R];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q = lane >> 2, t = lane & 3;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 32;
  for (int64_t y = blockIdx.y;; y += gridDim.y) {
    RowBlock rb;
    if (!find_row_block(p, y, R, rb)) return;
    const int8_t* B = p.B + static_cast<int64_t>(rb.g) * p.N * p.K;
    const int8_t* wrow[4];
    bool wok[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t n = n0 + q + 8 * i;
      wok[i] = n < p.N;
      wrow[i] = B + (wok[i] ? n : 0) * p.K + 16 * t;
    }
    const int8_t* arow[NT];
    bool aok[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      aok[i] = q + 8 * i < rb.rows;
      arow[i] = p.A + (rb.row0 + (aok[i] ? q + 8 * i : 0)) * p.K + 16 * t;
    }
    float acc[2][NT][4] = {};
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int64_t k0 = warp * 128; k0 < p.K; k0 += 8 * 128) {
      uint4 w[2][4], a[2][NT];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const bool in = k0 + 64 * c + 16 * t < p.K;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[c][i] = in && wok[i] ? __ldcs(reinterpret_cast<const uint4*>(wrow[i] + k0 + 64 * c)) : zero;
#pragma unroll
        for (int i = 0; i < NT; ++i)
          a[c][i] = in && aok[i] ? *reinterpret_cast<const uint4*>(arow[i] + k0 + 64 * c) : zero;
      }
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          auto word = [&](const uint4& v) { return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w; };
          uint32_t fa[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            widen4(word(w[c][2 * h]), fa[h][0], fa[h][2]);
            widen4(word(w[c][2 * h + 1]), fa[h][1], fa[h][3]);
          }
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            uint32_t b0, b1;
            widen4(word(a[c][i]), b0, b1);
            mma_16816(acc[0][i], fa[0], b0, b1);
            mma_16816(acc[1][i], fa[1], b0, b1);
          }
        }
    }
    // accumulator element: channel q (+8) of half h, rows 2t, 2t+1 of row tile i
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sums[warp][(8 * i + 2 * t + (e & 1)) * 32 + 16 * h + q + 8 * (e >> 1)] = acc[h][i][e];
    __syncthreads();
    for (int o = threadIdx.x; o < 32 * rb.rows; o += 256) {
      const int64_t n = n0 + (o & 31), m = rb.row0 + (o >> 5);
      if (n < p.N) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) s += sums[w][o];
        s *= p.sA[m] * p.sB[static_cast<int64_t>(rb.g) * p.N + n];
        if (p.bias) s += __bfloat162float(p.bias[n]);
        store_out<F32>(p.D, m * p.N + n, s);
      }
    }
    if (!p.m_sizes && (y + gridDim.y) * R >= p.total_M) return;
  }
}

template <int NT>
bsmma_status launch_rows(const Int8Params& p, bool f32, cudaStream_t stream) {
  int64_t blocks = (p.total_M + 8 * NT - 1) / (8 * NT);
  if (p.m_sizes) blocks += p.G < p.total_M ? p.G : p.total_M;
  if (blocks < 1) blocks = 1;   // the sizes are still checked
  const dim3 grid(static_cast<unsigned>((p.N + 31) / 32),
                  static_cast<unsigned>(blocks < 32768 ? blocks : 32768));
  if (f32)
    int8_rows_kernel<NT, true><<<grid, 256, 0, stream>>>(p);
  else
    int8_rows_kernel<NT, false><<<grid, 256, 0, stream>>>(p);
  count_launches(1);
  return cuda_ok(cudaGetLastError());
}

}  // namespace

bsmma_status launch_int8_quantize(const void* x, bool f32, int64_t x_rows, int64_t rows, int64_t K,
                                  const int32_t* src, int k, int8_t* codes, float* scales,
                                  cudaStream_t stream) {
  QuantParams p;
  p.x = x;
  p.src = src;
  p.rows = rows;
  p.x_rows = x_rows;
  p.vecs = static_cast<int>(K / (f32 ? 4 : 8));
  p.k = k;
  p.codes = codes;
  p.scales = scales;
  return f32 ? launch_quantize_t<true>(p, stream) : launch_quantize_t<false>(p, stream);
}

bsmma_status launch_int8_gemm(const int8_t* A, const float* sA, const int8_t* B, const float* sB,
                              const void* bias, void* D, bool f32, const int64_t* m_sizes,
                              int64_t total_M, int G, int64_t N, int64_t K, cudaStream_t stream) {
  bsmma_status st;
  const DeviceInfo* dev = current_device(&st);
  if (!dev) return st;
  Int8Params p;
  p.A = A;
  p.sA = sA;
  p.B = B;
  p.sB = sB;
  p.bias = static_cast<const __nv_bfloat16*>(bias);
  p.D = D;
  p.m_sizes = m_sizes;
  p.total_M = total_M;
  p.N = N;
  p.K = K;
  p.G = G;
  p.status = dev->status;
  const int64_t per_group = (total_M + G - 1) / G;
  const int tile = int8_tile();
  // The few-row kernel has the shorter start (1 x 1024 x 1024: 10.7 against 12.8 us), the
  // SM-pair kernel streams faster (4 x 14336 x 4096: 35.3 against 23.0 us).
  const bool few = tile == 1 || (tile == 0 && per_group <= 8 &&
                                 static_cast<int64_t>(G) * N * K <= (int64_t(8) << 20));
  if (!few && K > 0) return int8::launch_pair(p, f32, dev, stream);
  if (per_group <= 8) return launch_rows<1>(p, f32, stream);
  if (per_group <= 16) return launch_rows<2>(p, f32, stream);
  return launch_rows<4>(p, f32, stream);
}

}  // namespace bsmma
