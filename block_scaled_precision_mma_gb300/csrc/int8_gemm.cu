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
  const bool in = r < p.rows;   // (a warp's other rows may still be)
  int64_t xr = in ? r : -1;
  if (p.src && in) {
    const int32_t slot = p.src[r];
    xr = slot < 0 ? -1 : slot / p.k;
    if (xr >= p.x_rows) xr = -1;
  }
  const uint4* x = static_cast<const uint4*>(p.x) + xr * p.vecs;
  constexpr int kHeld = V > 0 ? V : 1;
  uint4 held[kHeld];
  uint32_t amax = 0;
  // BF16: the maximum of two magnitudes at a time, kept in a pair.  NaN is above infinity in the
  // order of the bits, and passes the pairs' maximum too.
  auto fold = [&](const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (F32) {
        amax = max(amax, w[i] & 0x7FFFFFFFu);
      } else {
        __nv_bfloat162 a = *reinterpret_cast<__nv_bfloat162*>(&amax);
        a = __hmax2_nan(a, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[i])));
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
  if constexpr (TPR < 32) {
#pragma unroll
    for (int o = TPR / 2; o; o >>= 1) amax = max(amax, __shfl_xor_sync(kFull, amax, o));
  } else {
    amax = __reduce_max_sync(kFull, amax);
  }
  if constexpr (TPR > 32) {
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) amax = max(amax, part[i]);
  }
  float s = __fmul_rn(__uint_as_float(amax), 1.f / 127.f);
  if (s == 0.f) s = 1.f;
  if (!in) return;
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
  // short rows share a warp, and rows of up to 256 pieces take one warp each (no barrier)
  constexpr int V = 8;
  const unsigned blocks4 = static_cast<unsigned>((p.rows + 3) / 4);
  if (p.vecs <= 8 * 4)
    int8_quantize_kernel<F32, 8, 4><<<static_cast<unsigned>((p.rows + 15) / 16), 128, 0, stream>>>(p);
  else if (p.vecs <= 32 * 4)
    int8_quantize_kernel<F32, 32, 4><<<blocks4, 128, 0, stream>>>(p);
  else if (p.vecs <= 32 * V)
    int8_quantize_kernel<F32, 32, V><<<blocks4, 128, 0, stream>>>(p);
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

__device__ __forceinline__ void cp_async_16(uint32_t dst_smem, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst_smem), "l"(src),
               "r"(in ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}

// Products of few rows: bound by reading B once, so everything is arranged to keep its bytes
// in flight.  One block of 8 warps an SM takes units of 32 channels x up to 8 * NT rows in
// turn; its warps share out K in pieces of 128, each warp with a ring of kStages pieces of its
// own (160 KB in flight an SM) that runs on across units, and their sums meet in shared memory
// at a unit's end.  A lane copies and reads back its own 16 consecutive K of a channel and uses
// the same 16 K of A, so no barrier is needed inside a unit and the order of K inside an MMA
// step (the same for both operands) needs no shuffle.
template <int NT>
struct RowsCfg {
  static constexpr int kPieceBytes = (8 + 2 * NT) * 512;   // a warp's 128 K: 32 channels, 8 NT rows
  static constexpr int kStages = NT == 1 ? 5 : 4;
  static constexpr int kRingBytes = 8 * kStages * kPieceBytes;
  static constexpr int kSumBytes = 8 * 32 * 8 * NT * 4;
  static constexpr int kSmemBytes = kRingBytes + kSumBytes + static_cast<int>(sizeof(int8::GroupTable<256>));
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

template <int NT, bool F32>
__global__ void __launch_bounds__(256, 1) int8_rows_kernel(const Int8Params p) {
  using C = RowsCfg<NT>;
  constexpr int R = 8 * NT, S = C::kStages;
  extern __shared__ __align__(16) uint8_t smem[];
  float* sums = reinterpret_cast<float*>(smem + C::kRingBytes);   // [warp][row][channel]
  int8::GroupTable<256>& table =
      *reinterpret_cast<int8::GroupTable<256>*>(smem + C::kRingBytes + C::kSumBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q = lane >> 2, t = lane & 3;
  int8::build_table(table, p, R);
  if (table.bad) return;
  const int tiles = static_cast<int>((p.N + 31) / 32), units = table.tile0[p.G] * tiles;
  const int pieces = static_cast<int>((p.K + 127) / 128);
  const int mine = pieces > warp ? (pieces - warp + 7) / 8 : 0;   // of every unit
  const uint32_t ring = smem_u32(smem) + warp * (S * C::kPieceBytes) + lane * 16;

  struct Place {
    int g, row0, rows;
    int64_t n0;
  };
  auto place = [&](int u) {
    Place r;
    const int mt = u / tiles;
    r.n0 = static_cast<int64_t>(u - mt * tiles) * 32;
    r.g = int8::find_group(table, p.G, mt);
    const int off = (mt - table.tile0[r.g]) * R;
    r.row0 = table.start[r.g] + off;
    const int left = table.start[r.g + 1] - r.row0;
    r.rows = left < R ? left : R;
    return r;
  };

  // the copies run kStages - 1 pieces ahead of the products
  int pu = mine > 0 ? static_cast<int>(blockIdx.x) : units, pi = 0, pslot = 0;
  const int8_t *wsrc = nullptr, *asrc = nullptr;
  uint32_t ok = 0;   // bits 0-3: the lane's channels exist; 4..: its rows
  auto issue = [&] {
    if (pu < units) {
      if (pi == 0) {
        const Place u = place(pu);
        ok = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) ok |= (u.n0 + q + 8 * i < p.N ? 1u : 0u) << i;
#pragma unroll
        for (int i = 0; i < NT; ++i) ok |= (q + 8 * i < u.rows ? 1u : 0u) << (4 + i);
        wsrc = p.B + (static_cast<int64_t>(u.g) * p.N + u.n0 + q) * p.K + 16 * t + warp * 128;
        asrc = p.A + static_cast<int64_t>(u.row0 + q) * p.K + 16 * t + warp * 128;
      }
      const int64_t k = static_cast<int64_t>(pi) * 1024, k_lane = k + warp * 128 + 16 * t;
      const uint32_t dst = ring + pslot * C::kPieceBytes;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const bool in = k_lane + 64 * c < p.K;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool some = in && (ok >> i & 1u);
          cp_async_16(dst + (c * 4 + i) * 512, some ? wsrc + k + 64 * c + 8 * i * p.K : p.B, some);
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const bool some = in && (ok >> (4 + i) & 1u);
          cp_async_16(dst + (8 + c * NT + i) * 512, some ? asrc + k + 64 * c + 8 * i * p.K : p.B, some);
        }
      }
      if (++pi == mine) {
        pi = 0;
        pu += gridDim.x;
      }
    }
    cp_async_commit();
    if (++pslot == S) pslot = 0;
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue();

  int slot = 0;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const Place un = place(u);
    // the scales of this thread's outputs, loaded ahead of the sums
    float sa[NT], sb[NT], bias[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int o = i * 256 + threadIdx.x;
      const int64_t n = un.n0 + (o & 31);
      sa[i] = sb[i] = bias[i] = 0.f;
      if (n < p.N && (o >> 5) < un.rows) {
        sa[i] = p.sA[un.row0 + (o >> 5)];
        sb[i] = p.sB[un.g * p.N + n];
        if (p.bias) bias[i] = __bfloat162float(p.bias[n]);
      }
    }
    float acc[2][NT][4] = {};
    for (int it = 0; it < mine; ++it) {
      cp_async_wait<S - 2>();
      const uint32_t from = ring + slot * C::kPieceBytes;
      if (++slot == S) slot = 0;
      uint4 w[2][4], a[2][NT];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[c][i] = lds16(from + (c * 4 + i) * 512);
#pragma unroll
        for (int i = 0; i < NT; ++i) a[c][i] = lds16(from + (8 + c * NT + i) * 512);
      }
      issue();   // into the slot that the piece before this one was read from
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
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sums[(warp * R + 8 * i + 2 * t + (e & 1)) * 32 + 16 * h + q + 8 * (e >> 1)] = acc[h][i][e];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int o = i * 256 + threadIdx.x;
      const int64_t n = un.n0 + (o & 31);
      if (n < p.N && (o >> 5) < un.rows) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) s += sums[w * R * 32 + o];
        store_out<F32>(p.D, static_cast<int64_t>(un.row0 + (o >> 5)) * p.N + n,
                       int8::scale_sum(s, sa[i], sb[i], bias[i]));
      }
    }
    __syncthreads();
  }
  cp_async_wait_all();
}

template <int NT, bool F32>
bsmma_status launch_rows(const Int8Params& p, const DeviceInfo* dev, cudaStream_t stream) {
  using C = RowsCfg<NT>;
  static PerDevice ready;
  const bsmma_status st = ready.allow_smem(dev->device, int8_rows_kernel<NT, F32>, C::kSmemBytes);
  if (st != BSMMA_OK) return st;
  int64_t blocks = (p.total_M + 8 * NT - 1) / (8 * NT);
  if (p.m_sizes) blocks += p.G < p.total_M ? p.G : p.total_M;
  if (blocks < 1) blocks = 1;   // the sizes are still checked
  const int64_t units = blocks * ((p.N + 31) / 32);
  const int64_t grid = units < dev->sm_count ? units : dev->sm_count;
  int8_rows_kernel<NT, F32><<<static_cast<unsigned>(grid), 256, C::kSmemBytes, stream>>>(p);
  count_launches(1);
  return cuda_ok(cudaGetLastError());
}

// SM cycles that the few-row kernel is expected to take: its units in turn, each the pieces of
// its slowest warp at 24 bytes a cycle (15.5 with 16 rows) or, where units are short, 1000 a
// piece and 2600 for the sums and the next unit's start; a fifth more for uneven groups, some of
// which take several blocks; 5000 for the launch.  It wins where one or two row blocks read B
// once or B is small.  Graph replays with L2 flushed, a replay's start of some 4 us among them,
// against SM-pair tiles of 32: 4 x 14336 x 4096 16.9 and 23.0 us, 4 x 4096 x 4096 10.8 and 27.1,
// 32 x 4096 x 4096 14.8 and 27.1; but 32 x 14336 x 4096 31.2 and 23.0, 128 experts of 1408 x 2048
// with 4 rows each 92 and 84.  (One after another in a graph, B mostly in L2: 10.5 and 16.7, 5.2 and
// 17.2, 10.2 and 19.9; 26.0 and 16.7, 89 and 79.)
double rows_cycles(const Int8Params& p, const DeviceInfo* dev) {
  const double active = int8::groups_with_rows(p), rows = active > 0 ? p.total_M / active : 0;
  const int nt = (p.total_M + p.G - 1) / p.G <= 8 ? 1 : 2;
  const double units = int8::blocks_per_group(p, rows, 8 * nt) * active * ((p.N + 31) / 32);
  const double pieces = static_cast<double>((p.K + 1023) / 1024);   // of a warp
  const double unit = std::fmax(pieces * 32 * 1024 / (nt == 1 ? 24 : 15.5), 2600 + 1000 * pieces) + 300;
  return std::ceil(units / dev->sm_count) * unit * (p.G > 1 ? 1.2 : 1) + 5000;
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
  const bool few = tile == 1 || (tile == 0 && rows_cycles(p, dev) < int8::pair_cycles(p, dev));
  if (!few && K > 0) return int8::launch_pair(p, f32, dev, stream);
  if (per_group <= 8)
    return f32 ? launch_rows<1, true>(p, dev, stream) : launch_rows<1, false>(p, dev, stream);
  return f32 ? launch_rows<2, true>(p, dev, stream) : launch_rows<2, false>(p, dev, stream);
}

}  // namespace bsmma
