// moe_step.cu -- the experts and the weighted sum of a few tokens.
//
// What bounds it is reading the chosen experts' weights once, so the two products' kernels are
// built around keeping their bytes in flight with few instructions a byte: one block of 16 warps
// an SM, each warp with a ring of asynchronous copies of its own that runs on from one unit of
// work to the next (and, in the first product, up to four warps more that finish units).
//
// The products use mma.sync with the weights as the 16-row operand and up to 8 * NT tokens as
// columns: with a row or a few an expert the tensor cores wait for memory whatever their
// instruction, and this form needs no tile of tokens in shared memory.  BF16 weights meet BF16
// tokens.  Codes are widened to FP16, which holds every INT8, E4M3, E5M2 and E2M1 value, by
// one conversion for two values; the tokens are then FP16 too, times a power of two of their
// own that brings their largest value to 2^14 .. 2^15: a BF16 value's eight bits fit, and only
// what is below 2^-29 of the largest loses any.  (Widening to BF16 instead, by moving bits and a
// multiplication, kept the integer pipe busy at 52% with DRAM at 38%: 363 MB of E4M3 experts
// 115 us.)  The 32 K of a matrix step are one MX block, so a block's scale multiplies its sum,
// four FMAs for 16 rows, and no weight.  Sums are FP32.  The inner row is rounded once, to what the second
// product's operand can be beside its weights: FP16 over a power of two for each 32 values with codes,
// BF16 with BF16 weights, as it is between the grouped products (2 tokens, 1024 x 2048: 0.0024 off the 64-bit
// value, and 0.0017 with an FP32 inner row, which is the output's own rounding).
//
// First launch, for codes: the tokens in FP16.  Every block of the other two makes the table of who
// takes what (the chosen experts and their columns) for itself from the ids, in its ring's place.  (A
// table made by one block of a launch ahead of them cost a call 1 to 2 us more, and BF16 a launch.)
// Second: units of 32 inner columns (32 rows of Wg and the 32 of Wu) of one expert, or of 128 where
// rows are short and units many; the warps share out K and the rows, their sums meet in shared
// memory, and the inner row leaves in BF16, or in FP16 with a power of two for each 32 values.  Gate and
// up rows are put into the upper and lower half of the same 16-row operand, so that the lane that has a gate's sum has its up's
// too.  Third: units of 32 output columns over all chosen experts, the warps sharing out
// (expert, K) in runs; a warp adds an expert's columns, times their tokens' weights, to its
// tokens' sums, and the warps' sums are added in order.  Each starts under the one before
// (programmatic launch), but reads nothing before its own wait for it, not the ids nor the weights
// either: what a launch further ahead wrote is there for certain only then.
#include <cuda_fp16.h>

#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "epilogue.cuh"
#include "moe_step.h"
#include "ptx.cuh"

namespace bsmma {
namespace {

constexpr uint32_t kFull = 0xFFFFFFFFu;
constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int kMaxSlots = 1024, kMaxExperts = 1024;

// ------------------------------------------------------------------------- weights
// A stage is 64 bytes of each of a warp's 32 rows: `kBlocks` blocks of 32 K, of which a row's four
// lanes have eight consecutive values each, `kLaneBytes`.  (Stages of 128 bytes save a few
// instructions, but where the sums of many tokens leave room for two of them only one is on its
// way: 32 tokens of INT8 experts 554 us against 498; one token of E4M3 experts 81 and 84.)
constexpr int kRowStage = 64, kSetStage = 8 * kRowStage, kCodeStage = 4 * kSetStage;
template <int FORM>
struct Form {
  static constexpr bool kMx = FORM >= BSMMA_OPERAND_E4M3, kBf16 = FORM == BSMMA_OPERAND_BF16;
  static constexpr int kLaneBytes = kBf16 ? 16 : FORM == BSMMA_OPERAND_E2M1 ? 4 : 8;
  static constexpr int kBlockBytes = 4 * kLaneBytes, kBlocks = kRowStage / kBlockBytes;
  static constexpr int kStageK = 32 * kBlocks;
  static constexpr int kStage = kCodeStage + (kMx ? 32 * 8 : 0);   // a warp's: codes, then two words of scales a row
  // Block b of row g (of a set of eight) lies at the place of block b ^ (g / 2) of the row, so that
  // the lanes of one shared-memory access are in different banks (rows two apart share them).
  static __device__ __forceinline__ uint32_t place(int g, int byte) {
    return g * kRowStage + (byte ^ ((g >> 1) & (kBlocks - 1)) * kBlockBytes);
  }
};
template <int FORM>
__device__ __forceinline__ int row_bytes(int K) {   // (at most 2^17)
  return FORM == BSMMA_OPERAND_BF16 ? 2 * K : FORM == BSMMA_OPERAND_E2M1 ? K / 2 : K;
}

// Two E8M0 codes as FP32 (through BF16, which holds 2^-127 and has a NaN for 255).
__device__ __forceinline__ float2 e8m0x2(uint32_t codes) {
  uint32_t two;
  asm("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.bf16x2.ue8m0x2 %0, a;}" : "=r"(two) : "r"(codes));
  return make_float2(__uint_as_float(two << 16), __uint_as_float(two & 0xFFFF0000u));
}

// A lane's eight weights of a block, at shared address `at`, as four pairs (BF16 or FP16).
template <int FORM>
__device__ __forceinline__ void load_weights(uint32_t at, uint32_t (&o)[4]) {
  if constexpr (FORM == BSMMA_OPERAND_BF16) {
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
                 : "r"(at));
  } else if constexpr (FORM == BSMMA_OPERAND_E2M1) {
    uint32_t w;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(at));
    asm("{.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;}"
        : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
        : "r"(w));
  } else {
    uint32_t w[2];
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (FORM == BSMMA_OPERAND_INT8) {
        // 0x64 above a byte u is 1024 + u in FP16; u = code + 128
        const uint32_t u = w[i] ^ 0x80808080u, off = 0x64806480u;   // 1152
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(o[2 * i]) : "r"(__byte_perm(u, 0x64646464u, 0x4140)), "r"(off));
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(o[2 * i + 1]) : "r"(__byte_perm(u, 0x64646464u, 0x4342)), "r"(off));
      } else if constexpr (FORM == BSMMA_OPERAND_E4M3) {
        asm("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;}"
            : "=r"(o[2 * i]), "=r"(o[2 * i + 1])
            : "r"(w[i]));
      } else {   // E5M2 is the upper byte of FP16
        o[2 * i] = __byte_perm(w[i], 0u, 0x1404);
        o[2 * i + 1] = __byte_perm(w[i], 0u, 0x3424);
      }
    }
  }
}

// d += (or, FIRST, =) the product of a 16-row operand and eight columns over 16 K.
template <bool BF16, bool FIRST>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else if constexpr (FIRST)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void cp_async_16(uint32_t dst_smem, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst_smem), "l"(src),
               "r"(in ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_16(uint32_t dst_smem, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst_smem), "l"(src) : "memory");
}
// (bytes < 4: the rest is zero; the address is a word's)
__device__ __forceinline__ void cp_async_4(uint32_t dst_smem, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst_smem), "l"(src), "r"(bytes) : "memory");
}

// A value's power of two and FP16 form: the largest finite magnitude of a group of values goes to
// 2^14 .. 2^15 (FP16 ends at 65504).  2^-126 bounds the power below, so that it is a float.
__device__ __forceinline__ float group_power(float amax) {
  const int e = static_cast<int>(__float_as_uint(amax) >> 23) - 127 - 14;
  return amax > 0.f ? __uint_as_float(static_cast<uint32_t>(max(e, -126) + 127) << 23) : 1.f;
}

// ------------------------------------------------------------------------- who takes what
// The chosen experts in order, each with its columns (tokens) in tiles of `tile`.  A token that
// names an expert twice is one column with both weights.
struct Table {
  int entries;
  uint16_t expert[kMaxSlots];       // of each tile
  uint16_t first[kMaxSlots + 2];    // its first column; it ends where the next begins
  uint16_t slot[kMaxSlots];         // of each column: token * k + choice
  uint16_t token[kMaxSlots];
};
struct WeightedTable : Table {
  float weight[kMaxSlots];          // of each column
};
struct TableScratch {
  int start[kMaxExperts];           // counts, then first columns
  int32_t ids[kMaxSlots];
  uint16_t rank[kMaxSlots];
};
constexpr uint16_t kNone = 0xFFFF;

// By every thread of the block; what is at `s` is free again afterwards.
template <typename T>
__device__ __forceinline__ void build_table(T& t, TableScratch& s, const StepArgs& a, int tile) {
  const int tid = threadIdx.x, lane = tid & 31, slots = static_cast<int>(a.T) * a.k;
  const int threads = static_cast<int>(blockDim.x);
  for (int e = tid; e < a.E; e += threads) s.start[e] = 0;
  for (int i = tid; i < slots; i += threads) {
    const int32_t id = a.ids[i];
    s.ids[i] = id >= 0 && id < a.E ? id : -1;
  }
  __syncthreads();
  if (tid < 32) {
    // ranks in the slots' order: lanes with one expert find each other, the lowest counts them
    for (int c = 0; c < slots; c += 32) {
      const int i = c + lane;
      int id = i < slots ? s.ids[i] : -1;
      if (id >= 0)
        for (int j = i - i % a.k; j < i; ++j)
          if (s.ids[j] == id) {
            id = -1;
            break;
          }
      const uint32_t same = __match_any_sync(kFull, id >= 0 ? id : -1 - lane);
      const int before = __popc(same & ((1u << lane) - 1));
      const int base = id >= 0 ? s.start[id] : 0;
      __syncwarp();
      if (id >= 0 && before == 0) s.start[id] = base + __popc(same);
      __syncwarp();
      if (i < slots) s.rank[i] = id >= 0 ? static_cast<uint16_t>(base + before) : kNone;
    }
    int column = 0, entry = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + lane;
      const int n = e < a.E ? s.start[e] : 0, tiles = (n + tile - 1) / tile;
      int in = n, it = tiles;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kFull, in, o), v = __shfl_up_sync(kFull, it, o);
        if (lane >= o) in += u, it += v;
      }
      const int c0 = column + in - n, t0 = entry + it - tiles;
      if (e < a.E) s.start[e] = c0;
      for (int i = 0; i < tiles; ++i) {
        t.expert[t0 + i] = static_cast<uint16_t>(e);
        t.first[t0 + i] = static_cast<uint16_t>(c0 + i * tile);
      }
      column += __shfl_sync(kFull, in, 31);
      entry += __shfl_sync(kFull, it, 31);
    }
    if (lane == 0) {
      t.entries = entry;
      t.first[entry] = static_cast<uint16_t>(column);
    }
  }
  __syncthreads();
  for (int i = tid; i < slots; i += threads) {
    if (s.rank[i] == kNone) continue;
    const int id = s.ids[i], c = s.start[id] + s.rank[i];
    t.slot[c] = static_cast<uint16_t>(i);
    t.token[c] = static_cast<uint16_t>(i / a.k);
    if constexpr (std::is_same_v<T, WeightedTable>) {
      float w = a.weights[i];
      for (int j = i + 1; j % a.k; ++j)
        if (s.ids[j] == id) w += a.weights[j];
      t.weight[c] = w;
    }
  }
  __syncthreads();
}

// Block t: token t in FP16 and its power of two.
__global__ void __launch_bounds__(kThreads) step_tokens_kernel(const StepArgs a) {
  __shared__ uint32_t part[kWarps];
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t t = blockIdx.x;
  const uint4* x = static_cast<const uint4*>(a.x) + t * (a.H / 8);
  uint4* out = reinterpret_cast<uint4*>(a.x16) + t * (a.H / 8);
  const int vecs = static_cast<int>(a.H / 8);
  uint32_t amax = 0;   // of the finite values, as bits of a BF16 value
  for (int v = threadIdx.x; v < vecs; v += kThreads) {
    const uint4 q = x[v];
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t m = w[j] >> (16 * h) & 0x7FFFu;
        if (m < 0x7F80u) amax = max(amax, m);
      }
  }
  amax = __reduce_max_sync(kFull, amax);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
  __syncthreads();
  amax = __reduce_max_sync(kFull, part[threadIdx.x & (kWarps - 1)]);
  const float power = group_power(__uint_as_float(amax << 16)), inv = 1.f / power;
  for (int v = threadIdx.x; v < vecs; v += kThreads) {
    const uint4 q = x[v];
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __half2 h = __floats2half2_rn(__uint_as_float(w[j] << 16) * inv,
                                          __uint_as_float(w[j] & 0xFFFF0000u) * inv);
      o[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    out[v] = make_uint4(o[0], o[1], o[2], o[3]);
  }
  if (threadIdx.x == 0) a.x_power[t] = power;
}

// ------------------------------------------------------------------------- products
// A run of stages of a warp's 32 rows, four sets of eight: set r starts set_bytes[r] behind
// the first (a set past the matrix repeats the first: its sums are not used).
struct Source {
  const uint8_t* row;       // the lane's row of the first set (lane (g, t): row g), its chunk t
  const uint8_t* scales;    // the scales of row lane (of 32)
};
// A stage's scales are copied as the word that holds its first one and, where rows do not have whole
// words of them, the next word; never from behind `end`, the last scale of the matrix.
struct Scales {
  const uint8_t* end;
  bool whole;               // a stage's scales lie in one word
};
struct Sets {
  int64_t bytes[4];         // of codes
};

// Starts the copies of stage `stage` (from the row's first byte): lane (g, t) copies the 16-byte
// chunk t of its row in each set, lane l the word or words that have the scales of row l.
template <int FORM>
__device__ __forceinline__ void load_stage(uint32_t to, const Source& from, const Sets& sets, int stage,
                                           int bytes, const Scales& all) {
  using F = Form<FORM>;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int at = stage * kRowStage;
  const uint32_t d = to + F::place(g, 16 * t);
  const uint8_t* src = from.row + at;
  if (at + kRowStage <= bytes) {
#pragma unroll
    for (int r = 0; r < 4; ++r) cp_async_16(d + r * kSetStage, src + sets.bytes[r]);
  } else {   // the end of K: what is past it counts as zero
    const bool in = at + 16 * t < bytes;
#pragma unroll
    for (int r = 0; r < 4; ++r) cp_async_16(d + r * kSetStage, in ? src + sets.bytes[r] : from.row, in);
  }
  if constexpr (F::kMx) {
    const uint8_t* first = from.scales + stage * F::kBlocks;
    const uint8_t* word = first - (reinterpret_cast<uintptr_t>(first) & 3);
    const uint32_t d_scales = to + kCodeStage + 8 * lane;
    if (all.whole) {
      cp_async_4(d_scales, word, 4);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int64_t here = all.end - (word + 4 * i);
        cp_async_4(d_scales + 4 * i, here > 0 ? word + 4 * i : word,
                   here >= 4 ? 4 : here > 0 ? static_cast<int>(here) : 0);
      }
    }
  }
}

// What the columns bring to a stage: the lane's eight values of each block, and the powers of two
// of the lane's two result columns.  It is read from L2 or L1, so it is asked for ahead of the wait
// for the weights.
template <int FORM, int NT, bool POWERS>
struct Columns {
  uint4 x[Form<FORM>::kBlocks][NT];
  float p[POWERS ? Form<FORM>::kBlocks : 1][NT][2];
};
// x: where the lane's column (of each eight) has its first K of the stage, in bytes behind x0; left: K
// from there to the end; powers: where the stage's first blocks' are, in bytes behind p0.
template <int FORM, int NT, bool POWERS>
__device__ __forceinline__ void load_columns(Columns<FORM, NT, POWERS>& c, const uint8_t* x0, const uint32_t (&x)[NT],
                                             int left, const uint8_t* p0, const uint32_t (&powers)[NT][2]) {
  constexpr int kBlocks = Form<FORM>::kBlocks;
  const int t = threadIdx.x & 3;
  auto x_of = [&](int n, int j) { return *reinterpret_cast<const uint4*>(x0 + x[n] + 64 * j); };
  auto p_of = [&](int n, int c, int j) { return *reinterpret_cast<const float*>(p0 + powers[n][c] + 4 * j); };
  if (left + 8 * t >= 32 * kBlocks) {   // (uniform)
#pragma unroll
    for (int j = 0; j < kBlocks; ++j)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        c.x[j][n] = x_of(n, j);
      }
    if constexpr (POWERS) {   // (a slot's powers begin at a multiple of 16 bytes)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint8_t* from = p0 + powers[n][i];
          if constexpr (kBlocks == 4) {
            const float4 p = *reinterpret_cast<const float4*>(from);
            c.p[0][n][i] = p.x, c.p[1][n][i] = p.y, c.p[2][n][i] = p.z, c.p[3][n][i] = p.w;
          } else {
            static_assert(kBlocks == 2, "powers go with codes");
            const float2 p = *reinterpret_cast<const float2*>(from);
            c.p[0][n][i] = p.x, c.p[1][n][i] = p.y;
          }
        }
    }
  } else {
#pragma unroll
    for (int j = 0; j < kBlocks; ++j)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        c.x[j][n] = make_uint4(0, 0, 0, 0);
        if (32 * j < left) c.x[j][n] = x_of(n, j);
        if constexpr (POWERS) {
          const bool in = 32 * j < left + 8 * t;
          c.p[j][n][0] = in ? p_of(n, 0, j) : 0.f;
          c.p[j][n][1] = in ? p_of(n, 1, j) : 0.f;
        }
      }
  }
}

// A stage of the ring: the columns' values asked for, the wait for the weights, the next stage's
// load, and the products into acc: operand m has set 2 m in its upper and set 2 m + 1 in its lower
// eight rows.  scale_at: the address of the stage's first scale of the lane's row of the first set,
// of which only the place in its word matters, and set_blocks[r] that of set r behind it.
template <int FORM, int NT, bool POWERS, int PENDING, typename Load>
__device__ __forceinline__ void stage_products(float (&acc)[2][NT][4], const uint8_t* x0, const uint32_t (&x)[NT],
                                               const uint8_t* p0, const uint32_t (&powers)[NT][2], int left,
                                               uint32_t ring, const Load& load, uint32_t scale_at,
                                               const uint32_t (&set_blocks)[4], const Scales& all) {
  using F = Form<FORM>;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  Columns<FORM, NT, POWERS> c;
  load_columns<FORM, NT, POWERS>(c, x0, x, left, p0, powers);
  cp_async_wait<PENDING>();
  __syncwarp();   // the other lanes' copies, and their reads of the slot that is filled next
  load();
  float2 sw[F::kMx ? 4 : 1][F::kMx ? F::kBlocks / 2 : 1];
  if constexpr (F::kMx) {
    // a block past K counts as 2^-127 times zero: the scale there is the next row's, which may be NaN
    const int here = left + 8 * t;
    const uint32_t in_row = here < F::kStageK ? (1u << (here / 4)) - 1 : kFull;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      uint32_t codes;
      const uint32_t from = ring + kCodeStage + 8 * (r * 8 + g);
      if (all.whole) {
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(codes) : "r"(from));
        if (F::kBlocks == 2) codes >>= 8 * (scale_at & 2);
      } else {
        uint32_t more;
        asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(codes), "=r"(more) : "r"(from));
        codes = __funnelshift_r(codes, more, 8 * ((scale_at + set_blocks[r]) & 3)) & in_row;
      }
#pragma unroll
      for (int j = 0; j < F::kBlocks / 2; ++j) sw[r][j] = e8m0x2(codes >> (16 * j));
    }
  }
#pragma unroll
  for (int j = 0; j < F::kBlocks; ++j) {
    const uint32_t at = ring + F::place(g, j * F::kBlockBytes + t * F::kLaneBytes);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      uint32_t hi[4], lo[4];
      load_weights<FORM>(at + 2 * m * kSetStage, hi);
      load_weights<FORM>(at + (2 * m + 1) * kSetStage, lo);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint4& v = c.x[j][n];
        if constexpr (F::kMx || POWERS) {
          float d[4];
          mma<F::kBf16, true>(d, hi[0], lo[0], hi[1], lo[1], v.x, v.y);
          mma<F::kBf16, false>(d, hi[2], lo[2], hi[3], lo[3], v.z, v.w);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float f = 1.f;
            if constexpr (F::kMx) {
              const float2 two = sw[2 * m + (i >> 1)][j >> 1];
              f = j & 1 ? two.y : two.x;
            }
            if constexpr (POWERS) f *= c.p[j][n][i & 1];
            acc[m][n][i] = fmaf(d[i], f, acc[m][n][i]);
          }
        } else {
          mma<F::kBf16, false>(acc[m][n], hi[0], lo[0], hi[1], lo[1], v.x, v.y);
          mma<F::kBf16, false>(acc[m][n], hi[2], lo[2], hi[3], lo[3], v.z, v.w);
        }
      }
    }
  }
}

__device__ __forceinline__ float load_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ float activate(float x, int act) {
  if (act == BSMMA_ACT_RELU) return x < 0.f ? 0.f : x;
  if (act == BSMMA_ACT_GELU) return gelu_erf(x);
  return act == BSMMA_ACT_SILU ? x / (1.f + expf(-x)) : x;
}

// A block's walk over its units (every gridDim-th).  An expert's units are its tiles of rows, and
// within one its tiles of columns, so that what several of those read is read at one time.  Kept as
// a place in the expert's units: with few stages a unit its divisions would show.
struct Walk {
  int lead, tiles_c, at;   // the expert's first entry, its entries, the unit's number in the expert
  __device__ __forceinline__ void find(const Table& t) {
    int end = lead + 1;
    while (end < t.entries && t.expert[end] == t.expert[lead]) ++end;
    tiles_c = end - lead;
  }
  // step units further; false: past the last
  __device__ __forceinline__ bool forward(const Table& t, int step, int tiles) {
    at += step;
    while (at >= tiles * tiles_c) {
      at -= tiles * tiles_c;
      lead += tiles_c;
      if (lead >= t.entries) return false;
      find(t);
    }
    return true;
  }
  __device__ __forceinline__ bool begin(const Table& t, int unit, int tiles) {
    lead = tiles_c = at = 0;
    if (t.entries == 0) return false;
    find(t);
    return forward(t, unit, tiles);
  }
  __device__ __forceinline__ int entry() const { return tiles_c == 1 ? lead : lead + at % tiles_c; }
  __device__ __forceinline__ int rows() const { return tiles_c == 1 ? at : at / tiles_c; }
};

// Powers of two of an inner row: one for 32 values, whole fours of them.
__host__ __device__ constexpr int64_t power_stride(int64_t F) { return (F + 127) / 128 * 4; }

// The inner rows.  A unit is 16 inner columns for each of kWarps / G parts; warp w has part w % (16 / G)
// and every G-th stage of K from w / (16 / G) on.  More warps, one for each eight columns and 32 inner
// values, at most four, add the sums up and finish a unit while the others are at the next (done by one of
// theirs, the other fifteen waited for it a quarter of their time; with one for all of a unit 32 tokens,
// 32 experts of 2048 x 2048 in INT8 took 77 us for 69).
template <int FORM, int NT, int G>
struct InCfg {
  static constexpr int kParts = kWarps / G, kTile = 16 * kParts;   // a unit's parts and inner columns
  static constexpr int kStage = Form<FORM>::kStage;
  static constexpr int kSums = kWarps * 2 * NT * 512;
  static constexpr int kFixed = kSums + static_cast<int>(sizeof(Table)) + 32;
  static constexpr int kStages = (232448 - kFixed) / (kWarps * kStage);
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kBytes = kRing + kFixed;
  static_assert(kStages >= 2, "one stage in flight");
  static constexpr int kEnds = kTile / 32 * NT < 4 ? kTile / 32 * NT : 4;   // warps that finish units
  static constexpr int kThreadsIn = kThreads + 32 * kEnds;
};

template <int FORM, int NT, int G>
__global__ void __launch_bounds__(InCfg<FORM, NT, G>::kThreadsIn, 1) step_in_kernel(const StepArgs a) {
  using C = InCfg<FORM, NT, G>;
  using F = Form<FORM>;
  extern __shared__ __align__(128) uint8_t smem[];
  float4* sums = reinterpret_cast<float4*>(smem + C::kRing);   // [operand: two a part][NT][group][lane]
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kRing + C::kSums);   // the sums are there
  uint64_t* empty = full + 1;                                                 // ... have been read
  volatile int* abort = reinterpret_cast<volatile int*>(full + 2);
  Table& table = *reinterpret_cast<Table*>(smem + C::kRing + C::kSums + 32);
  if (threadIdx.x == 0) {
    mbar_init(full, kWarps);
    mbar_init(empty, C::kEnds);
    fence_mbar_init();
    *abort = 0;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int part = warp % C::kParts, group = warp / C::kParts;
  grid_dependency_wait();
  grid_launch_dependents();
  build_table(table, *reinterpret_cast<TableScratch*>(smem), a, 8 * NT);
  static_assert(sizeof(TableScratch) <= C::kRing, "the ring's place");

  const int K = static_cast<int>(a.H), bytes = row_bytes<FORM>(K), blocks = K / 32;
  const uint8_t* x0 = F::kBf16 ? static_cast<const uint8_t*>(a.x) : reinterpret_cast<const uint8_t*>(a.x16);
  const Scales all = {static_cast<const uint8_t*>(a.s_in) + static_cast<int64_t>(a.E) * 2 * a.F * blocks, blocks % 4 == 0};
  const int tiles = static_cast<int>((a.F + C::kTile - 1) / C::kTile), step = static_cast<int>(gridDim.x);
  const int stages = static_cast<int>((K + F::kStageK - 1) / F::kStageK);
  const int mine = group < stages ? (stages - group + G - 1) / G : 0;   // of a unit
  const uint32_t ring = smem_u32(smem) + warp * C::kStages * C::kStage;
  // A part's sets of rows from its first row f on (F % 8 == 0: a set is in the matrix
  // or not): Wg's f .. f + 7, Wu's, Wg's f + 8 .. f + 15, Wu's.
  auto set_row = [&](int64_t f, int r) { return (r & 1 ? a.F : 0) + (r >> 1 && f + 8 < a.F ? 8 : 0); };
  auto first_row = [&](int rows) {
    const int64_t f = static_cast<int64_t>(rows) * C::kTile + 16 * part;
    return f < a.F ? f : 0;
  };
  if (warp >= kWarps) {
    // What a unit's end needs beside the sums is asked for before them: lane t has the power of token t,
    // and the rows' INT8 scales are read ahead of the wait (read after it: 32 tokens, 32 experts of
    // 2048 x 2048 96 us for 77).
    const float powers = !F::kBf16 && lane < a.T ? a.x_power[lane] : 1.f;
    constexpr bool AHEAD = FORM == BSMMA_OPERAND_INT8 && C::kTile == 32;
    float row_scales[2][4];   // of the gate's rows and the up's
    int done = 0;
    Walk here;
    for (bool more = here.begin(table, blockIdx.x, tiles); more; more = here.forward(table, step, tiles), ++done) {
      const int entry = here.entry(), rows = here.rows();
      const int first = table.first[entry], count = table.first[entry + 1] - first;
      const int64_t expert = table.expert[entry];
      auto load_scales = [&](int64_t f0) {
        const float* of = static_cast<const float*>(a.s_in) + expert * 2 * a.F;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const int64_t f = f0 + 8 * m + g;
          row_scales[0][m] = f < a.F ? of[f] : 0.f, row_scales[1][m] = f < a.F ? of[a.F + f] : 0.f;
        }
      };
      if constexpr (AHEAD) load_scales(static_cast<int64_t>(rows) * C::kTile);
      if (!mbar_wait(full, done & 1, a.limit_ns, abort, a.status)) return;
      // eight columns and 32 inner values at a time: values 8 m + g of columns 2 t and 2 t + 1
      for (int qn = warp - kWarps; qn < C::kTile / 32 * ((count + 7) / 8); qn += C::kEnds) {
        const int q = qn % (C::kTile / 32), n = qn / (C::kTile / 32);
        const int64_t f0 = static_cast<int64_t>(rows) * C::kTile + 32 * q;
        if (f0 >= a.F) continue;
        if constexpr (FORM == BSMMA_OPERAND_INT8 && !AHEAD) load_scales(f0);
        int64_t slots[2];
        float power[2] = {1.f, 1.f};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int col = 8 * n + 2 * t + c;
          slots[c] = col < count ? table.slot[first + col] : -1;
          if constexpr (!F::kBf16) power[c] = __shfl_sync(kFull, powers, table.token[first + min(col, count - 1)]);
        }
        float v[2][4], amax[2] = {0.f, 0.f};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < G; ++w) {
            const float4 one = sums[(((4 * q + m) * NT + n) * G + w) * 32 + lane];
            s.x += one.x, s.y += one.y, s.z += one.z, s.w += one.w;
          }
          const int64_t f = f0 + 8 * m + g;
          if constexpr (FORM == BSMMA_OPERAND_INT8) {
            s.x *= row_scales[0][m], s.y *= row_scales[0][m];
            s.z *= row_scales[1][m], s.w *= row_scales[1][m];
          }
          v[0][m] = activate(s.x * power[0], a.act) * (s.z * power[0]);
          v[1][m] = activate(s.y * power[1], a.act) * (s.w * power[1]);
#pragma unroll
          for (int c = 0; c < 2; ++c)
            if (f < a.F && fabsf(v[c][m]) <= FLT_MAX) amax[c] = fmaxf(amax[c], fabsf(v[c][m]));
        }
        float inv[2] = {1.f, 1.f};
        if constexpr (!F::kBf16) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) amax[c] = fmaxf(amax[c], __shfl_xor_sync(kFull, amax[c], o));
            const float p = group_power(amax[c]);
            inv[c] = 1.f / p;
            if (g == 0 && slots[c] >= 0) a.inner_power[slots[c] * power_stride(a.F) + f0 / 32] = p;
          }
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const int64_t f = f0 + 8 * m + g;
          if (f >= a.F) continue;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if (slots[c] < 0) continue;
            uint16_t* to = a.inner + slots[c] * a.F + f;
            if constexpr (F::kBf16) *to = __bfloat16_as_ushort(__float2bfloat16_rn(v[c][m]));
            else *to = __half_as_ushort(__float2half_rn(v[c][m] * inv[c]));
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty);
    }
    return;
  }
  // the loads run ahead of the products through the block's units
  Walk ahead;
  bool to_load = ahead.begin(table, blockIdx.x, tiles) && mine;
  int li = 0, slot = 0;
  Source src = {};
  Sets sets = {};
  auto enter_unit = [&] {
    const int64_t f = first_row(ahead.rows());
    const int64_t base = static_cast<int64_t>(table.expert[ahead.lead]) * 2 * a.F + f;
    src.row = static_cast<const uint8_t*>(a.w_in) + (base + g) * bytes + 16 * t;
#pragma unroll
    for (int r = 0; r < 4; ++r) sets.bytes[r] = set_row(f, r) * bytes;
    if constexpr (F::kMx)
      src.scales = static_cast<const uint8_t*>(a.s_in) + (base + set_row(f, lane >> 3) + (lane & 7)) * blocks;
  };
  auto load = [&] {
    if (to_load) {
      load_stage<FORM>(ring + slot * C::kStage, src, sets, group + li * G, bytes, all);
      if (++li == mine) {
        li = 0;
        to_load = ahead.forward(table, step, tiles);
        if (to_load) enter_unit();
      }
    }
    cp_async_commit();
    slot = slot + 1 == C::kStages ? 0 : slot + 1;
  };
  if (to_load) enter_unit();
#pragma unroll
  for (int i = 0; i < C::kStages - 1; ++i) load();

  int at = 0, done = 0;
  Walk here;
  for (bool more = here.begin(table, blockIdx.x, tiles); more; more = here.forward(table, step, tiles), ++done) {
    const int entry = here.entry(), first = table.first[entry], count = table.first[entry + 1] - first;
    const int64_t expert = table.expert[entry], f_first = first_row(here.rows());
    uint32_t scale_at = static_cast<uint32_t>((expert * 2 * a.F + f_first + g) * blocks), set_blocks[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) set_blocks[r] = static_cast<uint32_t>(set_row(f_first, r) * blocks);
    // n_cols tiles of eight columns; a column past the entry's repeats its last
    auto products = [&](auto n_cols) {
      constexpr int N = decltype(n_cols)::value;
      uint32_t x[N];
      const uint32_t no_powers[N][2] = {};
      int k = group * F::kStageK;
#pragma unroll
      for (int n = 0; n < N; ++n)
        x[n] = 2 * (table.token[first + min(8 * n + g, count - 1)] * K + k + 8 * t);
      float acc[2][N][4] = {};
      for (int i = 0; i < mine; ++i) {
        stage_products<FORM, N, false, C::kStages - 2>(
            acc, x0, x, x0, no_powers, K - k - 8 * t, ring + at * C::kStage, load, scale_at + k / 32,
            set_blocks, all);
        k += G * F::kStageK;
#pragma unroll
        for (int n = 0; n < N; ++n) x[n] += 2 * G * F::kStageK;
        at = at + 1 == C::kStages ? 0 : at + 1;
      }
      // the sums of the unit before have been read
      if (done > 0 && !mbar_wait(empty, (done - 1) & 1, a.limit_ns, abort, a.status)) return false;
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < N; ++n)
          sums[(((2 * part + m) * NT + n) * G + group) * 32 + lane] =
              make_float4(acc[m][n][0], acc[m][n][1], acc[m][n][2], acc[m][n][3]);
      __syncwarp();
      if (lane == 0) mbar_arrive(full);
      return true;
    };
    if (!(NT == 1 || count <= 8 ? products(std::integral_constant<int, 1>{})
                                : products(std::integral_constant<int, NT>{})))
      break;
  }
  cp_async_wait_all();
}

// The output rows.  A cluster of `kCluster` blocks shares a unit of 32 rows: (expert, K) in runs over
// all of their warps.
template <int FORM, int NT>
struct OutCfg {
  static constexpr int kStage = Form<FORM>::kStage;
  static constexpr int kTokens = NT == 1 ? 8 : 32;
  static constexpr int kSums = (kWarps + 2) * kTokens * 32 * 4;   // of each warp, and twice the block's
  static constexpr int kStages = (232448 - kSums - static_cast<int>(sizeof(WeightedTable))) / (kWarps * kStage);
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kBytes = kRing + static_cast<int>(sizeof(WeightedTable)) + kSums;
  static_assert(kStages >= 2, "one stage in flight");
};

template <int FORM, int NT>
__global__ void __launch_bounds__(kThreads, 1) step_out_kernel(const StepArgs a, int cluster) {
  using C = OutCfg<FORM, NT>;
  using F = Form<FORM>;
  constexpr bool kPowers = !F::kBf16;
  extern __shared__ __align__(128) uint8_t smem[];
  WeightedTable& table = *reinterpret_cast<WeightedTable*>(smem + C::kRing);
  float* sums = reinterpret_cast<float*>(smem + C::kRing + sizeof(WeightedTable));   // [warp][token][32]
  const int T = static_cast<int>(a.T), values = T * 32;
  float* totals = sums + kWarps * values;                                  // [2][token][32]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rank = static_cast<int>(blockIdx.x) % cluster, clusters = static_cast<int>(gridDim.x) / cluster;
  float* own = sums + warp * values;
  for (int i = lane; i < values; i += 32) own[i] = 0.f;
  grid_dependency_wait();
  build_table(table, *reinterpret_cast<TableScratch*>(smem), a, 8 * NT);
  static_assert(sizeof(TableScratch) <= C::kRing, "the ring's place");

  const int K = static_cast<int>(a.F), bytes = row_bytes<FORM>(K), blocks = K / 32, powers_at = static_cast<int>(power_stride(K));
  const uint8_t* x0 = reinterpret_cast<const uint8_t*>(a.inner);
  const uint8_t* p0 = reinterpret_cast<const uint8_t*>(a.inner_power);
  const Scales all = {static_cast<const uint8_t*>(a.s_out) + static_cast<int64_t>(a.E) * a.H * blocks, blocks % 4 == 0};
  const int units = static_cast<int>((a.H + 31) / 32);
  const int stages = static_cast<int>((K + F::kStageK - 1) / F::kStageK);
  // the warp's run of (entry, stage)
  const int64_t items = static_cast<int64_t>(table.entries) * stages;
  const int runner = rank * kWarps + warp, runners = cluster * kWarps;
  const int64_t i0 = items * runner / runners, i1 = items * (runner + 1) / runners;
  const int entry0 = static_cast<int>(i0 / stages), stage0 = static_cast<int>(i0 % stages);
  const uint32_t ring = smem_u32(smem) + warp * C::kStages * C::kStage;
  // sets of rows: H % 8 == 0
  auto set_row = [&](int64_t row0, int r) { return row0 + 8 * r < a.H ? 8 * r : 0; };

  int lu = static_cast<int>(blockIdx.x) / cluster, slot = 0, le = entry0, ls = stage0;
  int64_t left = i1 - i0;
  Source src = {};
  Sets sets = {};
  auto rows_of = [&] {
    const int64_t row0 = static_cast<int64_t>(lu) * 32;
    const int64_t base = static_cast<int64_t>(table.expert[le]) * a.H + row0;
    src.row = static_cast<const uint8_t*>(a.w_out) + (base + g) * bytes + 16 * t;
#pragma unroll
    for (int r = 0; r < 4; ++r) sets.bytes[r] = set_row(row0, r) * bytes;
    if constexpr (F::kMx)
      src.scales = static_cast<const uint8_t*>(a.s_out) + (base + set_row(row0, lane >> 3) + (lane & 7)) * blocks;
  };
  if (i1 > i0 && lu < units) rows_of();
  auto load = [&] {
    if (i1 > i0 && lu < units) {
      load_stage<FORM>(ring + slot * C::kStage, src, sets, ls, bytes, all);
      bool moved = false;
      if (++ls == stages) ls = 0, ++le, moved = true;
      if (--left == 0) {
        left = i1 - i0;
        le = entry0, ls = stage0, moved = true;
        lu += clusters;
      }
      if (moved && lu < units) rows_of();
    }
    cp_async_commit();
    slot = slot + 1 == C::kStages ? 0 : slot + 1;
  };
#pragma unroll
  for (int i = 0; i < C::kStages - 1; ++i) load();

  int at = 0, turn = 0;
  for (int u = static_cast<int>(blockIdx.x) / cluster; u < units; u += clusters, turn ^= 1) {
    const int64_t row0 = static_cast<int64_t>(u) * 32;
    int entry = entry0, stage = stage0;
    int64_t todo = i1 - i0;
    while (todo > 0) {
      const int n_here = static_cast<int>(todo < stages - stage ? todo : stages - stage);
      const int first = table.first[entry], count = table.first[entry + 1] - first;
      const int64_t base = static_cast<int64_t>(table.expert[entry]) * a.H + row0;
      uint32_t scale_at = static_cast<uint32_t>((base + g) * blocks), set_blocks[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) set_blocks[r] = static_cast<uint32_t>(set_row(row0, r) * blocks);
      auto products = [&](auto n_cols) {
        constexpr int N = decltype(n_cols)::value;
        int k = stage * F::kStageK;
        uint32_t x[N], powers[N][2];   // (at most 2^27 bytes)
#pragma unroll
        for (int n = 0; n < N; ++n) {
          x[n] = 2 * (table.slot[first + min(8 * n + g, count - 1)] * K + k + 8 * t);
#pragma unroll
          for (int c = 0; c < 2; ++c)
            powers[n][c] = 4 * (table.slot[first + min(8 * n + 2 * t + c, count - 1)] * powers_at + k / 32);
        }
        float acc[2][N][4] = {};
        for (int i = 0; i < n_here; ++i) {
          stage_products<FORM, N, kPowers, C::kStages - 2>(
              acc, x0, x, p0, powers, K - k - 8 * t, ring + at * C::kStage, load, scale_at + k / 32,
              set_blocks, all);
          k += F::kStageK;
#pragma unroll
          for (int n = 0; n < N; ++n) {
            x[n] += 2 * F::kStageK;
            powers[n][0] += 4 * F::kBlocks;
            powers[n][1] += 4 * F::kBlocks;
          }
          at = at + 1 == C::kStages ? 0 : at + 1;
        }
        if constexpr (FORM == BSMMA_OPERAND_INT8) {
          const float* of = static_cast<const float*>(a.s_out) + base + g;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float s = of[set_row(row0, r)];
#pragma unroll
            for (int n = 0; n < N; ++n) {
              acc[r >> 1][n][2 * (r & 1)] *= s;
              acc[r >> 1][n][2 * (r & 1) + 1] *= s;
            }
          }
        }
        // an entry's columns are different tokens, so no two lanes add to one place
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int col = 8 * n + 2 * t + c;
            if (col < count) {
              const float w = table.weight[first + col];
              float* to = own + table.token[first + col] * 32 + g;
#pragma unroll
              for (int r = 0; r < 4; ++r) to[8 * r] = fmaf(w, acc[r >> 1][n][2 * (r & 1) + c], to[8 * r]);
            }
          }
      };
      if (NT == 1 || count <= 8) products(std::integral_constant<int, 1>{});
      else products(std::integral_constant<int, NT>{});
      __syncwarp();
      todo -= n_here;
      stage = 0;
      ++entry;
    }
    // the warps' sums, then (over the cluster) the blocks'; each block finishes its share of them
    __syncthreads();
    float* total = totals + turn * values;
    for (int i = threadIdx.x; i < values; i += kThreads) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        s += sums[w * values + i];
        sums[w * values + i] = 0.f;
      }
      total[i] = s;
    }
    if (cluster > 1) cluster_sync();
    else __syncthreads();
    for (int i = rank * kThreads + static_cast<int>(threadIdx.x); i < values; i += cluster * kThreads) {
      float s = 0.f;
      if (cluster > 1) {
        for (int b = 0; b < cluster; ++b) s += load_cluster(map_to_cta(smem_u32(total + i), b));
      } else {
        s = total[i];
      }
      if (row0 + (i & 31) < a.H) a.out[(i >> 5) * a.H + row0 + (i & 31)] = __float2bfloat16_rn(s);
    }
  }
  cp_async_wait_all();
  if (cluster > 1) cluster_sync();   // the others have read this block's sums
}

// How the work is cut goes by a GB300's room, SMs and clusters of 1, 2, 4 and 8 blocks that run at one
// time, as numbers: sizes and ids alone give the sums' order, and with it every bit, on a device with
// more or less of it too, which only takes the units in other waves.
constexpr int kRoom[4] = {152, 76, 36, 15};

// Blocks that share a unit of the third launch: as many as make its last wave fullest.
inline int cluster_shift(int64_t units) {
  int best = 0;
  double least = 0;
  for (int i = 0; i < 4; ++i) {
    const double waves = static_cast<double>((units + kRoom[i] - 1) / kRoom[i]) / (1 << i);
    if (i == 0 || waves < 0.95 * least) least = waves, best = i;
  }
  return best;
}

template <int FORM, int NT>
bsmma_status launch_out(const StepArgs& a, const DeviceInfo* dev, cudaStream_t stream) {
  using C = OutCfg<FORM, NT>;
  static PerDevice smem_set, fit[4];
  bsmma_status st = smem_set.allow_smem(dev->device, step_out_kernel<FORM, NT>, C::kBytes);
  if (st != BSMMA_OK) return st;
  const int64_t units = (a.H + 31) / 32;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {1, 1, 1};
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  const int shift = cluster_shift(units), shared = 1 << shift;
  int active = 0;   // clusters that run at one time here
  st = fit[shift].get(dev->device, &active, [&](int* v) {
    if (shared == 1) {
      *v = dev->sm_count;
      return BSMMA_OK;
    }
    cudaLaunchConfig_t q = cfg;
    q.gridDim = dim3(static_cast<unsigned>(shared));
    attr[1].val.clusterDim.x = static_cast<unsigned>(shared);
    q.attrs = attr + 1;
    q.numAttrs = 1;
    return cuda_ok(cudaOccupancyMaxActiveClusters(v, step_out_kernel<FORM, NT>, &q));
  });
  if (st != BSMMA_OK) return st;
  if (active < 1) return BSMMA_ERR_CUDA;
  attr[1].val.clusterDim.x = static_cast<unsigned>(shared);
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(units, active) * shared));
  cfg.numAttrs = 2;
  return cuda_ok(cudaLaunchKernelEx(&cfg, step_out_kernel<FORM, NT>, a, shared));
}

template <int FORM, int NT, int G>
bsmma_status launch_in(const StepArgs& a, const DeviceInfo* dev, cudaStream_t stream) {
  using C = InCfg<FORM, NT, G>;
  static PerDevice set;
  const bsmma_status st = set.allow_smem(dev->device, step_in_kernel<FORM, NT, G>, C::kBytes);
  if (st != BSMMA_OK) return st;
  // at most as many entries as slots
  const int64_t units = a.T * a.k * ((a.F + C::kTile - 1) / C::kTile);
  return cuda_ok(launch_dependent(step_in_kernel<FORM, NT, G>,
                                  dim3(static_cast<unsigned>(std::min<int64_t>(units, dev->sm_count))),
                                  dim3(C::kThreadsIn), C::kBytes, stream, a));
}

template <int FORM, int NT>
bsmma_status launch_step(StepArgs a, const DeviceInfo* dev, cudaStream_t stream) {
  a.limit_ns = wait_limit_ns();
  a.status = dev->status;
  if (FORM != BSMMA_OPERAND_BF16) {
    if (launch_dependent(step_tokens_kernel, dim3(static_cast<unsigned>(a.T)), dim3(kThreads), 0, stream, a) !=
        cudaSuccess)
      return BSMMA_ERR_CUDA;
    count_launches(1);
  }
  // K over eight groups of warps where that leaves each three stages of a unit or more; short rows over
  // two, in units of four times the columns (what a unit costs beside its stages, and the groups' unequal
  // shares: 29 tokens, 8 of 63 experts of 8640 x 544 in E5M2 494 and 369 us; 18 tokens, 7 of 14 experts of
  // 4720 x 432 in INT8 72 and 60), as long as those are two for an SM or more: no more experts than E or
  // slots are chosen.  (Longer rows in wide units: 32 tokens of INT8 experts of 2048 x 7168 500 and 535 us, 8
  // of E2M1 experts of 14336 x 4096 199 and 222.)
  using F = Form<FORM>;
  const int64_t stages = (a.H + F::kStageK - 1) / F::kStageK;
  const int64_t wide_units = std::min<int64_t>(a.E, a.T * a.k) * ((a.F + 127) / 128);
  bsmma_status st = stages < 24 && wide_units >= 2 * kRoom[0] ? launch_in<FORM, NT, 2>(a, dev, stream)
                                                              : launch_in<FORM, NT, 8>(a, dev, stream);
  if (st == BSMMA_OK) st = launch_out<FORM, NT>(a, dev, stream);
  count_launches(2);
  return st;
}

template <int FORM>
bsmma_status launch_step_form(const StepArgs& a, const DeviceInfo* dev, cudaStream_t stream) {
  // an expert's columns are at most the tokens
  return a.T <= 8 ? launch_step<FORM, 1>(a, dev, stream) : launch_step<FORM, 2>(a, dev, stream);
}

constexpr int64_t round_up(int64_t n) { return (n + 255) / 256 * 256; }

}  // namespace

int64_t step_workspace_bytes(int64_t T, int k, int64_t H, int64_t F) {
  return round_up(T * 4) + round_up(T * H * 2) + round_up(T * k * power_stride(F) * 4) +
         round_up(T * k * F * 2);
}

bsmma_status launch_moe_step(StepArgs a, int form, void* workspace, cudaStream_t stream) {
  bsmma_status st;
  const DeviceInfo* dev = current_device(&st);
  if (!dev) return st;
  uint8_t* p = static_cast<uint8_t*>(workspace);
  auto take = [&](int64_t n) {
    uint8_t* q = p;
    p += round_up(n);
    return q;
  };
  a.x_power = reinterpret_cast<float*>(take(a.T * 4));
  a.x16 = reinterpret_cast<uint16_t*>(take(a.T * a.H * 2));
  a.inner_power = reinterpret_cast<float*>(take(a.T * a.k * power_stride(a.F) * 4));
  a.inner = reinterpret_cast<uint16_t*>(take(a.T * a.k * a.F * 2));
  switch (form) {
    case BSMMA_OPERAND_BF16: return launch_step_form<BSMMA_OPERAND_BF16>(a, dev, stream);
    case BSMMA_OPERAND_INT8: return launch_step_form<BSMMA_OPERAND_INT8>(a, dev, stream);
    case BSMMA_OPERAND_E4M3: return launch_step_form<BSMMA_OPERAND_E4M3>(a, dev, stream);
    case BSMMA_OPERAND_E5M2: return launch_step_form<BSMMA_OPERAND_E5M2>(a, dev, stream);
    default: return launch_step_form<BSMMA_OPERAND_E2M1>(a, dev, stream);
  }
}

}  // namespace bsmma
