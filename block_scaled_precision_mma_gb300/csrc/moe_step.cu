// moe_step.cu -- the experts and the weighted sum of a few tokens, in two launches.
//
// What bounds it is reading the chosen experts' weights once, so both kernels are built around
// keeping their bytes in flight: one block of 16 warps an SM, each warp with a ring of
// asynchronous copies of its own that runs on from one unit of work to the next.  A lane reads
// back what it copied itself, so the ring needs no barrier, and since both operands of a product
// may take K in any order, a lane's 16 bytes of a weight row and the same K of a token go into
// the matrix instruction as they are.
//
// The products use mma.sync with the weights as the 16-row operand and up to 8 * NT tokens as
// columns: with a row or a few an expert the tensor cores wait for memory whatever their
// instruction, and the few-row form needs no tile of tokens in shared memory.  Weights are widened
// to BF16 in registers, exactly: INT8 codes are BF16 values, and an MX code's bits, moved into
// BF16's fields, are the code times a power of two, which one multiplication by another takes
// to the scaled value.  Sums are FP32.
//
// First launch: units of 16 inner columns (16 rows of Wg and the 16 of Wu) of one expert; the
// warps share out K, their sums meet in shared memory, and the inner row leaves in BF16.  Gate and
// up rows are put into the upper and lower half of the same 16-row operand, so that the lane
// that has a gate's sum has its up's too.  Second launch: units of 16 output columns over all
// chosen experts, the warps sharing out (expert, K) in runs; a warp adds an expert's columns, times
// their tokens' weights, to its tokens' sums, and the warps' sums are added in order.  It starts
// under the first one (programmatic launch) and has its ring full when the inner rows are done.
#include <algorithm>

#include "epilogue.cuh"
#include "moe_step.h"
#include "ptx.cuh"

namespace bsmma {
namespace {

constexpr uint32_t kFull = 0xFFFFFFFFu;
constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int kMaxSlots = 1024, kMaxExperts = 1024;

// ------------------------------------------------------------------------- weights
// How a form's codes lie in a lane's 16 bytes, by granules of eight consecutive K.
template <int FORM>
struct Form {
  static constexpr bool kMx = FORM >= BSMMA_OPERAND_E4M3;
  static constexpr int kGranules = FORM == BSMMA_OPERAND_BF16 ? 1 : FORM == BSMMA_OPERAND_E2M1 ? 4 : 2;
  static constexpr int kLaneK = 8 * kGranules;     // K of a lane's 16 bytes
  static constexpr int kPieceK = 4 * kLaneK;       // of the four lanes that share a row
  // a scaled value is its code's bits in BF16's fields times 2^(scale + this - 127) (as a
  // BF16 exponent field: scale + this)
  static constexpr int kField = FORM == BSMMA_OPERAND_E4M3 ? 120 : FORM == BSMMA_OPERAND_E5M2 ? 112 : 126;
};

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// The multiplier(s) of a block's E8M0 scale, twice in a word.  A scale too large for one
// multiplier (2^8 and more for E4M3) takes a second; 255 is NaN.
struct MxScale {
  uint32_t first, second;   // second 0: one multiplier
};
template <int FORM>
__device__ __forceinline__ MxScale mx_scale(uint32_t code) {
  MxScale m;
  const uint32_t field = code + Form<FORM>::kField;
  m.first = field << 7;
  m.second = 0;
  if (field > 254) {
    m.first = static_cast<uint32_t>(Form<FORM>::kField + 127) << 7;
    m.second = code == 255 ? 0x7FC07FC0u : code << 7 | code << 23;
  }
  m.first |= m.first << 16;
  return m;
}

// Granule q of a lane's 16 bytes as four pairs of BF16 values.
template <int FORM>
__device__ __forceinline__ void decode(const uint4& w, int q, const MxScale& s, uint32_t (&o)[4]) {
  if constexpr (FORM == BSMMA_OPERAND_BF16) {
    o[0] = w.x, o[1] = w.y, o[2] = w.z, o[3] = w.w;
  } else if constexpr (FORM == BSMMA_OPERAND_INT8) {
    const uint32_t c[2] = {q ? w.z : w.x, q ? w.w : w.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // 0x43 above a code's byte: its low seven bits are 128 + those, its sign 128 or 256, and the
      // difference is the code
      const uint32_t v = __byte_perm(c[i >> 1], 0x43434343u, i & 1 ? 0x4342 : 0x4140);
      o[i] = sub_bf16x2(v & 0xFF7FFF7Fu, v & 0xFF80FF80u);
    }
  } else if constexpr (FORM == BSMMA_OPERAND_E2M1) {
    const uint32_t c = q == 0 ? w.x : q == 1 ? w.y : q == 2 ? w.z : w.w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {   // K i and i + 4 of the granule
      const uint32_t t = c >> (4 * i);
      o[i] = (t & 0x00070007u) << 6 | (t & 0x00080008u) << 12;
    }
  } else {
    constexpr int kShift = FORM == BSMMA_OPERAND_E4M3 ? 4 : 3;
    constexpr uint32_t kBits = 0x7F007F00u >> kShift;
    const uint32_t c[2] = {q ? w.z : w.x, q ? w.w : w.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t v = __byte_perm(c[i >> 1], 0u, i & 1 ? 0x3424 : 0x1404);
      o[i] = (v >> kShift & kBits) | (v & 0x80008000u);
    }
  }
  if constexpr (Form<FORM>::kMx) {
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = mul_bf16x2(o[i], s.first);
    if (s.second)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = mul_bf16x2(o[i], s.second);
  }
}
// A token's granule in the order of decode()'s pairs.
template <int FORM>
__device__ __forceinline__ void order_token(uint4& x) {
  if constexpr (FORM == BSMMA_OPERAND_E2M1)
    x = make_uint4(__byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632),
                   __byte_perm(x.y, x.w, 0x5410), __byte_perm(x.y, x.w, 0x7632));
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t a0, const uint32_t a1,
                                         const uint32_t a2, const uint32_t a3, const uint32_t b0,
                                         const uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

// ------------------------------------------------------------------------- who takes what
// The chosen experts in order, each with its columns (tokens) in tiles of `tile`.  A token that
// names an expert twice is one column with both weights.
struct Table {
  int entries;
  uint16_t expert[kMaxSlots];       // of each tile
  uint16_t first[kMaxSlots];        // its first column
  uint16_t count[kMaxSlots];
  uint16_t slot[kMaxSlots];         // of each column (token * k + choice)
  float weight[kMaxSlots];
};
struct TableScratch {
  int start[kMaxExperts];           // counts, then first columns
  int32_t ids[kMaxSlots];
  uint16_t rank[kMaxSlots];
};
constexpr uint16_t kNone = 0xFFFF;

__device__ __forceinline__ void build_table(Table& t, TableScratch& s, const StepArgs& a, int tile) {
  const int tid = threadIdx.x, lane = tid & 31, slots = static_cast<int>(a.T) * a.k;
  for (int e = tid; e < a.E; e += kThreads) s.start[e] = 0;
  for (int i = tid; i < slots; i += kThreads) {
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
        t.count[t0 + i] = static_cast<uint16_t>(min(tile, n - i * tile));
      }
      column += __shfl_sync(kFull, in, 31);
      entry += __shfl_sync(kFull, it, 31);
    }
    if (lane == 0) t.entries = entry;
  }
  __syncthreads();
  for (int i = tid; i < slots; i += kThreads) {
    if (s.rank[i] == kNone) continue;
    const int id = s.ids[i], c = s.start[id] + s.rank[i];
    float w = a.weights[i];
    for (int j = i + 1; j % a.k; ++j)
      if (s.ids[j] == id) w += a.weights[j];
    t.slot[c] = static_cast<uint16_t>(i);
    t.weight[c] = w;
  }
  __syncthreads();
}

// ------------------------------------------------------------------------- products
// A lane's share of one stage: PIECES * 16 bytes of each of ROWS rows, 512 bytes a piece and warp.
constexpr int kPieces = 2;
template <int ROWS>
constexpr int kStageBytes = ROWS * kPieces * 512;

// Multiplies a stage's weights into acc.  MT operands of 16 rows: operand m has rows
// 2 m (upper half, lane's row g) and 2 m + 1 (lower half) of the stage's ROWS = 2 * MT.
// x: rows of the columns (a lane's column of each 8), or nullptr; k: the lane's first K.
template <int FORM, int MT, int NT>
__device__ __forceinline__ void multiply(float (&acc)[MT][NT][4], uint32_t ring,
                                         const __nv_bfloat16* const (&x)[NT], int nt_used, int64_t k,
                                         int64_t K, const uint8_t* const (&scale)[2 * MT]) {
  using F = Form<FORM>;
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {
    const int64_t kp = k + p * F::kPieceK;
    const bool in = kp < K;
    MxScale s[2 * MT] = {};
    if constexpr (F::kMx) {
#pragma unroll
      for (int r = 0; r < 2 * MT; ++r) s[r] = mx_scale<FORM>(in && scale[r] ? scale[r][kp >> 5] : 127u);
    }
    uint4 w[2 * MT];
#pragma unroll
    for (int r = 0; r < 2 * MT; ++r) w[r] = lds16(ring + (r * kPieces + p) * 512);
#pragma unroll
    for (int q = 0; q < F::kGranules; ++q) {
      uint4 b[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        b[n] = make_uint4(0, 0, 0, 0);
        if (in && x[n]) b[n] = *reinterpret_cast<const uint4*>(x[n] + kp + 8 * q);
        order_token<FORM>(b[n]);
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        uint32_t hi[4], lo[4];
        decode<FORM>(w[2 * m], q, s[2 * m], hi);
        decode<FORM>(w[2 * m + 1], q, s[2 * m + 1], lo);
#pragma unroll
        for (int n = 0; n < NT; ++n)
          if (n < nt_used) {
            mma_bf16(acc[m][n], hi[0], lo[0], hi[1], lo[1], b[n].x, b[n].y);
            mma_bf16(acc[m][n], hi[2], lo[2], hi[3], lo[3], b[n].z, b[n].w);
          }
      }
    }
  }
}

__device__ __forceinline__ float activate(float x, int act) {
  if (act == BSMMA_ACT_RELU) return x < 0.f ? 0.f : x;
  if (act == BSMMA_ACT_GELU) return gelu_erf(x);
  return act == BSMMA_ACT_SILU ? x / (1.f + expf(-x)) : x;
}

// Bytes of a row of K codes.
template <int FORM>
__device__ __forceinline__ int64_t row_bytes(int64_t K) {
  return FORM == BSMMA_OPERAND_BF16 ? 2 * K : FORM == BSMMA_OPERAND_E2M1 ? K / 2 : K;
}

// The inner rows: [slot][F] BF16.
template <int FORM, int NT>
struct InCfg {
  static constexpr int kStage = kStageBytes<4>;
  static constexpr int kStages = NT == 1 ? 3 : 2;
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kSums = kWarps * 2 * NT * 512;
  static constexpr int kBytes = kRing + kSums + static_cast<int>(sizeof(Table));
  static_assert(sizeof(TableScratch) <= kRing && kBytes <= 232448, "shared memory budget");
};

template <int FORM, int NT>
__global__ void __launch_bounds__(kThreads, 1) step_in_kernel(const StepArgs a) {
  using C = InCfg<FORM, NT>;
  using F = Form<FORM>;
  extern __shared__ __align__(128) uint8_t smem[];
  float4* sums = reinterpret_cast<float4*>(smem + C::kRing);
  Table& table = *reinterpret_cast<Table*>(smem + C::kRing + C::kSums);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  grid_dependency_wait();
  grid_launch_dependents();
  build_table(table, *reinterpret_cast<TableScratch*>(smem), a, 8 * NT);

  const int64_t K = a.H, bytes = row_bytes<FORM>(K);
  const int tiles = static_cast<int>((a.F + 15) / 16), units = table.entries * tiles;
  const int stages = static_cast<int>((K + kPieces * F::kPieceK - 1) / (kPieces * F::kPieceK));
  const int mine = warp < stages ? (stages - warp + kWarps - 1) / kWarps : 0;   // of a unit
  const uint32_t ring = smem_u32(smem) + warp * C::kStages * C::kStage + lane * 16;
  // row r (0, 2: gate, 1, 3: up) of a unit: its number in the expert, or -1
  auto row_of = [&](int u, int r) -> int64_t {
    const int64_t f = static_cast<int64_t>(u % tiles) * 16 + 8 * (r >> 1) + g;
    return f < a.F ? (r & 1 ? a.F + f : f) : -1;
  };
  // the loads run ahead of the products through the block's units
  int lu = blockIdx.x, li = 0, slot = 0;
  const uint8_t* src[4];
  auto enter_unit = [&] {
    if (lu >= units) return;
    const int64_t e = table.expert[lu / tiles];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int64_t row = row_of(lu, r);
      src[r] = row < 0 ? nullptr : static_cast<const uint8_t*>(a.w_in) + (e * 2 * a.F + row) * bytes;
    }
  };
  auto load = [&] {
    if (mine && lu < units) {
      const int64_t at = static_cast<int64_t>(warp + li * kWarps) * (kPieces * 64) + t * 16;
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
          const bool in = src[r] && at + 64 * p < bytes;
          cp_async_16(ring + slot * C::kStage + (r * kPieces + p) * 512,
                      in ? src[r] + at + 64 * p : static_cast<const uint8_t*>(a.w_in), in);
        }
      if (++li == mine) {
        li = 0;
        lu += gridDim.x;
        enter_unit();
      }
    }
    cp_async_commit();
    slot = slot + 1 == C::kStages ? 0 : slot + 1;
  };
  enter_unit();
#pragma unroll
  for (int i = 0; i < C::kStages - 1; ++i) load();

  int at = 0;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const int entry = u / tiles, first = table.first[entry], count = table.count[entry];
    const int nt_used = (count + 7) / 8;
    const __nv_bfloat16* x[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
      x[n] = 8 * n + g < count
                 ? static_cast<const __nv_bfloat16*>(a.x) + table.slot[first + 8 * n + g] / a.k * a.H
                 : nullptr;
    const uint8_t* scale[4] = {};
    if constexpr (F::kMx) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int64_t row = row_of(u, r);
        if (row >= 0)
          scale[r] = static_cast<const uint8_t*>(a.s_in) + (table.expert[entry] * 2 * a.F + row) * (K / 32);
      }
    }
    float acc[2][NT][4] = {};
    for (int i = 0; i < mine; ++i) {
      load();
      cp_async_wait<C::kStages - 1>();
      multiply<FORM, 2, NT>(acc, ring + at * C::kStage, x, nt_used,
                            static_cast<int64_t>(warp + i * kWarps) * (kPieces * F::kPieceK) + t * F::kLaneK,
                            K, scale);
      at = at + 1 == C::kStages ? 0 : at + 1;
    }
    __syncthreads();   // the sums of the unit before have been read
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
        if (n < nt_used)
          sums[((m * NT + n) * kWarps + warp) * 32 + lane] =
              make_float4(acc[m][n][0], acc[m][n][1], acc[m][n][2], acc[m][n][3]);
    __syncthreads();
    // a warp an operand and eight columns
    for (int j = warp; j < 2 * NT; j += kWarps) {
      const int m = j / NT, n = j % NT;
      if (n >= nt_used) continue;
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 v = sums[(j * kWarps + w) * 32 + lane];
        s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
      }
      const int64_t f = static_cast<int64_t>(u % tiles) * 16 + 8 * m + g;
      if (f >= a.F) continue;
      if constexpr (FORM == BSMMA_OPERAND_INT8) {
        const float* of = static_cast<const float*>(a.s_in) + table.expert[entry] * 2 * a.F;
        const float sg = of[f], su = of[a.F + f];
        s.x *= sg, s.y *= sg, s.z *= su, s.w *= su;
      }
      const float v[2] = {activate(s.x, a.act) * s.z, activate(s.y, a.act) * s.w};
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (8 * n + 2 * t + c < count)
          a.inner[table.slot[first + 8 * n + 2 * t + c] * a.F + f] = __float2bfloat16_rn(v[c]);
    }
  }
  cp_async_wait_all();
}

// The output rows.
template <int FORM, int NT>
struct OutCfg {
  static constexpr int kStage = kStageBytes<2>;
  static constexpr int kStages = 4;
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kFixed = kRing + static_cast<int>(sizeof(Table));
  static int bytes(int64_t T) { return kFixed + kWarps * static_cast<int>(T) * 16 * 4; }
  static_assert(sizeof(TableScratch) <= kRing && kFixed + kWarps * 64 * 64 <= 232448, "shared memory budget");
};

template <int FORM, int NT>
__global__ void __launch_bounds__(kThreads, 1) step_out_kernel(const StepArgs a) {
  using C = OutCfg<FORM, NT>;
  using F = Form<FORM>;
  extern __shared__ __align__(128) uint8_t smem[];
  Table& table = *reinterpret_cast<Table*>(smem + C::kRing);
  float* sums = reinterpret_cast<float*>(smem + C::kFixed);   // [warp][token][16]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int T = static_cast<int>(a.T);
  // ids, weights and w_out were there before the first launch began (it waited for what was
  // before it); only the inner rows are waited for
  build_table(table, *reinterpret_cast<TableScratch*>(smem), a, 8 * NT);
  float* own = sums + warp * T * 16;
  for (int i = lane; i < T * 16; i += 32) own[i] = 0.f;
  __syncwarp();

  const int64_t K = a.F, bytes = row_bytes<FORM>(K);
  const int units = static_cast<int>((a.H + 15) / 16);
  const int stages = static_cast<int>((K + kPieces * F::kPieceK - 1) / (kPieces * F::kPieceK));
  // the warp's run of (entry, stage)
  const int64_t items = static_cast<int64_t>(table.entries) * stages;
  const int64_t i0 = items * warp / kWarps, i1 = items * (warp + 1) / kWarps;
  const int entry0 = static_cast<int>(i0 / stages), stage0 = static_cast<int>(i0 % stages);
  const uint32_t ring = smem_u32(smem) + warp * C::kStages * C::kStage + lane * 16;

  int lu = blockIdx.x, slot = 0, le = entry0, ls = stage0;
  int64_t left = i1 - i0;
  const uint8_t* src[2];
  auto rows_of = [&] {
    const int64_t e = table.expert[le];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int64_t row = static_cast<int64_t>(lu) * 16 + 8 * r + g;
      src[r] = row < a.H ? static_cast<const uint8_t*>(a.w_out) + (e * a.H + row) * bytes : nullptr;
    }
  };
  if (i1 > i0) rows_of();
  auto load = [&] {
    if (i1 > i0 && lu < units) {
      const int64_t at = static_cast<int64_t>(ls) * (kPieces * 64) + t * 16;
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
          const bool in = src[r] && at + 64 * p < bytes;
          cp_async_16(ring + slot * C::kStage + (r * kPieces + p) * 512,
                      in ? src[r] + at + 64 * p : static_cast<const uint8_t*>(a.w_out), in);
        }
      bool moved = false;
      if (++ls == stages) ls = 0, ++le, moved = true;
      if (--left == 0) {
        left = i1 - i0;
        le = entry0, ls = stage0, moved = true;
        lu += gridDim.x;
      }
      if (moved && lu < units) rows_of();
    }
    cp_async_commit();
    slot = slot + 1 == C::kStages ? 0 : slot + 1;
  };
#pragma unroll
  for (int i = 0; i < C::kStages - 1; ++i) load();
  grid_dependency_wait();

  int at = 0;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t row0 = static_cast<int64_t>(u) * 16;
    int entry = entry0, stage = stage0;
    int64_t todo = i1 - i0;
    while (todo > 0) {
      const int n_here = static_cast<int>(todo < stages - stage ? todo : stages - stage);
      const int first = table.first[entry], count = table.count[entry], nt_used = (count + 7) / 8;
      const int64_t e = table.expert[entry];
      const __nv_bfloat16* x[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n)
        x[n] = 8 * n + g < count ? a.inner + table.slot[first + 8 * n + g] * a.F : nullptr;
      const uint8_t* scale[2] = {};
      if constexpr (F::kMx) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
          if (row0 + 8 * r + g < a.H)
            scale[r] = static_cast<const uint8_t*>(a.s_out) + (e * a.H + row0 + 8 * r + g) * (K / 32);
      }
      float acc[1][NT][4] = {};
      for (int i = 0; i < n_here; ++i) {
        load();
        cp_async_wait<C::kStages - 1>();
        multiply<FORM, 1, NT>(acc, ring + at * C::kStage, x, nt_used,
                              static_cast<int64_t>(stage + i) * (kPieces * F::kPieceK) + t * F::kLaneK, K,
                              scale);
        at = at + 1 == C::kStages ? 0 : at + 1;
      }
      float rs[2] = {1.f, 1.f};
      if constexpr (FORM == BSMMA_OPERAND_INT8) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
          if (row0 + 8 * r + g < a.H) rs[r] = static_cast<const float*>(a.s_out)[e * a.H + row0 + 8 * r + g];
      }
      // an entry's columns are different tokens, so no two lanes add to one place
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int col = 8 * n + 2 * t + c;
          if (col < count) {
            const float w = table.weight[first + col];
            float* to = own + table.slot[first + col] / a.k * 16 + g;
            to[0] = fmaf(w, acc[0][n][c] * rs[0], to[0]);
            to[8] = fmaf(w, acc[0][n][2 + c] * rs[1], to[8]);
          }
        }
      __syncwarp();
      todo -= n_here;
      stage = 0;
      ++entry;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < T * 16; i += kThreads) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        s += sums[w * T * 16 + i];
        sums[w * T * 16 + i] = 0.f;
      }
      if (row0 + (i & 15) < a.H) a.out[(i >> 4) * a.H + row0 + (i & 15)] = __float2bfloat16_rn(s);
    }
    __syncthreads();
  }
  cp_async_wait_all();
}

template <int FORM, int NT>
bsmma_status launch_step(const StepArgs& a, const DeviceInfo* dev, cudaStream_t stream) {
  static PerDevice in_set, out_set;
  constexpr int kIn = InCfg<FORM, NT>::kBytes, kOut = OutCfg<FORM, NT>::kFixed + kWarps * 64 * 64;
  bsmma_status st = in_set.allow_smem(dev->device, step_in_kernel<FORM, NT>, kIn);
  if (st == BSMMA_OK) st = out_set.allow_smem(dev->device, step_out_kernel<FORM, NT>, kOut);
  if (st != BSMMA_OK) return st;
  const int64_t slots = a.T * a.k;   // at most this many entries
  const int64_t in_units = slots * ((a.F + 15) / 16), out_units = (a.H + 15) / 16;
  const unsigned in_blocks = static_cast<unsigned>(std::min<int64_t>(in_units, dev->sm_count));
  const unsigned out_blocks = static_cast<unsigned>(std::min<int64_t>(out_units, dev->sm_count));
  cudaError_t e = launch_dependent(step_in_kernel<FORM, NT>, dim3(in_blocks), dim3(kThreads), kIn, stream, a);
  count_launches(1);
  if (e != cudaSuccess) return BSMMA_ERR_CUDA;
  e = launch_dependent(step_out_kernel<FORM, NT>, dim3(out_blocks), dim3(kThreads),
                       OutCfg<FORM, NT>::bytes(a.T), stream, a);
  count_launches(1);
  return cuda_ok(e);
}

template <int FORM>
bsmma_status launch_step_form(const StepArgs& a, const DeviceInfo* dev, cudaStream_t stream) {
  // an expert's columns are at most the tokens: tiles no wider than those
  if (a.T <= 8) return launch_step<FORM, 1>(a, dev, stream);
  if (a.T <= 16) return launch_step<FORM, 2>(a, dev, stream);
  return launch_step<FORM, 4>(a, dev, stream);
}

}  // namespace

bsmma_status launch_moe_step(const StepArgs& a, int form, cudaStream_t stream) {
  bsmma_status st;
  const DeviceInfo* dev = current_device(&st);
  if (!dev) return st;
  switch (form) {
    case BSMMA_OPERAND_BF16: return launch_step_form<BSMMA_OPERAND_BF16>(a, dev, stream);
    case BSMMA_OPERAND_INT8: return launch_step_form<BSMMA_OPERAND_INT8>(a, dev, stream);
    case BSMMA_OPERAND_E4M3: return launch_step_form<BSMMA_OPERAND_E4M3>(a, dev, stream);
    case BSMMA_OPERAND_E5M2: return launch_step_form<BSMMA_OPERAND_E5M2>(a, dev, stream);
    default: return launch_step_form<BSMMA_OPERAND_E2M1>(a, dev, stream);
  }
}

}  // namespace bsmma
