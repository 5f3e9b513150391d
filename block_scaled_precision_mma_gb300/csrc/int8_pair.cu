// int8_pair.cu -- INT8 products on SM pairs: the tensor-core kernel of int8_gemm and
// grouped_int8_gemm for more rows than the few-row kernel takes.
//
// The accumulator holds D transposed: its rows are 256 channels (128 a CTA), its columns up
// to TN rows of A ("tokens").  Both operands arrive as INT8 by TMA and are widened to FP16
// on the SM, where they are exact: the channels' values go from registers into tensor
// memory, the A operand of tcgen05.mma, and the tokens' into shared memory, its B operand.
// So DRAM and L2 carry one byte a value, and the channels' widened values never cross shared
// memory, which the MMAs' own reads of the tokens fill (an FP16 tile by TMA would write and
// read two bytes each).
//
// What bounds it, as measured (graph replays, L2 flushed, each after a pause): many rows the
// tensor pipe, 4096 x 14336 x 4096 268 us with the widening pass, 1.80 PFLOP/s, and 8 experts of
// 7168 x 2304 with 16384 rows 322 us, 1.68 PFLOP/s (tensor pipe 76% busy under ncu at the clock it
// holds there; one after another the power cap makes them 285 and 340 us); few rows the streaming
// of the channels, 64 experts of 2048 x 7168 with 256 rows between them 131 us for 738 MB, 5.6
// TB/s; in between (192 rows an expert) the widening warps' latencies, tensor pipe and DRAM both
// near half.  A single short product is launch, setup and pipeline start: 4 x 14336 x 4096 takes
// 23 us, of which its bytes are 9 (the few-row kernel, which gets it, 17 us).
//
// One persistent launch over 2-CTA clusters, 512 threads a CTA:
//   warp 0       TMA producer: 128 K of the CTA's 128 channels and of its half of the tokens
//                (one box for a full half, else boxes of 32 and 8 rows) into a ring;
//   warp 1       in the leader, issues the M = 256 FP16 MMAs, eight per stage;
//   warps 4-11   two widening warpgroups, stages in turn: a thread widens one channel's 128
//                values into its tensor-memory lane and its share of the tokens into the
//                128-byte-swizzled shared-memory tile (with PRE the tokens come as FP16, by
//                warp 2);
//   warps 12-15  output: accumulator columns out of tensor memory, times the scales, plus
//                the bias, rounded, turned through shared memory and stored by rows of D.
// Units (a token block of one group x 256 channels) are dealt round robin; the last wave's
// are split along K over the pairs that would idle (stream_k.cuh), the partial sums added in
// K order by the last pair to finish.
#include <cuda.h>
#include <cuda_runtime.h>

#include <optional>
#include <type_traits>

#include "int8.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "stream_k.cuh"

namespace bsmma {
namespace int8 {
namespace {

constexpr uint32_t kFull = 0xFFFFFFFFu;
constexpr int kThreads = 512;
constexpr int kWideWarp0 = 4, kOutWarp0 = 12;
constexpr int kSlotCols = 64;                 // tensor-memory columns of a slot's 128 FP16 values
constexpr uint16_t kPairMask = 3;
constexpr int kOutBarrier = 1;                // named barriers: the output warps,
constexpr int kFixBarrier = 2;                // the output and widening warps (3-5: each warpgroup)
constexpr int kSetupBarrier = 6;              // all but the channel producer
constexpr uint32_t kNone = 0xFFFFFFFFu;

struct Table {
  GroupTable<kThreads> groups;
  int fixes, fix[2];           // split units whose parts this CTA adds (two at most)
};

// PRE: the tokens are FP16 already (a widening pass before the launch).
template <int TN, bool PRE, bool F32>
struct Cfg {
  static constexpr int kHalf = TN / 2;                        // tokens of a CTA
  // a stage: 128 K in INT8, of the channels alone with PRE
  static constexpr int kRawBytes = 128 * 128 + (PRE ? 0 : kHalf * 128);
  static constexpr int kWideBytes = kHalf * 256;              // a slot: 128 K of the tokens in FP16
  // accumulators, and slots of widened channels in the rest of tensor memory
  static constexpr int kBufs = 2 * TN + 2 * kSlotCols <= 512 ? 2 : 1;
  static constexpr int kFree = (512 - kBufs * TN) / kSlotCols;
  static constexpr int kSlots = kFree < 4 ? kFree : 4;
  // slots of tokens in shared memory: two without PRE, half as many as of channels, so that a
  // stage's channels are stored without a wait while the tokens' slot is still being read (64
  // experts of 2048 x 7168: 192 rows 266 -> 257 us, 256 rows in tiles of 128 383 -> 346)
  static constexpr int kTokSlots = PRE ? (TN > 192 ? (F32 ? 3 : 4) : 5) : 2;
  static constexpr int kOutRow = F32 ? 512 + 16 : 256 + 64;   // output tile: 32 tokens x 128 channels
  static constexpr int kOutBytes = 32 * kOutRow;
  static constexpr int kOutTiles = F32 && TN > 192 && !PRE ? 1 : 2;   // one: room for a fourth stage
  static constexpr int kTail = 1024 + static_cast<int>(sizeof(Table)) + 512 + kOutTiles * kOutBytes;
  static constexpr int kFit = (232448 - kTail - kTokSlots * kWideBytes) / kRawBytes;
  // a widening warpgroup waits for the MMAs of as many stages before its own
  static constexpr int kBehind = PRE ? kSlots : kTokSlots;
  static constexpr int kMost = kFit > 12 ? 12 : kFit;
  // With an odd number of stages a stage goes back and forth between the two widening
  // warpgroups, and each of them waits for every second load of it.  A wait by parity takes the
  // load two before for the awaited one while the load between them is still under way, so that
  // one must be known to have come: it is stage i - kStages when the warpgroup waits for stage
  // i, and the slot of the warpgroup's last stage, i - 2, was freed by the MMAs of stage
  // i - 2 - kBehind, which follow those of every stage before.
  static constexpr int kStages = kMost % 2 == 0 || kMost >= kBehind + 2 ? kMost : kMost - 1;
  static constexpr int kSmemBytes = kTail + kTokSlots * kWideBytes + kStages * kRawBytes;
  static_assert((2 * kStages + 2 * kSlots + 5 + (PRE ? 2 * kTokSlots : 0)) * 8 + 8 <= 512,
                "barriers fit below the group table");
  static_assert(kStages >= 4 && (kStages % 2 == 0 || kStages >= kBehind + 2), "a wait cannot be a load behind");
  static_assert(kSlots % 2 == 0 && (PRE || (kSlots == 4 && kTokSlots == 2)) && 2 * kOutTiles * kOutBytes <= kStages * kRawBytes + kTokSlots * kWideBytes,
                "shared memory budget");
  static_assert(kBufs * TN + kSlots * kSlotCols <= 512, "tensor memory budget");
};

struct PairParams {
  Int8Params a;
  int tn, num_n_tiles, stages_k, halves_k;
  float* part;
  int* arrivals;
  uint64_t limit_ns;
};

// The library's bounded wait (mbar_wait) with a suspend hint: a waiting warp stays off the
// shared-memory pipe until the phase completes or 20 us have passed.  Without it a dozen
// polling warps a CTA slow the widening warps' loads (64 experts x 2048 x 7168, 256 rows:
// 152 us without, 144 us with).  CLUSTER: the peer CTA arrives on the barrier as well.
template <bool CLUSTER>
__device__ __forceinline__ bool try_wait_hint(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  if constexpr (CLUSTER)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(20000)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(20000)
        : "memory");
  return ok != 0;
}
template <bool CLUSTER = false>
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, uint64_t limit_ns,
                                           volatile int* abort, int* status) {
  if (try_wait_hint<CLUSTER>(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!try_wait_hint<CLUSTER>(bar, parity)) {
    if (*abort) return false;
    if (globaltimer_ns() - t0 > limit_ns) {
      report_status(status, kDevTimeout);
      *abort = 1;
      return false;
    }
  }
  return true;
}

// Arrives on the leader's barrier, releasing at CTA scope: what it announces (values in this
// CTA's shared and tensor memory, or accumulator columns read) concerns this CTA's own tensor
// core.  Release at cluster scope waits for every earlier store of the warp to be visible to
// the cluster: 800 to 1100 cycles a slot for the widening warps, and all of a tile's output
// stores for the output warps (4096 x 14336 x 4096 at that time: 605 us with it, 486 without).
__device__ __forceinline__ void arrive_leader(uint32_t bar_cluster) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}

// D(tmem) (+)= A(tmem) x B(smem) over the pair, FP16 operands, FP32 accumulation.
__device__ __forceinline__ void mma_f16_pair_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                                uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// True in one lane of the (whole) warp, the same one every time.  A role that issues copies or
// MMAs runs its loop on all lanes and elects the issuing one at the instruction, so that loop
// state and descriptors are warp-uniform for the compiler; under a divergent `lane == 0` each
// MMA cost its issuer about 180 cycles, longer than the MMA itself (4096 x 14336 x 4096: 550
// us with it, 392 without).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(r));
  return r != 0;
}

// 32 registers into 32 lanes x 32 consecutive columns of tensor memory.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void fence_async_proxy() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// A unit: its group, first token, tokens, and first channel.
struct Unit {
  int g, row0, rows, n0;
};
constexpr int kBand = 16;   // token blocks walked together over all channels, for L2
__device__ __forceinline__ Unit find_unit(const GroupTable<kThreads>& t, const PairParams& p, int u) {
  const int NT = p.num_n_tiles, blocks = t.tile0[p.a.G];
  const int b = u / (kBand * NT), first = b * kBand;
  const int h = blocks - first < kBand ? blocks - first : kBand;
  const int v = u - b * kBand * NT;
  const int mt = first + v % h;
  const int lo = find_group(t, p.a.G, mt);
  Unit r;
  r.g = lo;
  const int off = (mt - t.tile0[lo]) * p.tn;
  const int left = t.start[lo + 1] - t.start[lo] - off;
  r.row0 = t.start[lo] + off;
  r.rows = left < p.tn ? left : p.tn;
  r.n0 = v / h * 256;
  return r;
}
// Columns of the unit's MMAs: its tokens, rounded up to 16 (8 for each CTA).
__device__ __forceinline__ int unit_cols(const Unit& u) { return (u.rows + 15) & ~15; }

// The worker's units in turn, whole ones and then its share of the split ones.
struct Walk {
  int dp, it, end;
  __device__ __forceinline__ Walk(const DSched& s, int c) {
    dp = c;
    it = c < s.P ? dsk_begin(s, c) : 0;
    end = c < s.P ? dsk_begin(s, c + 1) : 0;
  }
  __device__ __forceinline__ bool next(const DSched& s, int workers, int& u, int& k0, int& k1) {
    if (dp < s.t_dp) {
      u = dp;
      k0 = 0;
      k1 = s.KS;
      dp += workers;
      return true;
    }
    if (it >= end) return false;
    const int v = it / s.gpu;
    k0 = it - v * s.gpu;
    k1 = s.gpu - k0 <= end - it ? s.gpu : k0 + (end - it);
    it += k1 - k0;
    u = s.t_dp + v;
    return true;
  }
};

// True on all 128 output threads if `mine` is on all of them.
__device__ __forceinline__ bool out_agree(bool mine) {
  uint32_t all;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "barrier.cta.red.and.pred p, %2, 128, q;\n\tselp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(all)
      : "r"(static_cast<uint32_t>(mine)), "n"(kOutBarrier)
      : "memory");
  return all != 0;
}

// 32 tokens (from the unit's token c) of the lane's channel: scaled, turned and stored by a
// warpgroup.  A lane has a channel's tokens, a row of D wants a token's channels: the tile
// passes through shared memory ([token][128 channels], two such tiles in turn) and leaves in
// 16-byte pieces, a token's 128 channels contiguous.  Where rows of D are not 16-byte aligned
// (N not a multiple of 16 bytes) a token's channels are put at the offset that its row has in
// D, so that the tile's pieces are D's aligned ones all the same, and the elements before the
// first and after the last whole one follow by themselves.
// ONE: a single tile, free when all of the warpgroup have read it.
// sa: the scale of token c + lane; sb, bias: the lane's channel's.
template <bool F32, int ROW, bool ONE>
__device__ __forceinline__ void emit_tile(const Int8Params& a, const Unit& un, int chan0, int c,
                                          float sa, float sb, float bias, const uint32_t (&r)[32],
                                          uint8_t* tile, int barrier) {
  using Elem = typename std::conditional<F32, float, __nv_bfloat16>::type;
  constexpr int kPer = 16 / sizeof(Elem), kRow = 128 / kPer;
  const int tid = threadIdx.x & 127;
  const int64_t at = static_cast<int64_t>(un.row0 + c) * a.N + chan0;
  const int step = static_cast<int>(a.N & (kPer - 1)), off0 = static_cast<int>(at & (kPer - 1));
  Elem* mine = reinterpret_cast<Elem*>(tile) + tid;
  float y[32];
  // the range of the tokens' scales (0 aside) decides for the warp whether all products of two
  // scales are normal
  const uint32_t size = __float_as_uint(fabsf(sa));
  const float lo = __uint_as_float(__reduce_min_sync(kFull, size ? size : kNone));
  const float hi = __uint_as_float(__reduce_max_sync(kFull, size));
  if (__all_sync(kFull, sb == 0.f || normal_product(lo, hi, fabsf(sb)))) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      y[i] = fmaf(__uint_as_float(r[i]), __shfl_sync(kFull, sa, i) * sb, bias);
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      y[i] = scale_sum(__uint_as_float(r[i]), __shfl_sync(kFull, sa, i), sb, bias);
  }
  if constexpr (ONE) named_barrier_sync(barrier, 128);
  if (!F32 && step == 0) {
    // neighbouring lanes pair up their channels, the even one taking the even token: half the
    // stores, which share the banks with the MMAs' operands
    const bool odd = tid & 1;
    uint8_t* pair = tile + (tid & ~1) * 2 + odd * ROW;
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const float theirs = __shfl_xor_sync(kFull, odd ? y[i] : y[i + 1], 1);
      *reinterpret_cast<uint32_t*>(pair + i * ROW) =
          odd ? pack_bf16x2(theirs, y[i + 1]) : pack_bf16x2(y[i], theirs);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      store_out<F32>(mine, i * (ROW / static_cast<int>(sizeof(Elem))) + ((off0 + i * step) & (kPer - 1)), y[i]);
  }
  named_barrier_sync(barrier, 128);
  const int tokens = un.rows - c < 32 ? un.rows - c : 32;
  const int left = a.N - chan0 < 128 ? static_cast<int>(a.N - chan0) : 128;   // channels here
  Elem* D = static_cast<Elem*>(a.D) + at;
  if (step == 0) {
#pragma unroll
    for (int i = 0; i < 32 * kRow / 128; ++i) {
      const int e = i * 128 + tid, t = e / kRow, v = e % kRow * kPer;
      if (t < tokens && v < left)
        __stcs(reinterpret_cast<uint4*>(D + t * a.N + v),
               *reinterpret_cast<const uint4*>(tile + t * ROW + v * sizeof(Elem)));
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 32 * kRow / 128; ++i) {
    const int e = i * 128 + tid, t = e / kRow, v = e % kRow * kPer;
    const int off = (off0 + t * step) & (kPer - 1);
    if (t < tokens && v >= off && v + kPer <= off + left)
      __stcs(reinterpret_cast<uint4*>(D + t * a.N + v - off),
             *reinterpret_cast<const uint4*>(tile + t * ROW + v * sizeof(Elem)));
  }
  // four threads a token: the elements of the pieces that its row cuts
  const int t = tid >> 2, off = (off0 + t * step) & (kPer - 1), end = off + left;
  const Elem* from = reinterpret_cast<const Elem*>(tile + t * ROW);
  if (t < tokens) {
#pragma unroll
    for (int j = tid & 3; j < kPer; j += 4) {
      const int tail = (end & ~(kPer - 1)) + j;
      if (j >= off && j < end && (off > 0 || end < kPer)) D[t * a.N + j - off] = from[j];
      if (tail >= kPer && tail >= off && tail < end) D[t * a.N + tail - off] = from[tail];
    }
  }
}

// Worker c's part of split unit v, this CTA's half: [token][128 channels].
__device__ __forceinline__ float* part_slot(const PairParams& p, const DSched& s, int c, int v,
                                            int rank) {
  return p.part + static_cast<int64_t>((c * 2 + dsk_slot(s, c, v)) * 2 + rank) * (128 * 256);
}

template <int TN, bool PRE, bool F32>
__global__ void __launch_bounds__(kThreads, 1)
    int8_pair_kernel(const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmA8,
                     const __grid_constant__ CUtensorMap tmA32,
                     const __grid_constant__ CUtensorMap tmAll, const PairParams p) {
  using C = Cfg<TN, PRE, F32>;
  constexpr int kStages = C::kStages, kSlots = C::kSlots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* raw = smem;
  uint8_t* wide = raw + kStages * C::kRawBytes;
  uint8_t* stage_out = wide + C::kTokSlots * C::kWideBytes;   // the output tiles
  uint64_t* full = reinterpret_cast<uint64_t*>(stage_out + C::kOutTiles * C::kOutBytes);
  uint64_t* empty = full + kStages;
  uint64_t* wide_full = empty + kStages;        // in the leader: widening warps of both CTAs
  uint64_t* wide_empty = wide_full + kSlots;    // in both: the MMAs' commit
  uint64_t* acc_full = wide_empty + kSlots;     // [2] in both
  uint64_t* acc_empty = acc_full + 2;           // [2] in the leader: output warps of both CTAs
  uint64_t* drain = acc_empty + 2;
  uint64_t* tok_full = drain + 1;               // PRE: in the leader, both CTAs' bytes
  uint64_t* tok_empty = tok_full + C::kTokSlots;   // PRE: in both, the MMAs' commit
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1 + (PRE ? 2 * C::kTokSlots : 0));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  Table& table = *reinterpret_cast<Table*>(reinterpret_cast<uint8_t*>(full) + 512);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 4);       // a widening warpgroup
    }
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&wide_full[s], 8);   // a widening warpgroup of each CTA
      mbar_init(&wide_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&acc_full[s], 1);
      mbar_init(&acc_empty[s], 8);   // output warps of both CTAs
    }
    mbar_init(drain, 1);
    if constexpr (PRE)
      for (int s = 0; s < C::kTokSlots; ++s) {
        mbar_init(&tok_full[s], 1);
        mbar_init(&tok_empty[s], 1);
      }
    *abort_flag = 0;
    table.fixes = 0;
    fence_mbar_init();
    prefetch_tmap(&tmB);
    prefetch_tmap(&tmA8);
    prefetch_tmap(&tmA32);
    prefetch_tmap(&tmAll);
  }
  build_table(table.groups, p.a, p.tn);
  // both CTAs read the same sizes, so a bad table stops the whole cluster here.  (With PRE
  // the launch may have started before the widening pass has ended: one warp of every CTA
  // waits for that, so that this grid's end is the pass's too.)
  if (table.groups.bad) {
    if (PRE && warp == 2) grid_dependency_wait();
    return;
  }

  // warp 0 starts loading at once: its copies complete on barriers of this CTA alone
  uint32_t tmem = 0;
  if (warp == 0) {
    cluster_arrive();
  } else {
    if (warp == 1) {
      tmem_alloc_pair(tmem_slot, 512);
      tmem_relinquish_pair();
    }
    tc_fence_before();
    named_barrier_sync(kSetupBarrier, kThreads - 32);
    cluster_arrive();
    cluster_wait();
    tc_fence_after();
    tmem = *tmem_slot;
  }
  const uint32_t tmem_wide = tmem + 512 - kSlots * kSlotCols;
  const int worker = static_cast<int>(blockIdx.x >> 1), workers = static_cast<int>(gridDim.x >> 1);
  const DSched sched = make_dsched(table.groups.tile0[p.a.G] * p.num_n_tiles, p.stages_k, 1, workers,
                                   p.part != nullptr, 14, 4);
  Walk walk(sched, worker);
  int u, k0, k1;

  if (warp == 0) {
    // ---------------------------------------------------------------- producer, channels
    // (and, without PRE, the tokens on the same barrier)
    int stage = 0;
    uint32_t phase = 0, armed = 0, armed_parity = 0;
    bool ok = true;
    while (ok && walk.next(sched, workers, u, k0, k1)) {
      const Unit un = find_unit(table.groups, p, u);
      const int half = unit_cols(un) / 2;
      const int row = un.row0 + rank * half;
      const int chan = static_cast<int>(un.g * p.a.N) + un.n0 + rank * 128;
      for (int k = k0; k < k1; ++k) {
        if (!wait_phase(&empty[stage], phase ^ 1, p.limit_ns, abort_flag, p.a.status)) {
          ok = false;
          break;
        }
        armed |= 1u << stage;
        armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
        if (elect_one()) {
          mbar_arrive_expect_tx(&full[stage], 128 * 128 + (PRE ? 0 : half * 128));
          uint8_t* dst = raw + stage * C::kRawBytes;
          tma_load_2d(&tmB, &full[stage], dst, k * 128, chan);
          if constexpr (!PRE) {
            dst += 128 * 128;
            int r = 0;
            if (half == p.tn / 2) {
              tma_load_2d(&tmAll, &full[stage], dst, k * 128, row);
              r = half;
            }
            for (; r + 32 <= half; r += 32)
              tma_load_2d(&tmA32, &full[stage], dst + r * 128, k * 128, row + r);
            for (; r < half; r += 8) tma_load_2d(&tmA8, &full[stage], dst + r * 128, k * 128, row + r);
          }
        }
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    // no copy may land after the block has finished
    for (int s = 0; s < kStages; ++s)
      if (armed & (1u << s)) {
        volatile int no_abort = 0;
        wait_phase(&full[s], (armed_parity >> s) & 1u, p.limit_ns / 4 + 1, &no_abort, nullptr);
      }
    __syncwarp();
    cluster_wait();
  } else if (PRE && warp == 2) {
    // ---------------------------------------------------------------- producer, FP16 tokens
    // A warp of its own: with both on one warp the issuing itself (some 1100 cycles for a
    // stage's three copies) was longer than the stage's MMAs.
    grid_dependency_wait();   // for the widening pass that wrote the tokens
    int tok = 0;
    uint32_t phase = 0, armed = 0, armed_parity = 0;
    bool ok = true;
    while (ok && walk.next(sched, workers, u, k0, k1)) {
      const Unit un = find_unit(table.groups, p, u);
      const int half = unit_cols(un) / 2;
      const int row = un.row0 + rank * half;
      for (int k = k0; k < k1; ++k) {
        if (!wait_phase(&tok_empty[tok], phase ^ 1, p.limit_ns, abort_flag, p.a.status)) {
          ok = false;
          break;
        }
        if (rank == 0) {
          armed |= 1u << tok;
          armed_parity = (armed_parity & ~(1u << tok)) | (phase << tok);
        }
        if (elect_one()) {
          const uint32_t bar = map_to_cta(smem_u32(&tok_full[tok]), 0);
          const int halves = p.halves_k - 2 * k < 2 ? 1 : 2;
          if (rank == 0) mbar_arrive_expect_tx(&tok_full[tok], halves * 2 * half * 128);
          for (int h = 0; h < halves; ++h) {
            uint8_t* dst = wide + tok * C::kWideBytes + h * (C::kWideBytes / 2);
            const int x = (2 * k + h) * 128;
            int r = 0;
            if (half == p.tn / 2) {
              tma_load_2d_pair(&tmAll, bar, dst, x, row);
              r = half;
            }
            for (; r + 32 <= half; r += 32) tma_load_2d_pair(&tmA32, bar, dst + r * 128, x, row + r);
            for (; r < half; r += 8) tma_load_2d_pair(&tmA8, bar, dst + r * 128, x, row + r);
          }
        }
        if (++tok == C::kTokSlots) {
          tok = 0;
          phase ^= 1;
        }
      }
    }
    // both CTAs' copies complete on the leader's barriers
    for (int s = 0; s < C::kTokSlots; ++s)
      if (armed & (1u << s)) {
        volatile int no_abort = 0;
        wait_phase(&tok_full[s], (armed_parity >> s) & 1u, p.limit_ns / 4 + 1, &no_abort, nullptr);
      }
  } else if (warp == 1) {
    if (rank == 0) {
      // -------------------------------------------------------------- MMA issuer (leader)
      uint32_t tcount = 0, slot = 0, slot_phase = 0, tok = 0, tok_phase = 0;
      const uint64_t b_desc = make_sdesc(smem_u32(wide), 16, 1024, kSwizzle128B);
      bool ok = true;
      while (ok && walk.next(sched, workers, u, k0, k1)) {
        const Unit un = find_unit(table.groups, p, u);
        const uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(unit_cols(un) >> 3) << 17) |
                               ((256u >> 4) << 24);   // FP32 accumulator, FP16 operands, M = 256
        const uint32_t buf = tcount % C::kBufs;
        if (!wait_phase<true>(&acc_empty[buf], ((tcount / C::kBufs) & 1) ^ 1, p.limit_ns, abort_flag,
                               p.a.status))
          break;
        ++tcount;
        const uint32_t d = tmem + buf * TN;
        for (int k = k0; k < k1; ++k) {
          if (!wait_phase<true>(&wide_full[slot], slot_phase, p.limit_ns, abort_flag, p.a.status)) {
            ok = false;
            break;
          }
          if constexpr (PRE) {
            if (!wait_phase<true>(&tok_full[tok], tok_phase, p.limit_ns, abort_flag, p.a.status)) {
              ok = false;
              break;
            }
          }
          tc_fence_after();
          if (elect_one()) {
            const uint64_t b = b_desc + ((PRE ? tok : slot & 1) * C::kWideBytes >> 4);
            const uint32_t a = tmem_wide + slot * kSlotCols;
            mma_f16_pair_ts(d, a, b, idesc, k != k0);
#pragma unroll
            for (int j = 1; j < 4; ++j) mma_f16_pair_ts(d, a + j * 8, b + 2 * j, idesc, 1);
            if (2 * k + 1 < p.halves_k) {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                mma_f16_pair_ts(d, a + 32 + j * 8, b + (C::kWideBytes / 2 >> 4) + 2 * j, idesc, 1);
            }
            tc_commit_pair(&wide_empty[slot], kPairMask);
            if constexpr (PRE) tc_commit_pair(&tok_empty[tok], kPairMask);
          }
          if (++slot == kSlots) {
            slot = 0;
            slot_phase ^= 1;
          }
          if constexpr (PRE) {
            if (++tok == C::kTokSlots) {
              tok = 0;
              tok_phase ^= 1;
            }
          }
        }
        if (!ok) break;
        if (elect_one()) tc_commit_pair(&acc_full[buf], kPairMask);
      }
      // every MMA must be finished before tensor memory is freed
      __syncwarp();
      if (elect_one()) tc_commit_pair(drain, 1);
      volatile int no_abort = 0;
      wait_phase(drain, 0, p.limit_ns, &no_abort, nullptr);
    }
  } else if (warp >= kWideWarp0 && warp < kOutWarp0) {
    // ---------------------------------------------------------------- widening (both CTAs)
    // The warpgroups take stages in turn: a stage is a chain of waits and latencies, and a
    // whole stage a warpgroup has half as many of them as half of every stage.
    const int wg = (warp - kWideWarp0) >> 2, tid = threadIdx.x & 127;
    const uint32_t taddr = tmem_wide + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    // 16-byte piece j of a 64-K half of the thread's channel is at chan ^ (j << 4) of the
    // stage, ^ 64 for the second half (the 128-byte swizzle exchanges pieces by the row's
    // number modulo 8)
    const uint32_t chan = static_cast<uint32_t>(tid) * 128 + ((tid & 7) << 4);
    constexpr int kPieces = PRE ? 0 : (C::kHalf + 31) / 32;   // of a half's tokens, a thread
    // Loads of both halves first, one latency for all.  With few tokens a thread everything is
    // in registers then; else the channels are widened and stored half by half.
    constexpr bool kWhole = PRE || kPieces <= 1;
    int stage = wg, slot = wg % kSlots, k_off = wg;
    uint32_t phase = 0, slot_phase = 0;
    bool ok = true;
    auto widen16 = [](const uint4 (&c)[4], uint32_t (&w)[32]) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        widen4(c[j].x, w[8 * j], w[8 * j + 1]);
        widen4(c[j].y, w[8 * j + 2], w[8 * j + 3]);
        widen4(c[j].z, w[8 * j + 4], w[8 * j + 5]);
        widen4(c[j].w, w[8 * j + 6], w[8 * j + 7]);
      }
    };
    auto store_tokens = [](const uint4& x, uint32_t dst) {
      uint32_t v[8];
      widen4(x.x, v[0], v[1]);
      widen4(x.y, v[2], v[3]);
      widen4(x.z, v[4], v[5]);
      widen4(x.w, v[6], v[7]);
      sts128(dst, v[0], v[1], v[2], v[3]);
      sts128(dst ^ 16, v[4], v[5], v[6], v[7]);
    };
    while (ok && walk.next(sched, workers, u, k0, k1)) {
      const Unit un = find_unit(table.groups, p, u);
      const int half = unit_cols(un) / 2;
      // the thread's i-th 16-byte piece of the tokens is that of token e % half, piece
      // e / half of its four, e = i * 128 + tid: where it is in a stage, and where its first
      // eight FP16 values go in a slot (the others 16 bytes on, before the swizzle)
      uint32_t from[kPieces + 1], to[kPieces + 1];
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int e = i * 128 + tid, piece = e / half, r = e - piece * half;
        from[i] = piece < 4 ? 128 * 128 + r * 128 + ((piece ^ (r & 7)) << 4) : kNone;
        to[i] = r * 128 + (((2 * piece) ^ (r & 7)) << 4);
      }
      int k = k0 + k_off;
      for (; k < k1; k += 2) {
        if (!wait_phase(&full[stage], phase, p.limit_ns, abort_flag, p.a.status)) {
          ok = false;
          break;
        }
        const uint32_t base = smem_u32(raw + stage * C::kRawBytes);
        const uint32_t out = smem_u32(wide + (slot & 1) * C::kWideBytes);   // (not with PRE)
        const uint32_t tslot = taddr + slot * kSlotCols;
        const int halves = 2 * k + 1 < p.halves_k ? 2 : 1;
        auto release_stage = [&] {
          __syncwarp();
          if (lane == 0) mbar_arrive(&empty[stage]);
        };
        // PRE: the channels' slot is free.  Else the tokens' is, once the MMAs of the stage
        // two back are done; the warpgroup's last stage waited for those of four back, which
        // had this one's slot of channels.
        auto slot_free = [&] {
          const int of = PRE ? slot : slot ^ 2;
          const uint32_t parity = PRE || slot < 2 ? slot_phase ^ 1 : slot_phase;
          ok = wait_phase(&wide_empty[of], parity, p.limit_ns, abort_flag, p.a.status);
          tc_fence_after();
          return ok;
        };
        if constexpr (kWhole) {
          uint4 c[4], d[4], x[2];
          uint32_t w[32], y[32];
#pragma unroll
          for (int j = 0; j < 4; ++j) c[j] = lds128(base + (chan ^ (j << 4)));
#pragma unroll
          for (int j = 0; j < 4; ++j) d[j] = lds128(base + (chan ^ 64 ^ (j << 4)));
          if (kPieces > 0 && from[0] != kNone) {
            x[0] = lds128(base + from[0]);
            x[1] = lds128(base + (from[0] ^ 64));
          }
          widen16(c, w);
          widen16(d, y);
          release_stage();
          if (PRE && !slot_free()) break;
          tmem_st32(tslot, w);
          if (halves == 2) tmem_st32(tslot + 32, y);
          if (!PRE && !slot_free()) {
            tmem_st_wait();
            break;
          }
          if (kPieces > 0 && from[0] != kNone) {
            store_tokens(x[0], out + to[0]);
            store_tokens(x[1], out + C::kWideBytes / 2 + to[0]);
          }
        } else {
          // everything is loaded and the stage handed back first, the registers then freed half
          // by half
          uint4 c[8], x[2][kPieces + 1];
#pragma unroll
          for (int j = 0; j < 8; ++j) c[j] = lds128(base + (chan ^ (j << 4)));
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < kPieces; ++i)
              if (from[i] != kNone) x[h][i] = lds128(base + (from[i] ^ (h << 6)));
          release_stage();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (h == halves) break;
            uint32_t w[32];
            const uint4 half_c[4] = {c[4 * h], c[4 * h + 1], c[4 * h + 2], c[4 * h + 3]};
            widen16(half_c, w);
            tmem_st32(tslot + h * 32, w);
          }
          if (!slot_free()) {
            tmem_st_wait();
            break;
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (h == halves) break;
#pragma unroll
            for (int i = 0; i < kPieces; ++i)
              if (from[i] != kNone) store_tokens(x[h][i], out + h * (C::kWideBytes / 2) + to[i]);
          }
        }
        tmem_st_wait();
        fence_async_proxy();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_leader(map_to_cta(smem_u32(&wide_full[slot]), 0));
        if ((stage += 2) >= kStages) {
          stage -= kStages;
          phase ^= 1;
        }
        if ((slot += 2) >= kSlots) {
          slot -= kSlots;
          slot_phase ^= 1;
        }
      }
      k_off = k - k1;
    }
  } else if (warp >= kOutWarp0) {
    // ---------------------------------------------------------------- output (both CTAs)
    // The four warps move together: every step that could give up is agreed on at a barrier
    // first, so none is left waiting.
    const int q = warp & 3, tid = threadIdx.x & 127;
    const uint32_t acc_empty_leader = map_to_cta(smem_u32(acc_empty), 0);
    uint32_t tcount = 0, flip = 0;
    while (walk.next(sched, workers, u, k0, k1)) {
      const Unit un = find_unit(table.groups, p, u);
      const int cols = unit_cols(un), chan0 = un.n0 + rank * 128;
      const int64_t n = chan0 + tid;
      const bool ok = n < p.a.N;
      const float sb = ok ? p.a.sB[un.g * p.a.N + n] : 0.f;
      const float bias = ok && p.a.bias ? __bfloat162float(p.a.bias[n]) : 0.f;
      // loaded ahead of the accumulator: lane l has the scales of tokens l, l + 32, ...
      float sa[TN / 32];
#pragma unroll
      for (int i = 0; i < TN / 32; ++i)
        sa[i] = 32 * i + lane < un.rows ? p.a.sA[un.row0 + 32 * i + lane] : 0.f;
      const uint32_t buf = tcount % C::kBufs;
      const bool got = wait_phase(&acc_full[buf], (tcount / C::kBufs) & 1, p.limit_ns, abort_flag, p.a.status);
      if (!out_agree(got)) break;
      ++tcount;
      tc_fence_after();
      const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * TN;
      const bool whole = k1 - k0 == p.stages_k;
      const int v = u - sched.t_dp;
      float* mine = whole ? nullptr : part_slot(p, sched, worker, v, rank) + tid;
#pragma unroll 1
      for (int c = 0; c < cols; c += 32) {
        uint32_t r[32];
        tmem_ld32(taddr + c, r);
        tmem_ld_wait(r);
        if (c + 32 >= cols) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_leader(acc_empty_leader + buf * 8);
        }
        if (whole) {
          emit_tile<F32, C::kOutRow, C::kOutTiles == 1>(p.a, un, chan0, c, sa[0], sb, bias, r,
                                                        stage_out + flip * C::kOutBytes, kOutBarrier);
          flip ^= C::kOutTiles - 1;
#pragma unroll
          for (int i = 0; i + 1 < TN / 32; ++i) sa[i] = sa[i + 1];
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (c + i < un.rows) __stcg(mine + (c + i) * 128, __uint_as_float(r[i]));
        }
      }
      if (whole) continue;
      // counted in; the last contributor's CTA adds the parts when its walk is over
      __threadfence();
      named_barrier_sync(kOutBarrier, 128);
      if (tid == 0) {
        int* ctr = p.arrivals + (v * 2 + rank) * 8;
        if (atomicAdd(ctr, 1) + 1 == dsk_last_worker(sched, v) - dsk_first_worker(sched, v) + 1) {
          *ctr = 0;   // every contributor has counted itself in
          table.fix[table.fixes++] = u;
        }
      }
    }
  }
  if (sched.P > 0 && warp >= kWideWarp0) {
    // ---------------------------------------------------------------- split units' sums
    // By the output and the widening warpgroups together, 32 tokens each in turn: the sum is
    // bound by the latency of the parts' loads, so what counts is how many are in flight.
    // The parts are added in K order, whoever came last.
    named_barrier_sync(kFixBarrier, 384);
    const int wg = (warp - kWideWarp0) >> 2, tid = threadIdx.x & 127;
    uint8_t* tiles = wg == 2 ? stage_out : raw + wg * C::kOutTiles * C::kOutBytes;   // the rings are idle now
    uint32_t flip = 0;
    if (table.fixes > 0) __threadfence();
    for (int f = 0; f < table.fixes; ++f) {
      const int v = table.fix[f] - sched.t_dp;
      const Unit un = find_unit(table.groups, p, table.fix[f]);
      const int chan0 = un.n0 + rank * 128;
      const int64_t n = chan0 + tid;
      const bool ok = n < p.a.N;
      const float sb = ok ? p.a.sB[un.g * p.a.N + n] : 0.f;
      const float bias = ok && p.a.bias ? __bfloat162float(p.a.bias[n]) : 0.f;
      const int c_lo = dsk_first_worker(sched, v), c_hi = dsk_last_worker(sched, v);
#pragma unroll 1
      for (int c = wg * 32; c < un.rows; c += 96) {
        const float sa = c + lane < un.rows ? p.a.sA[un.row0 + c + lane] : 0.f;
        float sum[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) sum[i] = 0.f;
#pragma unroll 1
        for (int cc = c_lo; cc <= c_hi; cc += 2) {
          const bool two = cc < c_hi;
          const float* x = part_slot(p, sched, cc, v, rank) + tid + c * 128;
          const float* y = part_slot(p, sched, two ? cc + 1 : cc, v, rank) + tid + c * 128;
          float xs[32], ys[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            xs[i] = c + i < un.rows ? __ldcg(x + i * 128) : 0.f;
            ys[i] = two && c + i < un.rows ? __ldcg(y + i * 128) : 0.f;
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) sum[i] = sum[i] + xs[i] + ys[i];
        }
        uint32_t r[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(sum[i]);
        emit_tile<F32, C::kOutRow, C::kOutTiles == 1>(p.a, un, chan0, c, sa, sb, bias, r,
                                                      tiles + flip * C::kOutBytes, kOutBarrier + 2 + wg);
        flip ^= C::kOutTiles - 1;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // both CTAs are done with tensor memory and with each other's barriers
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
  cluster_sync();
}

// tok16: the tokens in FP16 ([total_M][K]) with PRE.
template <int TN, bool PRE, bool F32>
bsmma_status launch_tn(PairParams p, const void* tok16, const DeviceInfo* dev, cudaStream_t stream) {
  using C = Cfg<TN, PRE, F32>;
  auto kern = int8_pair_kernel<TN, PRE, F32>;
  static PerDevice clusters_fit;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int max_clusters = 0;
  bsmma_status st = clusters_fit.get(dev->device, &max_clusters, [&](int* fit) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes) !=
        cudaSuccess)
      return BSMMA_ERR_CUDA;
    cfg.gridDim = dim3(2 * (dev->sm_count / 2), 1, 1);
    if (cudaOccupancyMaxActiveClusters(fit, kern, &cfg) != cudaSuccess || *fit < 1) return BSMMA_ERR_CUDA;
    if (*fit > dev->sm_count / 2) *fit = dev->sm_count / 2;
    return BSMMA_OK;
  });
  if (st != BSMMA_OK) return st;
  CUtensorMap tb, ta8, ta32, tall;
  const Int8Params& a = p.a;
  st = encode_tmap_u8(&tb, a.B, a.K, static_cast<uint64_t>(a.G) * a.N, a.K, 128, 128);
  if (st != BSMMA_OK) return st;
  // with no rows there is no tile of A to load; B's address stands in for the map
  const void* A = a.total_M > 0 ? (PRE ? tok16 : a.A) : a.B;
  const uint64_t rows = a.total_M > 0 ? a.total_M : 1, row_bytes = PRE ? 2 * a.K : a.K;
  st = encode_tmap_u8(&ta8, A, row_bytes, rows, row_bytes, 128, 8);
  if (st != BSMMA_OK) return st;
  st = encode_tmap_u8(&ta32, A, row_bytes, rows, row_bytes, 128, 32);
  if (st != BSMMA_OK) return st;
  // blocks of tn tokens: a single group's are made equally large
  p.tn = TN;
  if (a.G == 1 && a.total_M > 0) {
    const int64_t blocks = (a.total_M + TN - 1) / TN;
    p.tn = static_cast<int>(((a.total_M + blocks - 1) / blocks + 15) / 16 * 16);
  }
  st = encode_tmap_u8(&tall, A, row_bytes, rows, row_bytes, 128, p.tn / 2);
  if (st != BSMMA_OK) return st;
  p.part = nullptr;
  p.arrivals = nullptr;
  st = split_workspace(stream, &p.part, &p.arrivals);
  if (st == BSMMA_ERR_WORKSPACE) {   // captured on a stream without one: no unit is split
    p.part = nullptr;
    p.arrivals = nullptr;
  } else if (st != BSMMA_OK) {
    return st;
  }
  p.num_n_tiles = static_cast<int>((a.N + 255) / 256);
  p.stages_k = static_cast<int>((a.K + 127) / 128);
  p.halves_k = static_cast<int>((a.K + 63) / 64);
  p.limit_ns = wait_limit_ns();
  cfg.gridDim = dim3(static_cast<unsigned>(2 * max_clusters), 1, 1);
  cfg.stream = stream;
  cfg.numAttrs = PRE ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, tb, ta8, ta32, tall, p);
  count_launches(1);
  return cuda_ok(e == cudaSuccess ? cudaGetLastError() : e);
}

}  // namespace

namespace {
// int8 [n16 * 16] -> FP16: four 16-byte loads in flight a thread.
constexpr int kWidenSteps = 4;
__global__ void __launch_bounds__(256) widen_kernel(const uint4* __restrict__ in,
                                                    uint4* __restrict__ out, int64_t n16) {
  grid_launch_dependents();
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (256 * kWidenSteps) + threadIdx.x;
  uint4 v[kWidenSteps];
#pragma unroll
  for (int j = 0; j < kWidenSteps; ++j)
    if (i0 + j * 256 < n16) v[j] = __ldcs(in + i0 + j * 256);
#pragma unroll
  for (int j = 0; j < kWidenSteps; ++j) {
    uint4 a, b;
    widen4(v[j].x, a.x, a.y);
    widen4(v[j].y, a.z, a.w);
    widen4(v[j].z, b.x, b.y);
    widen4(v[j].w, b.z, b.w);
    if (i0 + j * 256 < n16) {
      out[2 * (i0 + j * 256)] = a;
      out[2 * (i0 + j * 256) + 1] = b;
    }
  }
}
}  // namespace

// Which tile a launch takes: the cheapest by an estimate in SM cycles that the host makes from
// the sizes alone.
//   - A 128-K stage with the tokens widened in the kernel takes about 660 + 2.75 cycles a column
//     in tiles of 32 and 64, 770 + 0.75 in tiles of 128 (two accumulators, half the registers a
//     thread) and 700 + 2.7 in tiles of 256: fits to 32 to 256 columns, dense and grouped.  With
//     FP16 tokens it takes its eight MMAs, 9 + 0.5 cycles a column each and 14% more, or the
//     channels' arrival: the ring is four stages then, and without other blocks that bring the same channels to L2 a
//     stage waits some 1200 cycles for DRAM.
//   - A wave of units that leaves pairs idle is split over them when that is shorter; a
//     split costs some 18000 cycles and more with many parts (written, counted, read back).
//     Measured at 14336 x 4096, 128 rows: 27 us unsplit, 35 us split, 56 units on 76 pairs.
//   - Each block reads its channels from DRAM, at 3.3 KB a cycle; FP16 tokens cost a pass over
//     them first and twice the bytes.
// At 4096 x 14336 x 4096: 268 us with FP16 tokens (192 columns), 311 us without (256); 64
// experts of 2048 x 7168 with 192 rows each: 293 and 260 us, in tiles of 128 351; with 96 rows each
// 185 in tiles of 128, 208 of 256, which it takes all the same: it counts on uneven groups, some of
// them with more than 128 rows.  512 x 14336 x 4096: 54 us in tiles of 128 (chosen), 66 of 256, 62
// and 76 with FP16 tokens in tiles of 256 and 192.
struct Choice {
  int tn;
  bool pre;
};
double estimate(const Int8Params& a, int tn, bool pre, int pairs) {
  const double active = groups_with_rows(a);
  const double rows = active > 0 ? a.total_M / active : 0;
  const double blocks = blocks_per_group(a, rows, tn);
  const double cols = std::fmax(16, rows / blocks);
  const double stage = pre ? std::fmax(900 + 300 / std::fmax(1, blocks - 1), 8 * 1.14 * (9 + 0.5 * cols))
                     : tn > 128 ? 700 + 2.7 * cols
                     : tn > 64  ? 770 + 0.75 * cols
                                : 660 + 2.75 * cols;
  const double ks = static_cast<double>((a.K + 127) / 128);
  const double units = blocks * active * ((a.N + 255) / 256);
  const double full = std::floor(units / pairs), rem = units - full * pairs;
  // parts of a unit, read back two at a time for each 96 tokens
  const double parts = rem > 0 ? std::ceil(pairs / rem) + 1 : 0;
  const double join = 18000 + std::ceil(cols / 96) * std::ceil(parts / 2) * 2600;
  const double tail = rem > 0 ? std::fmin(ks, ks * rem / pairs + join / stage) : 0;
  const double drain = tn > 192 ? full * 5000 : 0;   // one accumulator: not overlapped
  const double size = static_cast<double>(a.K) * (pre ? 5 : 1);
  const double dram = (blocks * active * a.N * a.K + a.total_M * (size + 2 * a.N)) / 3300;
  return std::fmax((full * ks + tail) * stage + drain + (pre ? 8000 + a.total_M * a.K * 0.9e-3 : 0), dram);
}
Choice choose(const Int8Params& a, int pairs, double* cycles = nullptr) {
  const Choice all[] = {{32, false}, {64, false}, {128, false}, {256, false}, {192, true}, {256, true}};
  Choice best = all[0];
  double least = -1;
  for (const Choice& c : all) {
    const double t = estimate(a, c.tn, c.pre, pairs);
    if (least < 0 || t < least) {
      least = t;
      best = c;
    }
  }
  if (cycles) *cycles = least;
  return best;
}

// (9500: launch, setup and the start of the pipeline)
double pair_cycles(const Int8Params& a, const DeviceInfo* dev) {
  double t = 0;
  choose(a, dev->sm_count / 2, &t);
  return t + 9500;
}

bsmma_status launch_pair(const Int8Params& a, bool f32, const DeviceInfo* dev, cudaStream_t stream) {
  PairParams p;
  p.a = a;
  Choice c = int8_tile() > 1 ? Choice{int8_tile(), int8_fp16_tokens()} : choose(a, dev->sm_count / 2);
  if (a.total_M == 0) c = Choice{32, false};   // no rows to widen; the sizes are still checked
  void* tok16 = nullptr;
  std::optional<StreamLock> lock;   // from the widened tokens' lookup to the products
  if (c.pre) {
    lock.emplace(stream);
    // captured without a workspace, or no memory for one, or rows of more bytes than a copy's
    // coordinate counts: widened in the kernel
    const bsmma_status st = a.K < (int64_t(1) << 30) ? stream_workspace(a.total_M * a.K * 2, stream, &tok16)
                                                     : BSMMA_ERR_WORKSPACE;
    if (st != BSMMA_OK) {
      cudaGetLastError();
      c = Choice{256, false};
    }
  }
  if (c.pre) {
    const int64_t n16 = a.total_M * a.K / 16, per = 256 * kWidenSteps;
    widen_kernel<<<static_cast<unsigned>((n16 + per - 1) / per), 256, 0, stream>>>(
        reinterpret_cast<const uint4*>(a.A), static_cast<uint4*>(tok16), n16);
    count_launches(1);
    if (cudaGetLastError() != cudaSuccess) return BSMMA_ERR_CUDA;
  }
#define BSMMA_INT8_TN(T, PRE) \
  (f32 ? launch_tn<T, PRE, true>(p, tok16, dev, stream) : launch_tn<T, PRE, false>(p, tok16, dev, stream))
  if (c.pre) return c.tn == 192 ? BSMMA_INT8_TN(192, true) : BSMMA_INT8_TN(256, true);
  return c.tn == 32 ? BSMMA_INT8_TN(32, false) : c.tn == 64 ? BSMMA_INT8_TN(64, false) : c.tn == 128 ? BSMMA_INT8_TN(128, false)
                                                             : BSMMA_INT8_TN(256, false);
#undef BSMMA_INT8_TN
}

}  // namespace int8
}  // namespace bsmma
