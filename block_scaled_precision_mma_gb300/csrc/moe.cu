// moe.cu -- the operators around the experts' products: routing tokens to experts with
// its gradient, the expert order of the chosen slots, and the weighted sum of the
// experts' outputs with its gradients.
//
// All of them move far more bytes than they compute on, so each kernel reads its inputs
// once with loads that a warp covers whole sectors with, keeps what it needs in registers
// or shared memory, and writes its outputs once.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>

#include "internal.h"
#include "ptx.cuh"

namespace bsmma {
namespace {

constexpr uint32_t kFull = 0xFFFFFFFFu;

template <bool F32>
__device__ __forceinline__ float load_elem(const void* p, int64_t i) {
  if constexpr (F32)
    return static_cast<const float*>(p)[i];
  else
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
template <bool F32>
__device__ __forceinline__ void store_elem(void* p, int64_t i, float v) {
  if constexpr (F32)
    static_cast<float*>(p)[i] = v;
  else
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// FP32 as an unsigned integer of the same order (-inf lowest of the finite order).
__device__ __forceinline__ uint32_t ordered(float f) {
  const uint32_t b = __float_as_uint(f + 0.f);   // -0 and +0 are one key
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// A logit as the router reads it: NaN closes the expert like -inf does; +inf is the
// largest finite value, so that exp(x - max) is defined.
__device__ __forceinline__ float clean_logit(float x) {
  return x != x ? -INFINITY : fminf(x, FLT_MAX);
}
__device__ __forceinline__ float sigmoid(float x) { return 1.f / (1.f + expf(-x)); }

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// ------------------------------------------------------------------------- routing
// One warp per token; lane l holds experts l, l + 32, ... (V of them).  The k choices are
// k rounds of a warp-wide maximum over (key, lowest index): each lane keeps the best of
// its own V keys and only the round's winner looks for its next one.
struct RouteParams {
  const void* logits;
  const float* bias;
  int64_t T;
  int E, k, groups, topk_groups, group_top;
  int sigmoid, renormalize;
  float scale;
  int32_t* ids;
  float* weights;
};

// Both score functions increase with the logit, so without a bias the keys are the logits
// themselves and no rounding of a score can reorder the choice.
template <bool F32, int V>
__global__ void __launch_bounds__(128) route_kernel(const RouteParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= p.T) return;
  float key[V];
  float mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 32 * i;
    key[i] = e < p.E ? clean_logit(load_elem<F32>(p.logits, t * p.E + e)) : -INFINITY;
    mx = fmaxf(mx, key[i]);
  }
  const bool summed_groups = p.groups > 1 && p.group_top > 1;
  const bool all_scores = p.bias || summed_groups;
  float denom = 1.f;
  if (!p.sigmoid) {
    mx = warp_max(mx);
    if (mx == -INFINITY) mx = 0.f;
    if (all_scores || !p.renormalize) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) sum += expf(key[i] - mx);
      sum = warp_sum(sum);
      denom = sum > 0.f ? sum : 1.f;
    }
  }
  auto score = [&](float x) { return p.sigmoid ? sigmoid(x) : expf(x - mx) / denom; };

  float of[V];   // what a group is valued by
#pragma unroll
  for (int i = 0; i < V; ++i) of[i] = key[i];
  if (all_scores) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane + 32 * i;
      if (e < p.E) {
        float s = -INFINITY;
        if (key[i] != -INFINITY) {
          s = score(key[i]);
          if (p.bias) {
            s += p.bias[e];
            if (s != s) s = -INFINITY;
            key[i] = s;
          }
        }
        of[i] = s;
      }
    }
  }
  if (p.groups > 1) {
    // value of a group: the sum of its group_top largest keys (of its scores without a bias)
    const int per = p.E / p.groups;
    extern __shared__ float smem[];
    float* row = smem + (threadIdx.x >> 5) * p.E;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (lane + 32 * i < p.E) row[lane + 32 * i] = of[i];
    __syncwarp();
    // `width` lanes (a power of two) share a group
    int width = 32;
    while (width * p.groups > 32) width >>= 1;
    const int g = lane / width;
    float a = -INFINITY, b = -INFINITY;   // the group's largest and second largest
    if (g < p.groups)
      for (int i = lane % width; i < per; i += width) {
        const float v = row[g * per + i];
        if (v > a) {
          b = a;
          a = v;
        } else if (v > b) {
          b = v;
        }
      }
    for (int o = 1; o < width; o <<= 1) {
      const float a2 = __shfl_xor_sync(kFull, a, o), b2 = __shfl_xor_sync(kFull, b, o);
      b = fmaxf(fminf(a, a2), fmaxf(b, b2));
      a = fmaxf(a, a2);
    }
    float value = a;
    if (p.group_top > 1 && b != -INFINITY) value = a + b;
    // a group is open when fewer than topk_groups are ahead of it (ties: lower index first)
    int ahead = 0;
    for (int j = 0; j < p.groups; ++j) {
      const float v = __shfl_sync(kFull, value, j * width);
      ahead += v > value || (v == value && j < g);
    }
    const uint32_t open = __ballot_sync(kFull, g < p.groups && ahead < p.topk_groups);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane + 32 * i;
      if (e < p.E && !((open >> ((e / per) * width)) & 1u)) key[i] = -INFINITY;
    }
  }

  float best = -INFINITY;
  int at = 0;
  auto rescan = [&] {
    best = -INFINITY;
    at = 0;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i;
      }
  };
  rescan();
  int mine = -1;   // lane j keeps the j-th choice
  for (int j = 0; j < p.k; ++j) {
    const uint32_t o = ordered(best);
    const uint32_t top = __reduce_max_sync(kFull, o);
    if (top == ordered(-INFINITY)) break;
    const uint32_t e = __reduce_min_sync(kFull, o == top ? static_cast<uint32_t>(lane + 32 * at)
                                                         : 0xFFFFFFFFu);
    if (lane == j) mine = static_cast<int>(e);
    if (static_cast<int>(e & 31u) == lane) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i == at) key[i] = -INFINITY;
      rescan();
    }
  }
  // the chosen experts' logits are read again from the row (cached)
  float s = 0.f;
  if (mine >= 0) s = score(clean_logit(load_elem<F32>(p.logits, t * p.E + mine)));
  if (p.renormalize) {
    const float sum = warp_sum(s);
    s = sum > 0.f ? s / sum : 0.f;
  }
  if (lane < p.k) {
    p.ids[t * p.k + lane] = mine;
    p.weights[t * p.k + lane] = s * p.scale;
  }
}

// ------------------------------------------------------------------- routing, gradient
// With q the scores, d = scale * dL/dw of the chosen experts and, renormalised,
// w_j = scale * q_j / S with S the sum of the chosen scores and p_j = q_j / S:
//   softmax, renormalised:  dx_j = d_j' p_j,  d_j' = d_j - sum p d       (chosen only)
//   softmax:                dx_i = q_i (d_i - sum_m q_m d_m)             (every expert)
//   sigmoid, renormalised:  dx_j = q_j (1 - q_j) (d_j - sum p d) / S     (chosen only)
//   sigmoid:                dx_j = q_j (1 - q_j) d_j                     (chosen only)
// A warp builds its token's row in shared memory and writes it in 16-byte pieces where
// rows are 16-byte aligned.
struct RouteGradParams {
  const void* logits;
  const int32_t* ids;
  const float* dweights;
  int64_t T;
  int E, k;
  int sigmoid, renormalize;
  float scale;
  void* dlogits;
};

template <bool F32, bool VEC>
__global__ void __launch_bounds__(128) route_grad_kernel(const RouteGradParams p) {
  extern __shared__ __align__(16) float smem[];
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const int ld = (p.E + 7) & ~7;
  float* row = smem + (threadIdx.x >> 5) * ld;
  int id = lane < p.k ? p.ids[t * p.k + lane] : -1;
  if (id >= p.E) id = -1;
  const float d = id >= 0 ? p.scale * p.dweights[t * p.k + lane] : 0.f;
  const float x = id >= 0 ? clean_logit(load_elem<F32>(p.logits, t * p.E + id)) : -INFINITY;
  float out = 0.f;
  const bool every = !p.sigmoid && !p.renormalize;
  if (!p.sigmoid && p.renormalize) {
    float mx = warp_max(x);
    if (mx == -INFINITY) mx = 0.f;
    float e = expf(x - mx);
    const float sum = warp_sum(e);
    e = sum > 0.f ? e / sum : 0.f;
    out = e * (d - warp_sum(e * d));
  } else if (p.sigmoid) {
    const float q = x == -INFINITY ? 0.f : sigmoid(x);
    float g = d;
    if (p.renormalize) {
      const float sum = warp_sum(q);
      g = sum > 0.f ? (d - warp_sum(q / sum * d)) / sum : 0.f;
    }
    // 1 - q as 1 / (1 + e^x): no cancellation for large logits
    out = x == -INFINITY ? 0.f : q * sigmoid(-x) * g;
  }
  if (every) {
    float mx = -INFINITY;
    for (int e = lane; e < p.E; e += 32) {
      const float v = clean_logit(load_elem<F32>(p.logits, t * p.E + e));
      row[e] = v;
      mx = fmaxf(mx, v);
    }
    mx = warp_max(mx);
    if (mx == -INFINITY) mx = 0.f;
    float sum = 0.f;
    for (int e = lane; e < p.E; e += 32) {
      const float v = expf(row[e] - mx);
      row[e] = v;
      sum += v;
    }
    sum = warp_sum(sum);
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    const float q = x == -INFINITY ? 0.f : expf(x - mx) * inv;
    const float dot = warp_sum(q * d);
    out = q * (d - dot);
    for (int e = lane; e < p.E; e += 32) row[e] = -row[e] * inv * dot;
  } else {
    for (int e = lane; e < ld; e += 32) row[e] = 0.f;
  }
  __syncwarp();
  if (id >= 0) row[id] = out;
  __syncwarp();
  if constexpr (VEC) {
    if constexpr (F32) {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.dlogits) + t * p.E);
      for (int v = lane; v < p.E / 4; v += 32) o[v] = reinterpret_cast<const float4*>(row)[v];
    } else {
      uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.dlogits) + t * p.E);
      for (int v = lane; v < p.E / 8; v += 32) {
        const float4 a = reinterpret_cast<const float4*>(row)[2 * v];
        const float4 b = reinterpret_cast<const float4*>(row)[2 * v + 1];
        o[v] = make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w), pack_bf16x2(b.x, b.y),
                          pack_bf16x2(b.z, b.w));
      }
    }
  } else {
    for (int e = lane; e < p.E; e += 32) store_elem<F32>(p.dlogits, t * p.E + e, row[e]);
  }
}

// ------------------------------------------------------------------------ expert order
// A stable counting sort of the S = T * k slots by expert.  A block ranks kSlots
// consecutive slots: each of its warps walks its own share 32 slots at a time, finds the
// lanes with the same expert from one ballot per bit of the id (a fixed cost, whatever the
// ids), and counts in its own shared-memory histogram, so no atomics and no order of
// arrival enters a rank.
constexpr int kPlanThreads = 256;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanSlots = 4096;

struct PlanParams {
  const int32_t* ids;
  int64_t S;
  int E, bits, blocks;
  int32_t* block_hist;   // [E][blocks]: counts, then their exclusive prefix over blocks
  int32_t* totals;       // [E]
  int64_t* m_sizes;
  int32_t* src;
  int32_t* pos;
};

// Ranks the block's slots; each thread's ranks go through `emit(slot, id, rank)` after the
// warps' histograms have been prefix-summed.  hist: [kPlanWarps][E] counters.
template <typename Count, typename Emit>
__device__ __forceinline__ void rank_slots(const PlanParams& p, int64_t s0, int32_t* hist,
                                           Count count, Emit emit) {
  constexpr int kRows = kPlanSlots / kPlanWarps / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < kPlanWarps * p.E; i += kPlanThreads) hist[i] = 0;
  __syncthreads();
  int32_t* h = hist + warp * p.E;
  int id[kRows], rank[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int64_t s = s0 + warp * (kRows * 32) + r * 32 + lane;
    int e = s < p.S ? p.ids[s] : -1;
    id[r] = e < 0 || e >= p.E ? -1 : e;
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    uint32_t peers = __ballot_sync(kFull, id[r] >= 0);
    for (int b = 0; b < p.bits; ++b) {
      const bool bit = (id[r] >> b) & 1;
      const uint32_t v = __ballot_sync(kFull, bit);
      peers &= bit ? v : ~v;
    }
    rank[r] = 0;
    if (id[r] >= 0) rank[r] = h[id[r]] + __popc(peers & ((1u << lane) - 1u));
    __syncwarp();
    if (id[r] >= 0 && (peers >> lane) == 1u) h[id[r]] = rank[r] + 1;   // the last of its peers
    __syncwarp();
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += kPlanThreads) {
    int32_t sum = 0;
#pragma unroll
    for (int w = 0; w < kPlanWarps; ++w) {
      const int32_t c = hist[w * p.E + e];
      hist[w * p.E + e] = sum;
      sum += c;
    }
    count(e, sum);
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int64_t s = s0 + warp * (kRows * 32) + r * 32 + lane;
    if (s < p.S) emit(s, id[r], id[r] >= 0 ? h[id[r]] + rank[r] : -1);
  }
}

// Exclusive prefix of n <= 1024 counts in shared memory (in place), by every thread of the
// block; returns the total.
__device__ __forceinline__ int32_t block_prefix(int32_t* v, int n, int32_t* warp_sums) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kPer = 1024 / kPlanThreads;
  int32_t x[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = threadIdx.x * kPer + i;
    x[i] = e < n ? v[e] : 0;
    sum += x[i];
  }
  int32_t inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t y = __shfl_up_sync(kFull, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  int32_t base = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kPlanWarps; ++w) {
    if (w < warp) base += warp_sums[w];
    total += warp_sums[w];
  }
  base += inc - sum;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = threadIdx.x * kPer + i;
    if (e < n) v[e] = base;
    base += x[i];
  }
  __syncthreads();
  return total;
}

// All of it in one block (S <= kPlanSlots).
__global__ void __launch_bounds__(kPlanThreads) plan_one_kernel(const PlanParams p) {
  extern __shared__ int32_t smem_i[];
  int32_t* start = smem_i + kPlanWarps * p.E;
  __shared__ int32_t warp_sums[kPlanWarps];
  int32_t total = 0;
  // the expert starts are known only after the counts, before the ranks are emitted
  rank_slots(
      p, 0, smem_i,
      [&](int e, int32_t n) {
        start[e] = n;
        p.m_sizes[e] = n;
      },
      [&](int64_t s, int id, int32_t rank) { p.pos[s] = rank < 0 ? -1 : rank; });
  __syncthreads();
  total = block_prefix(start, p.E, warp_sums);
  for (int64_t s = threadIdx.x; s < p.S; s += kPlanThreads) {
    const int id = p.ids[s];
    if (id >= 0 && id < p.E) {
      const int32_t at = start[id] + p.pos[s];
      p.pos[s] = at;
      p.src[at] = static_cast<int32_t>(s);
    }
    if (s >= total) p.src[s] = -1;
  }
}

__global__ void __launch_bounds__(kPlanThreads) plan_rank_kernel(const PlanParams p) {
  extern __shared__ int32_t smem_i[];
  rank_slots(
      p, static_cast<int64_t>(blockIdx.x) * kPlanSlots, smem_i,
      [&](int e, int32_t n) { p.block_hist[static_cast<int64_t>(e) * p.blocks + blockIdx.x] = n; },
      [&](int64_t s, int, int32_t rank) { p.pos[s] = rank; });
}

// One warp per expert: exclusive prefix of its counts over the blocks.
__global__ void __launch_bounds__(128) plan_scan_kernel(const PlanParams p) {
  const int lane = threadIdx.x & 31;
  const int e = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (e >= p.E) return;
  int32_t* h = p.block_hist + static_cast<int64_t>(e) * p.blocks;
  int32_t base = 0;
  for (int b0 = 0; b0 < p.blocks; b0 += 32) {
    const int b = b0 + lane;
    const int32_t c = b < p.blocks ? h[b] : 0;
    int32_t inc = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t y = __shfl_up_sync(kFull, inc, o);
      if (lane >= o) inc += y;
    }
    if (b < p.blocks) h[b] = base + inc - c;
    base += __shfl_sync(kFull, inc, 31);
  }
  if (lane == 0) {
    p.totals[e] = base;
    p.m_sizes[e] = base;
  }
}

__global__ void __launch_bounds__(kPlanThreads) plan_place_kernel(const PlanParams p) {
  __shared__ int32_t start[1024];
  __shared__ int32_t warp_sums[kPlanWarps];
  for (int e = threadIdx.x; e < p.E; e += kPlanThreads) start[e] = p.totals[e];
  __syncthreads();
  const int32_t total = block_prefix(start, p.E, warp_sums);
  for (int e = threadIdx.x; e < p.E; e += kPlanThreads)
    start[e] += p.block_hist[static_cast<int64_t>(e) * p.blocks + blockIdx.x];
  __syncthreads();
  const int64_t s0 = static_cast<int64_t>(blockIdx.x) * kPlanSlots;
  for (int i = threadIdx.x; i < kPlanSlots; i += kPlanThreads) {
    const int64_t s = s0 + i;
    if (s >= p.S) break;
    const int id = p.ids[s];
    if (id >= 0 && id < p.E) {
      const int32_t at = start[id] + p.pos[s];
      p.pos[s] = at;
      p.src[at] = static_cast<int32_t>(s);
    }
    if (s >= total) p.src[s] = -1;
  }
}

// ------------------------------------------------------------------------ weighted sum
// 16 bytes of a row as FP32: 4 (FP32) or 8 (BF16) values.
template <bool F32>
struct Vec {
  static constexpr int kN = F32 ? 4 : 8;
  uint4 r;
  __device__ __forceinline__ float get(int i) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    if constexpr (F32)
      return __uint_as_float(w[i]);
    else
      return __uint_as_float((i & 1) ? (w[i >> 1] & 0xFFFF0000u) : (w[i >> 1] << 16));
  }
};
template <bool F32>
__device__ __forceinline__ uint4 pack_vec(const float* v) {
  if constexpr (F32)
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                      __float_as_uint(v[3]));
  else
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
}

struct CombineParams {
  const void* y;
  const int32_t* pos;
  const float* weights;   // nullptr: all one
  const int32_t* src;     // gradient only
  const void* dout;       // gradient only
  void* out;              // the sum, or dY
  float* dweights;        // gradient only; may be nullptr
  int64_t T, R;
  int k, vecs;            // 16-byte pieces of a row
};

// A thread owns one 16-byte piece of one token's output and has up to kUnroll rows' pieces
// in flight; the sum runs over the token's slots in order.
template <bool F32>
__global__ void __launch_bounds__(128) combine_kernel(const CombineParams p) {
  constexpr int kUnroll = 8, kN = Vec<F32>::kN;
  const int64_t t = blockIdx.x;
  const int v = blockIdx.y * 128 + threadIdx.x;
  if (v >= p.vecs) return;
  const uint4* y = static_cast<const uint4*>(p.y);
  float acc[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) acc[i] = 0.f;
  for (int j0 = 0; j0 < p.k; j0 += kUnroll) {
    Vec<F32> x[kUnroll];
    float w[kUnroll];
    bool used[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int j = j0 + u;
      const int32_t r = j < p.k ? p.pos[t * p.k + j] : -1;
      used[u] = r >= 0 && r < p.R;
      if (used[u]) {
        w[u] = p.weights ? p.weights[t * p.k + j] : 1.f;
        x[u].r = __ldcs(y + static_cast<int64_t>(r) * p.vecs + v);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (used[u])
#pragma unroll
        for (int i = 0; i < kN; ++i) acc[i] = fmaf(w[u], x[u].get(i), acc[i]);
  }
  static_cast<uint4*>(p.out)[t * p.vecs + v] = pack_vec<F32>(acc);
}

// One block per token: dY of its rows is w * dout, dw the dot product of dout and the row.
// The token's dout pieces are read once per kSlots slots.
template <bool F32>
__global__ void __launch_bounds__(256) combine_grad_kernel(const CombineParams p) {
  constexpr int kN = Vec<F32>::kN, kSlots = 8;
  __shared__ float part[8][kSlots];
  const int64_t t = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint4* y = static_cast<const uint4*>(p.y);
  const uint4* dout = static_cast<const uint4*>(p.dout) + t * p.vecs;
  uint4* dy = static_cast<uint4*>(p.out);
  for (int j0 = 0; j0 < p.k; j0 += kSlots) {
    float dot[kSlots], w[kSlots];
    int32_t r[kSlots];
#pragma unroll
    for (int u = 0; u < kSlots; ++u) {
      const int j = j0 + u;
      r[u] = j < p.k ? p.pos[t * p.k + j] : -1;
      if (r[u] >= p.R) r[u] = -1;
      w[u] = r[u] >= 0 ? (p.weights ? p.weights[t * p.k + j] : 1.f) : 0.f;
      dot[u] = 0.f;
    }
    for (int v = threadIdx.x; v < p.vecs; v += 256) {
      Vec<F32> d;
      d.r = dout[v];
      Vec<F32> x[kSlots];
      if (p.dweights)
#pragma unroll
        for (int u = 0; u < kSlots; ++u)
          if (r[u] >= 0) x[u].r = __ldcs(y + static_cast<int64_t>(r[u]) * p.vecs + v);
#pragma unroll
      for (int u = 0; u < kSlots; ++u)
        if (r[u] >= 0) {
          float o[kN];
#pragma unroll
          for (int i = 0; i < kN; ++i) o[i] = w[u] * d.get(i);
          __stcs(dy + static_cast<int64_t>(r[u]) * p.vecs + v, pack_vec<F32>(o));
          if (p.dweights)
#pragma unroll
            for (int i = 0; i < kN; ++i) dot[u] = fmaf(d.get(i), x[u].get(i), dot[u]);
        }
    }
    if (p.dweights) {
#pragma unroll
      for (int u = 0; u < kSlots; ++u) {
        const float s = warp_sum(dot[u]);
        if (lane == 0) part[warp][u] = s;
      }
      __syncthreads();
      if (threadIdx.x < kSlots && j0 + static_cast<int>(threadIdx.x) < p.k) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += part[i][threadIdx.x];
        p.dweights[t * p.k + j0 + threadIdx.x] = s;
      }
      __syncthreads();
    }
  }
  // rows that no slot uses have no gradient
  for (int j = 0; j < p.k; ++j) {
    const int64_t row = t * p.k + j;
    if (p.src[row] < 0)
      for (int v = threadIdx.x; v < p.vecs; v += 256) dy[row * p.vecs + v] = make_uint4(0, 0, 0, 0);
  }
}

template <bool F32, int V>
bsmma_status launch_route_v(const RouteParams& p, cudaStream_t stream) {
  // a few tokens: one warp per block, so that they spread over the SMs
  const int warps = p.T >= 1024 ? 4 : 1;
  const bool staged = p.groups > 1;
  route_kernel<F32, V><<<static_cast<unsigned>((p.T + warps - 1) / warps), warps * 32,
                         staged ? warps * p.E * 4 : 0, stream>>>(p);
  count_launches(1);
  return cuda_ok(cudaGetLastError());
}
template <bool F32>
bsmma_status launch_route_t(const RouteParams& p, cudaStream_t stream) {
  if (p.E <= 32) return launch_route_v<F32, 1>(p, stream);
  if (p.E <= 64) return launch_route_v<F32, 2>(p, stream);
  if (p.E <= 128) return launch_route_v<F32, 4>(p, stream);
  if (p.E <= 256) return launch_route_v<F32, 8>(p, stream);
  if (p.E <= 512) return launch_route_v<F32, 16>(p, stream);
  return launch_route_v<F32, 32>(p, stream);
}

int bits_for(int E) {
  int b = 0;
  while ((1 << b) < E) ++b;
  return b;
}

}  // namespace

bsmma_status launch_route(const void* logits, bool f32, int64_t T, int E, int k, bool sigmoid,
                          const float* bias, int groups, int topk_groups, int group_top,
                          bool renormalize, float scale, int32_t* ids, float* weights,
                          cudaStream_t stream) {
  RouteParams p;
  p.logits = logits;
  p.bias = bias;
  p.T = T;
  p.E = E;
  p.k = k;
  p.groups = topk_groups < groups ? groups : 1;   // every group open: no group step
  p.topk_groups = topk_groups;
  p.group_top = group_top;
  p.sigmoid = sigmoid;
  p.renormalize = renormalize;
  p.scale = scale;
  p.ids = ids;
  p.weights = weights;
  return f32 ? launch_route_t<true>(p, stream) : launch_route_t<false>(p, stream);
}

bsmma_status launch_route_backward(const void* logits, bool f32, int64_t T, int E, int k,
                                   bool sigmoid, bool renormalize, float scale, const int32_t* ids,
                                   const float* dweights, void* dlogits, cudaStream_t stream) {
  RouteGradParams p;
  p.logits = logits;
  p.ids = ids;
  p.dweights = dweights;
  p.T = T;
  p.E = E;
  p.k = k;
  p.sigmoid = sigmoid;
  p.renormalize = renormalize;
  p.scale = scale;
  p.dlogits = dlogits;
  const int warps = T >= 1024 ? 4 : 1;
  const unsigned grid = static_cast<unsigned>((T + warps - 1) / warps);
  const int smem = warps * ((E + 7) & ~7) * 4;
  const bool vec = E % (f32 ? 4 : 8) == 0;
  if (f32) {
    if (vec)
      route_grad_kernel<true, true><<<grid, warps * 32, smem, stream>>>(p);
    else
      route_grad_kernel<true, false><<<grid, warps * 32, smem, stream>>>(p);
  } else {
    if (vec)
      route_grad_kernel<false, true><<<grid, warps * 32, smem, stream>>>(p);
    else
      route_grad_kernel<false, false><<<grid, warps * 32, smem, stream>>>(p);
  }
  count_launches(1);
  return cuda_ok(cudaGetLastError());
}

int64_t plan_workspace_bytes(int64_t S, int E) {
  if (S <= kPlanSlots) return 0;
  const int64_t blocks = (S + kPlanSlots - 1) / kPlanSlots;
  return (blocks + 1) * E * 4;
}

bsmma_status launch_plan(const int32_t* ids, int64_t S, int E, int64_t* m_sizes, int32_t* src,
                         int32_t* pos, void* workspace, cudaStream_t stream) {
  PlanParams p;
  p.ids = ids;
  p.S = S;
  p.E = E;
  p.bits = bits_for(E);
  p.blocks = static_cast<int>((S + kPlanSlots - 1) / kPlanSlots);
  p.totals = static_cast<int32_t*>(workspace);
  p.block_hist = p.totals ? p.totals + E : nullptr;
  p.m_sizes = m_sizes;
  p.src = src;
  p.pos = pos;
  if (S <= kPlanSlots) {
    plan_one_kernel<<<1, kPlanThreads, (kPlanWarps + 1) * E * 4, stream>>>(p);
    count_launches(1);
    return cuda_ok(cudaGetLastError());
  }
  plan_rank_kernel<<<p.blocks, kPlanThreads, kPlanWarps * E * 4, stream>>>(p);
  plan_scan_kernel<<<(E + 3) / 4, 128, 0, stream>>>(p);
  plan_place_kernel<<<p.blocks, kPlanThreads, 0, stream>>>(p);
  count_launches(3);
  return cuda_ok(cudaGetLastError());
}

bsmma_status launch_combine(const void* y, bool f32, int64_t R, int64_t H, const int32_t* pos,
                            const float* weights, int64_t T, int k, void* out,
                            cudaStream_t stream) {
  CombineParams p = {};
  p.y = y;
  p.pos = pos;
  p.weights = weights;
  p.out = out;
  p.T = T;
  p.R = R;
  p.k = k;
  p.vecs = static_cast<int>(H / (f32 ? 4 : 8));
  const dim3 grid(static_cast<unsigned>(T), static_cast<unsigned>((p.vecs + 127) / 128));
  if (f32)
    combine_kernel<true><<<grid, 128, 0, stream>>>(p);
  else
    combine_kernel<false><<<grid, 128, 0, stream>>>(p);
  count_launches(1);
  return cuda_ok(cudaGetLastError());
}

bsmma_status launch_combine_backward(const void* dout, bool f32, int64_t H, const void* y,
                                     const int32_t* src, const int32_t* pos, const float* weights,
                                     int64_t T, int k, void* dy, float* dweights,
                                     cudaStream_t stream) {
  CombineParams p = {};
  p.y = y;
  p.pos = pos;
  p.weights = weights;
  p.src = src;
  p.dout = dout;
  p.out = dy;
  p.dweights = dweights;
  p.T = T;
  p.R = T * k;
  p.k = k;
  p.vecs = static_cast<int>(H / (f32 ? 4 : 8));
  if (f32)
    combine_grad_kernel<true><<<static_cast<unsigned>(T), 256, 0, stream>>>(p);
  else
    combine_grad_kernel<false><<<static_cast<unsigned>(T), 256, 0, stream>>>(p);
  count_launches(1);
  return cuda_ok(cudaGetLastError());
}

}  // namespace bsmma
