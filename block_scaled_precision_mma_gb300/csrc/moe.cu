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
#include <type_traits>

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

// A chosen expert's score over e^m (softmax) or over e^min(m, 0) (sigmoid), with m the largest
// chosen logit: renormalised weights are quotients of these, so that scores below FP32's range
// keep their ratios.  A sigmoid below 2^-1022 is 0, in 64 bits too: an expert masked by the
// type's lowest value.
constexpr float kVanished = -708.f;
__device__ __forceinline__ float renorm_score(bool of_sigmoid, float x, float m) {
  if (!of_sigmoid) return expf(x - m);
  if (m >= 0.f) return sigmoid(x);
  return x < kVanished ? 0.f : expf(x - m) / (1.f + expf(x));
}

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

// The largest x of the lanes that have one (not NaN), by one reduction.
__device__ __forceinline__ float warp_largest(bool have, float x) {
  const uint32_t o = __reduce_max_sync(kFull, have ? ordered(x) : 0u);
  return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}

// ------------------------------------------------------------------------- routing
// One warp per token, V experts a lane.  The k choices are k rounds of a warp-wide maximum.
// Instructions bound it, not its bytes (a token of 128 experts is 256 bytes), so a round is
// kept short: each lane holds the best of its own keys, and only what the round took changes.
struct RouteParams {
  const void* logits;
  const float* bias;
  int64_t T;
  int E, k, groups, topk_groups, group_top;
  uint32_t per_magic;   // e * per_magic >> 32 is e / (E / groups) for e < 1024
  int sigmoid, renormalize;
  float scale;
  int32_t* ids;
  float* weights;
};

// The weights of the chosen: lane j has the j-th's logit x (id -1: none).
__device__ __forceinline__ void write_choice(const RouteParams& p, int64_t t, int id, float x,
                                             float mx, float denom) {
  const int lane = threadIdx.x & 31;
  float s = 0.f;
  if (p.renormalize) {
    const float m = warp_largest(id >= 0, x);
    if (id >= 0) s = renorm_score(p.sigmoid, x, m);
    const float sum = warp_sum(s);
    s = sum > 0.f ? s / sum : 0.f;
  } else if (id >= 0) {
    s = p.sigmoid ? sigmoid(x) : expf(x - mx) / denom;
  }
  if (lane < p.k) {
    p.ids[t * p.k + lane] = id;
    p.weights[t * p.k + lane] = s * p.scale;
  }
}

// Both score functions increase with the logit, so without a bias the keys are the logits
// themselves and no rounding of a score can reorder the choice.  A BF16 logit's ordered 16
// bits and the complement of its index make one 32-bit key: one reduction finds the largest
// and, among equals, the lowest index.  Lane l holds experts 64 j + 2 l + {0, 1} (E even: pairs
// are 4-byte loads) or 32 j + l.
template <int V, bool PAIRS>
__global__ void __launch_bounds__(128) route_bf16_kernel(const RouteParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const uint16_t* row = static_cast<const uint16_t*>(p.logits) + t * p.E;
  uint32_t key[V];   // 0: closed or taken
#pragma unroll
  for (int i = 0; i < V; ++i) key[i] = 0;
  auto key_of = [](uint32_t bits, int e) {
    if ((bits & 0x7FFFu) > 0x7F80u || bits == 0xFF80u) return 0u;   // NaN, -inf
    if (bits == 0x8000u) bits = 0;                                  // -0 and +0 are one key
    const uint32_t o = (bits & 0x8000u) ? ~bits & 0xFFFFu : bits | 0x8000u;
    return o << 16 | static_cast<uint32_t>(0xFFFF - e);
  };
  if constexpr (PAIRS) {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const int e = 32 * i + 2 * lane;
      if (e < p.E) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(row + e);
        key[i] = key_of(w & 0xFFFFu, e);
        key[i + 1] = key_of(w >> 16, e + 1);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (32 * i + lane < p.E) key[i] = key_of(row[32 * i + lane], 32 * i + lane);
  }
  auto logit = [](uint32_t k) {
    const uint32_t o = k >> 16;
    return fminf(__uint_as_float((o & 0x8000u ? o & 0x7FFFu : ~o & 0xFFFFu) << 16), FLT_MAX);
  };
  uint32_t best = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) best = max(best, key[i]);
  uint32_t mine = 0, first = 0;   // lane j keeps the j-th choice
  for (int j = 0; j < p.k; ++j) {
    const uint32_t top = __reduce_max_sync(kFull, best);
    if (top == 0) break;
    if (j == 0) first = top;
    if (lane == j) mine = top;
    if (best == top) {
      best = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (key[i] == top) key[i] = 0;
        best = max(best, key[i]);
      }
    }
  }
  const float mx = first ? logit(first) : 0.f;
  float denom = 1.f;
  if (!p.sigmoid && !p.renormalize) {
    float sum = 0.f;   // the chosen are 0 in key[] by now: theirs come from `mine`
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (key[i]) sum += expf(logit(key[i]) - mx);
    if (mine) sum += expf(logit(mine) - mx);
    sum = warp_sum(sum);
    denom = sum > 0.f ? sum : 1.f;
  }
  write_choice(p, t, mine ? 0xFFFF - static_cast<int>(mine & 0xFFFFu) : -1, mine ? logit(mine) : 0.f, mx,
               denom);
}

// The same keys for many tokens: four lanes a token, eight tokens a warp, when k <= 8 and the
// rows are whole 64-byte pieces.  A lane keeps the eight largest keys of its experts in
// order: it sorts eight new ones (19 exchanges of a maximum and a minimum) and merges them in
// (eight maxima, 12 exchanges); two more merges across the four lanes leave all of them with
// the token's eight.  96 warp instructions a token at 128 experts against 440 for the rounds
// above: 65536 tokens 13 us against 34, both bound by issuing (56% of the slots; the 21 MB are
// 3 us).  From 1024 tokens on: there 2.8 us against 3.3 in launches one after another, at 4096
// 2.7 and 4.2; fewer take 2.4 to 2.8 us either way (64 experts, 64 tokens: 2.8 against 2.6).
// Softmax without renormalisation needs the row's sum as well, k above 8 more keys kept, and
// other E a ragged last piece: those stay with the rounds (65536 x 128 without renormalisation
// 36 us, with k = 12 41 us, of 100 experts 34 us).
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return max(a, b); }
__device__ __forceinline__ uint64_t larger(uint64_t a, uint64_t b) { return a > b ? a : b; }
__device__ __forceinline__ void exchange(uint32_t& a, uint32_t& b) {
  const uint32_t hi = max(a, b);
  b = min(a, b);
  a = hi;
}
__device__ __forceinline__ void exchange(uint64_t& a, uint64_t& b) {
  const bool swap = b > a;
  const uint64_t hi = swap ? b : a;
  b = swap ? a : b;
  a = hi;
}
template <typename Key>
__device__ __forceinline__ void sort8(Key (&v)[8]) {
  exchange(v[0], v[1]); exchange(v[2], v[3]); exchange(v[4], v[5]); exchange(v[6], v[7]);
  exchange(v[0], v[2]); exchange(v[1], v[3]); exchange(v[4], v[6]); exchange(v[5], v[7]);
  exchange(v[1], v[2]); exchange(v[5], v[6]);
  exchange(v[0], v[4]); exchange(v[1], v[5]); exchange(v[2], v[6]); exchange(v[3], v[7]);
  exchange(v[2], v[4]); exchange(v[3], v[5]);
  exchange(v[1], v[2]); exchange(v[3], v[4]); exchange(v[5], v[6]);
}
// v: first rising then falling or the other way round -> in falling order.
template <typename Key>
__device__ __forceinline__ void merge8(Key (&v)[8]) {
#pragma unroll
  for (int d = 4; d; d >>= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!(i & d)) exchange(v[i], v[i + d]);
}

__global__ void __launch_bounds__(128) route_quad_kernel(const RouteParams p) {
  const int lane = threadIdx.x & 31, q = lane & 3;
  const int64_t t = (static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x) >> 2;
  const bool in = t < p.T;
  const uint4* row =
      reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.logits) + (in ? t : 0) * p.E);
  uint32_t top[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) top[i] = 0;
#pragma unroll 4
  for (int b = q; b < p.E / 8; b += 4) {
    const uint4 w4 = row[b];
    const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
    const uint32_t low = 0xFFFF - 8 * b;
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // NaN becomes -inf, -0 becomes +0
      const float f = fmaxf(__uint_as_float(i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16), -INFINITY) + 0.f;
      const uint32_t bits = __float_as_uint(f);
      const uint32_t o = bits ^ (static_cast<uint32_t>(static_cast<int32_t>(bits) >> 31) | 0x80000000u);
      v[i] = (o & 0xFFFF0000u) | (low - i);
    }
    sort8(v);
#pragma unroll
    for (int i = 0; i < 8; ++i) top[i] = max(top[i], v[7 - i]);
    merge8(top);
  }
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = max(top[i], __shfl_xor_sync(kFull, top[7 - i], o));
    merge8(v);
#pragma unroll
    for (int i = 0; i < 8; ++i) top[i] = v[i];
  }
  constexpr uint32_t kClosed = 0x00800000u;   // keys of -inf are below
  auto logit = [](uint32_t k) {
    const uint32_t o = k >> 16;
    return fminf(__uint_as_float((o & 0x8000u ? o & 0x7FFFu : ~o & 0xFFFFu) << 16), FLT_MAX);
  };
  // lane q finishes choices q and q + 4
  const float mx = top[0] >= kClosed ? logit(top[0]) : 0.f;
  uint32_t c[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = q & 1 ? top[4 * h + 1] : top[4 * h], hi = q & 1 ? top[4 * h + 3] : top[4 * h + 2];
    c[h] = q & 2 ? hi : lo;
    if (q + 4 * h >= p.k || c[h] < kClosed) c[h] = 0;
  }
  float s[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float x = logit(c[h]);
    s[h] = c[h] ? (p.renormalize ? renorm_score(p.sigmoid, x, mx) : sigmoid(x)) : 0.f;
  }
  if (p.renormalize) {
    float sum = s[0] + s[1];
    sum += __shfl_xor_sync(kFull, sum, 1);
    sum += __shfl_xor_sync(kFull, sum, 2);
#pragma unroll
    for (int h = 0; h < 2; ++h) s[h] = sum > 0.f ? s[h] / sum : 0.f;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (in && q + 4 * h < p.k) {
      p.ids[t * p.k + q + 4 * h] = c[h] ? 0xFFFF - static_cast<int>(c[h] & 0xFFFFu) : -1;
      p.weights[t * p.k + q + 4 * h] = s[h] * p.scale;
    }
}

// FP32 logits, a bias or groups, many tokens: the same with 64-bit keys, a key's 32 bits above the
// complement of its index, and eight lanes a token.  Each lane's experts belong to one group
// (1, 2, 4 or 8 of them, whole pieces of eight experts), so that the lanes of a group come to
// its largest keys, which value it, before the other groups' lists are merged in and a closed
// group's list is empty.  Bound by issuing, 66% of the slots, most of it to the integer pipe (a
// 64-bit exchange is two compares and four selects): 65536 tokens of 256 experts with a bias and 8 groups 72 us, 105 with a warp a token
// and rounds; 128 FP32 experts 39 and 52.  16384 tokens 26 and 33; at 8192 both take 19 to 21 and
// below a token's longer chain shows, so the rounds keep those.
struct Logits8 {
  float x[8];
};
template <bool F32>
__device__ __forceinline__ Logits8 load_logits8(const void* logits, int64_t at) {
  Logits8 r;
  if constexpr (F32) {
    const float4* from = reinterpret_cast<const float4*>(static_cast<const float*>(logits) + at);
    const float4 a = from[0], b = from[1];
    const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) r.x[i] = clean_logit(v[i]);
  } else {
    const uint4 w4 = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(logits) + at);
    const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      r.x[i] = clean_logit(__uint_as_float(i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16));
  }
  return r;
}
__device__ __forceinline__ float of_key(uint64_t key) {
  const uint32_t o = static_cast<uint32_t>(key >> 32);
  return key == 0 ? -INFINITY : __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
// The eight largest keys of the lane and its partner, o lanes away, in both.
__device__ __forceinline__ void merge_lanes(uint64_t (&top)[8], int o) {
  uint64_t v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = larger(top[i], __shfl_xor_sync(kFull, top[7 - i], o));
  merge8(v);
#pragma unroll
  for (int i = 0; i < 8; ++i) top[i] = v[i];
}

template <bool F32>
__global__ void __launch_bounds__(128) route_eight_kernel(const RouteParams p) {
  const int q = threadIdx.x & 7;
  const int64_t t_of = (static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x) >> 3;
  const bool in = t_of < p.T;
  const int64_t t = in ? t_of : p.T - 1;
  const int per = p.E / p.groups, share = 8 / p.groups;   // a group's experts and lanes
  const int g = q / share, e0 = g * per;
  const int64_t row = t * p.E;
  auto segment_max = [](float v) {
#pragma unroll
    for (int o = 4; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
  };
  auto segment_sum = [](float v) {
#pragma unroll
    for (int o = 4; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
  };
  float mx = -INFINITY, denom = 1.f;
  // the scores' denominator, with mx known
  auto sum_scores = [&] {
    float sum = 0.f;
    for (int e = e0 + 8 * (q % share); e < e0 + per; e += 8 * share) {
      const Logits8 l = load_logits8<F32>(p.logits, row + e);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += expf(l.x[i] - mx);
    }
    sum = segment_sum(sum);
    denom = sum > 0.f ? sum : 1.f;
  };
  auto score = [&](float x) { return p.sigmoid ? sigmoid(x) : expf(x - mx) / denom; };
  const bool values = p.groups > 1 && p.group_top > 1;   // groups by the sum of two scores
  const bool before = !p.sigmoid && (p.bias || values);
  if (before) {
    for (int e = e0 + 8 * (q % share); e < e0 + per; e += 8 * share) {
      const Logits8 l = load_logits8<F32>(p.logits, row + e);
#pragma unroll
      for (int i = 0; i < 8; ++i) mx = fmaxf(mx, l.x[i]);
    }
    mx = segment_max(mx);
    if (mx == -INFINITY) mx = 0.f;
    sum_scores();
  }

  uint64_t top[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) top[i] = 0;
  for (int e = e0 + 8 * (q % share); e < e0 + per; e += 8 * share) {
    const Logits8 l = load_logits8<F32>(p.logits, row + e);
    float bias[8];
    if (p.bias) {
      const float4 a = *reinterpret_cast<const float4*>(p.bias + e), b = *reinterpret_cast<const float4*>(p.bias + e + 4);
      bias[0] = a.x, bias[1] = a.y, bias[2] = a.z, bias[3] = a.w;
      bias[4] = b.x, bias[5] = b.y, bias[6] = b.z, bias[7] = b.w;
    }
    uint64_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float key = l.x[i];
      if (p.bias && key != -INFINITY) {
        key = score(key) + bias[i];
        if (key != key) key = -INFINITY;
      }
      v[i] = key == -INFINITY ? 0 : static_cast<uint64_t>(ordered(key)) << 32 | (0xFFFFFFFFu - (e + i));
    }
    sort8(v);
    if (e < e0 + 8 * share) {   // the lane's first
#pragma unroll
      for (int i = 0; i < 8; ++i) top[i] = v[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) top[i] = larger(top[i], v[7 - i]);
      merge8(top);
    }
  }
  for (int o = 1; o < share; o <<= 1) merge_lanes(top, o);
  if (p.groups > 1) {
    // value of a group: the sum of its group_top largest; open when fewer than topk_groups are
    // ahead of it (ties: lower index first)
    float value = of_key(top[0]), second = of_key(top[1]);
    if (values) {
      if (!p.bias) {
        if (value != -INFINITY) value = score(value);
        if (second != -INFINITY) second = score(second);
      }
      if (second != -INFINITY) value += second;
    }
    int ahead = 0;
    for (int j = 0; j < p.groups; ++j) {
      const float v = __shfl_sync(kFull, value, (threadIdx.x & 24) + j * share);
      ahead += v > value || (v == value && j < g);
    }
    if (ahead >= p.topk_groups)
#pragma unroll
      for (int i = 0; i < 8; ++i) top[i] = 0;
    for (int o = share; o < 8; o <<= 1) merge_lanes(top, o);
  }

  // lane q finishes choice q
  uint64_t c = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i == q && i < p.k) c = top[i];
  const int id = static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(c));
  float x = -INFINITY;
  if (c) x = p.bias ? clean_logit(load_elem<F32>(p.logits, row + id)) : of_key(c);
  float s = 0.f;
  if (!p.renormalize) {
    if (!p.sigmoid && !before) {
      // the first choice is the largest logit: without a bias, and with groups valued by their
      // largest, its group is open
      mx = segment_max(x);
      if (mx == -INFINITY) mx = 0.f;
      sum_scores();
    }
    if (c) s = score(x);
  } else {
    const float m = segment_max(x);
    if (c) s = renorm_score(p.sigmoid, x, m);
    const float sum = segment_sum(s);
    s = sum > 0.f ? s / sum : 0.f;
  }
  if (in && q < p.k) {
    p.ids[t * p.k + q] = c ? id : -1;
    p.weights[t * p.k + q] = s * p.scale;
  }
}

// FP32 logits, a bias or groups otherwise: 32-bit keys, lane l holding experts 32 i + l.  A decoding
// step is its chain of latencies: 32 tokens of 256 experts with a bias and groups take 8.3 us
// a launch, one after another.
template <bool F32, int V>
__global__ void __launch_bounds__(128) route_kernel(const RouteParams p) {
  extern __shared__ float smem[];
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= p.T) return;
  float x[V], key[V], bias[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 32 * i;
    x[i] = -INFINITY;
    bias[i] = 0.f;
    if (e < p.E) {
      x[i] = load_elem<F32>(p.logits, t * p.E + e);
      if (p.bias) bias[i] = p.bias[e];
    }
  }
  float mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    key[i] = x[i] = clean_logit(x[i]);
    mx = fmaxf(mx, x[i]);
  }
  const bool all_scores = p.bias || (p.groups > 1 && p.group_top > 1);
  float denom = 1.f;
  if (!p.sigmoid) {
    mx = warp_max(mx);
    if (mx == -INFINITY) mx = 0.f;
    if (all_scores || !p.renormalize) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) sum += expf(x[i] - mx);
      sum = warp_sum(sum);
      denom = sum > 0.f ? sum : 1.f;
    }
  }
  float* row = smem + (threadIdx.x >> 5) * p.E;   // what a group is valued by (groups only)
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 32 * i;
    float value = x[i];
    if (all_scores && x[i] != -INFINITY) {
      value = (p.sigmoid ? sigmoid(x[i]) : expf(x[i] - mx) / denom) + bias[i];
      if (value != value) value = -INFINITY;
      if (p.bias) key[i] = value;
    }
    if (p.groups > 1 && e < p.E) row[e] = value;
  }
  if (p.groups > 1) {
    // value of a group: the sum of its group_top largest; `width` lanes (a power of two)
    // share a group
    __syncwarp();
    const int per = p.E / p.groups;
    int width = 32;
    while (width * p.groups > 32) width >>= 1;
    const int g = lane / width;
    float a = -INFINITY, b = -INFINITY;   // the group's largest and second largest
    if (g < p.groups)
#pragma unroll 4
      for (int i = lane % width; i < per; i += width) {
        const float v = row[g * per + i];
        b = fmaxf(b, fminf(a, v));
        a = fmaxf(a, v);
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
      const uint32_t e = lane + 32 * i;
      const int of = per == 1 ? static_cast<int>(e) : static_cast<int>(__umulhi(e, p.per_magic));
      if (e < p.E && !((open >> (of * width)) & 1u)) key[i] = -INFINITY;
    }
  }

  if constexpr (V == 1) {
    // up to 32 experts: every lane counts the keys ahead of its own, which is its place
    int ahead = 0;
    for (int j = 0; j < p.E; ++j) {
      const float other = __shfl_sync(kFull, key[0], j);
      ahead += other > key[0] || (other == key[0] && j < lane);
    }
    const bool chosen = key[0] != -INFINITY && ahead < p.k;
    float s = 0.f;
    if (!p.renormalize) {
      if (chosen) s = p.sigmoid ? sigmoid(x[0]) : expf(x[0] - mx) / denom;
    } else {
      const float m = warp_largest(chosen, x[0]);
      if (chosen) s = renorm_score(p.sigmoid, x[0], m);
      const float sum = warp_sum(s);
      s = sum > 0.f ? s / sum : 0.f;
    }
    if (chosen) {
      p.ids[t * p.k + ahead] = lane;
      p.weights[t * p.k + ahead] = s * p.scale;
    }
    if (lane >= __popc(__ballot_sync(kFull, chosen)) && lane < p.k) {
      p.ids[t * p.k + lane] = -1;
      p.weights[t * p.k + lane] = 0.f;
    }
    return;
  }
  uint32_t best = 0;    // of the lane's keys, in an order of unsigned integers
  int at = 0;
  float best_x = 0.f;   // its logit
  auto rescan = [&] {
    float k = -INFINITY;
    at = 0;
    best_x = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (key[i] > k) {
        k = key[i];
        at = i;
        best_x = x[i];
      }
    best = k == -INFINITY ? 0u : ordered(k);
  };
  rescan();
  int mine = -1;   // lane j keeps the j-th choice, and its logit
  float mine_x = 0.f;
  for (int j = 0; j < p.k; ++j) {
    const uint32_t top = __reduce_max_sync(kFull, best);
    if (top == 0) break;
    const uint32_t e = __reduce_min_sync(kFull, best == top ? static_cast<uint32_t>(lane + 32 * at)
                                                            : 0xFFFFFFFFu);
    const float chosen = __shfl_sync(kFull, best_x, e & 31);
    if (lane == j) {
      mine = static_cast<int>(e);
      mine_x = chosen;
    }
    if (static_cast<int>(e & 31u) == lane) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i == at) key[i] = -INFINITY;
      rescan();
    }
  }
  write_choice(p, t, mine, mine_x, mx, denom);
}

// ------------------------------------------------------------------- routing, gradient
// With q the scores, d = scale * dL/dw of the chosen experts and, renormalised,
// w_j = scale * q_j / S with S the sum of the chosen scores and p_j = q_j / S:
//   softmax, renormalised:  dx_j = d_j' p_j,  d_j' = d_j - sum p d       (chosen only)
//   softmax:                dx_i = q_i (d_i - sum_m q_m d_m)             (every expert)
//   sigmoid, renormalised:  dx_j = p_j (1 - q_j) (d_j - sum p d)         (chosen only)
//   sigmoid:                dx_j = q_j (1 - q_j) d_j                     (chosen only)
// A warp builds its token's row in shared memory, in the logits' type, and writes it in
// 16-byte pieces where rows are 16-byte aligned.
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

// EVERY: the second form, which reads the whole row, three times; the others read the chosen
// logits (65536 x 128 BF16 21 us and 7).
// LANES of a warp share a token: 8 where k <= 8, from 1024 tokens on, else 32.  128 experts, k = 8,
// launches one after another: 1024 tokens 2.4 us with 8 lanes, 2.65 with 32 lanes and four warps a
// block, 2.9 with one warp a block; 4096 tokens 2.45, 2.9 and 4.3; 64 tokens 2.05, 2.2 and 2.3,
// where one warp a block is kept for spreading over the SMs beside other kernels.
template <int LANES>
__device__ __forceinline__ float part_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
template <int LANES>
__device__ __forceinline__ float part_max(float v) {
#pragma unroll
  for (int o = LANES / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}
template <bool F32, bool EVERY, int LANES>
__global__ void __launch_bounds__(128) route_grad_kernel(const RouteGradParams p) {
  extern __shared__ __align__(16) uint8_t smem_b[];
  using Elem = typename std::conditional<F32, float, __nv_bfloat16>::type;
  const int lane = threadIdx.x % LANES;
  const int64_t t_of = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) / LANES;
  const bool in = t_of < p.T;   // (a warp's other tokens may still be)
  const int64_t t = in ? t_of : p.T - 1;
  constexpr int kPer = 16 / sizeof(Elem);
  const int pieces = (p.E + kPer - 1) / kPer;   // of the row, 16 bytes each
  Elem* row = reinterpret_cast<Elem*>(smem_b + (threadIdx.x / LANES) * pieces * 16);
  int id = lane < p.k ? p.ids[t * p.k + lane] : -1;
  if (id >= p.E) id = -1;
  float d = 0.f, x = -INFINITY;
  if (id >= 0) {
    d = p.scale * p.dweights[t * p.k + lane];
    x = clean_logit(load_elem<F32>(p.logits, t * p.E + id));
  }
  if constexpr (!EVERY)
    for (int v = lane; v < pieces; v += LANES) reinterpret_cast<uint4*>(row)[v] = make_uint4(0, 0, 0, 0);
  float out = 0.f;
  if constexpr (EVERY) {
    float mx = -INFINITY, sum = 0.f;
    for (int e = lane; e < p.E; e += LANES)
      mx = fmaxf(mx, clean_logit(load_elem<F32>(p.logits, t * p.E + e)));
    mx = part_max<LANES>(mx);
    if (mx == -INFINITY) mx = 0.f;
    for (int e = lane; e < p.E; e += LANES)
      sum += expf(clean_logit(load_elem<F32>(p.logits, t * p.E + e)) - mx);
    sum = part_sum<LANES>(sum);
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    const float q = x == -INFINITY ? 0.f : expf(x - mx) * inv;
    const float dot = part_sum<LANES>(q * d);
    out = q * (d - dot);
    for (int e = lane; e < p.E; e += LANES)
      store_elem<F32>(row, e, -expf(clean_logit(load_elem<F32>(p.logits, t * p.E + e)) - mx) * inv * dot);
  } else if (!p.sigmoid) {
    float mx = part_max<LANES>(x);
    if (mx == -INFINITY) mx = 0.f;
    float e = expf(x - mx);
    const float sum = part_sum<LANES>(e);
    e = sum > 0.f ? e / sum : 0.f;
    out = e * (d - part_sum<LANES>(e * d));
  } else {
    float q = x == -INFINITY ? 0.f : sigmoid(x);
    if (p.renormalize) {
      // q becomes p, and no sum or reciprocal of the scores leaves the range
      // (the sums outside the condition: a warp's tokens may differ in it)
      const float m = part_max<LANES>(x);
      if (x != -INFINITY) q = renorm_score(true, x, m);
      const float sum = part_sum<LANES>(q);
      q = sum > 0.f ? q / sum : 0.f;
      d -= part_sum<LANES>(q * d);
    }
    // 1 - q as 1 / (1 + e^x): no cancellation for large logits
    out = x == -INFINITY ? 0.f : q * sigmoid(-x) * d;
  }
  __syncwarp();
  if (id >= 0) store_elem<F32>(row, id, out);
  __syncwarp();
  if (!in) return;
  Elem* to = static_cast<Elem*>(p.dlogits) + t * p.E;
  if (p.E % kPer == 0) {
    for (int v = lane; v < pieces; v += LANES)
      reinterpret_cast<uint4*>(to)[v] = reinterpret_cast<const uint4*>(row)[v];
  } else {
    for (int e = lane; e < p.E; e += LANES) to[e] = row[e];
  }
}

template <bool F32>
void launch_route_grad(const RouteGradParams& p, cudaStream_t stream) {
  const int per = F32 ? 4 : 8, row_bytes = (p.E + per - 1) / per * 16;
  const bool every = !p.sigmoid && !p.renormalize;
  const int warps = p.T >= 1024 ? 4 : 1;
  if (p.k <= 8 && p.T >= 1024 && 16 * row_bytes <= 48 * 1024) {
    const unsigned grid = static_cast<unsigned>((p.T + 15) / 16);
    if (every)
      route_grad_kernel<F32, true, 8><<<grid, 128, 16 * row_bytes, stream>>>(p);
    else
      route_grad_kernel<F32, false, 8><<<grid, 128, 16 * row_bytes, stream>>>(p);
  } else {
    const unsigned grid = static_cast<unsigned>((p.T + warps - 1) / warps);
    if (every)
      route_grad_kernel<F32, true, 32><<<grid, warps * 32, warps * row_bytes, stream>>>(p);
    else
      route_grad_kernel<F32, false, 32><<<grid, warps * 32, warps * row_bytes, stream>>>(p);
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
constexpr int kPlanSlots = 2048;

struct PlanParams {
  const int32_t* ids;
  int64_t S;
  int E, blocks;
  int32_t* block_hist;   // [E][blocks]: counts, then their exclusive prefix over blocks
  int32_t* totals;       // [E]
  int64_t* m_sizes;
  int32_t* src;
  int32_t* pos;
};

// Ranks the block's slots; each thread's ranks go through `emit(slot, id, rank)` after the
// warps' histograms have been prefix-summed.  hist: [kPlanWarps][E] counters.
template <int BITS, typename Count, typename Emit>
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
#pragma unroll
    for (int b = 0; b < BITS; ++b) {
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
template <int BITS>
__global__ void __launch_bounds__(kPlanThreads) plan_one_kernel(const PlanParams p) {
  extern __shared__ int32_t smem_i[];
  int32_t* start = smem_i + kPlanWarps * p.E;
  __shared__ int32_t warp_sums[kPlanWarps];
  int32_t total = 0;
  // the expert starts are known only after the counts, before the ranks are emitted
  rank_slots<BITS>(
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

template <int BITS>
__global__ void __launch_bounds__(kPlanThreads) plan_rank_kernel(const PlanParams p) {
  extern __shared__ int32_t smem_i[];
  grid_launch_dependents();
  rank_slots<BITS>(
      p, static_cast<int64_t>(blockIdx.x) * kPlanSlots, smem_i,
      [&](int e, int32_t n) { p.block_hist[static_cast<int64_t>(e) * p.blocks + blockIdx.x] = n; },
      [&](int64_t s, int, int32_t rank) { p.pos[s] = rank; });
}

// One warp per expert: exclusive prefix of its counts over the blocks.
__global__ void __launch_bounds__(128) plan_scan_kernel(const PlanParams p) {
  const int lane = threadIdx.x & 31;
  const int e = blockIdx.x * 4 + (threadIdx.x >> 5);
  grid_launch_dependents();
  grid_dependency_wait();
  if (e >= p.E) return;
  int32_t* h = p.block_hist + static_cast<int64_t>(e) * p.blocks;
  // a lane scans 16 consecutive counts by itself, their loads in flight together, so that one
  // scan across the warp serves 512: what it takes is latency alone
  constexpr int kRun = 16;
  int32_t base = 0;
  for (int b0 = 0; b0 < p.blocks; b0 += 32 * kRun) {
    const int first = b0 + lane * kRun;
    int32_t c[kRun], sum = 0;
#pragma unroll
    for (int i = 0; i < kRun; ++i) c[i] = first + i < p.blocks ? h[first + i] : 0;
#pragma unroll
    for (int i = 0; i < kRun; ++i) sum += c[i];
    int32_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t y = __shfl_up_sync(kFull, inc, o);
      if (lane >= o) inc += y;
    }
    int32_t at = base + inc - sum;
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      if (first + i < p.blocks) h[first + i] = at;
      at += c[i];
    }
    base += __shfl_sync(kFull, inc, 31);
  }
  if (lane == 0) {
    p.totals[e] = base;
    p.m_sizes[e] = base;
  }
}

// A block's slots are put in expert order in shared memory first, so that what it writes to
// src is a run per expert and not a word here and there, and its loads are all in flight at
// once (1 M slots, 128 experts under ncu: 21 us with the words scattered and the loads in
// turn, 10 us so; the three kernels together 17.5 us, chains of latencies each, for 12.6 MB).
__global__ void __launch_bounds__(kPlanThreads) plan_place_kernel(const PlanParams p) {
  constexpr int kPer = kPlanSlots / kPlanThreads;
  __shared__ int32_t start[1024];     // first row of the expert in the block's run
  __shared__ int32_t local[1024];     // its place among the block's slots
  __shared__ int32_t order[kPlanSlots], row[kPlanSlots];
  __shared__ int32_t warp_sums[kPlanWarps];
  const int64_t s0 = static_cast<int64_t>(blockIdx.x) * kPlanSlots;
  int32_t id[kPer], rank[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int64_t s = s0 + i * kPlanThreads + threadIdx.x;
    const int32_t e = s < p.S ? p.ids[s] : -1;
    id[i] = e < 0 || e >= p.E ? -1 : e;
  }
  grid_dependency_wait();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int64_t s = s0 + i * kPlanThreads + threadIdx.x;
    rank[i] = s < p.S ? p.pos[s] : -1;
  }
  const int b = blockIdx.x;
  for (int e = threadIdx.x; e < p.E; e += kPlanThreads) start[e] = p.totals[e];
  __syncthreads();
  const int32_t total = block_prefix(start, p.E, warp_sums);
  for (int e = threadIdx.x; e < p.E; e += kPlanThreads) {
    const int32_t* h = p.block_hist + static_cast<int64_t>(e) * p.blocks;
    const int32_t before = h[b];
    start[e] += before;
    local[e] = (b + 1 < p.blocks ? h[b + 1] : p.totals[e]) - before;
  }
  __syncthreads();
  const int32_t used = block_prefix(local, p.E, warp_sums);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int64_t s = s0 + i * kPlanThreads + threadIdx.x;
    if (id[i] >= 0) {
      const int32_t at = start[id[i]] + rank[i], l = local[id[i]] + rank[i];
      p.pos[s] = at;
      order[l] = static_cast<int32_t>(s);
      row[l] = at;
    }
    if (s < p.S && s >= total) p.src[s] = -1;
  }
  __syncthreads();
  for (int l = threadIdx.x; l < used; l += kPlanThreads) p.src[row[l]] = order[l];
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
  uint64_t vecs_magic64;  // of short rows, sum only: a * magic >> 64 is a / vecs (a * vecs < 2^64)
  uint32_t vecs_magic;    // and a * magic >> 32 (a * vecs < 2^32)
};

// A thread owns PIECES 16-byte pieces of the output, 128 apart, and has the pieces of SLOTS rows
// in flight for each; the sum runs over the token's slots in order.  Bound by DRAM where a thread
// has enough in flight and few enough registers (eight blocks an SM): 8192 tokens of 8 rows of
// 4096 BF16 take 84 us, 604 MB at 7.2 TB/s (eight slots at once 88; FP32, half the arithmetic a
// byte, 170 with eight and 174 with four).  One or two slots a token leave room for two pieces:
// 16384 x 2 rows of 4096 BF16 62 us, 64 with one piece, 70 with four.
// FLAT: rows of fewer than 512 pieces that would leave threads idle, threads numbered over
// (token, piece): 65536 x 1 rows of 520 FP32 52 us, 109 with a block a row.
template <bool F32, bool FLAT, int PIECES, int SLOTS>
__global__ void __launch_bounds__(128, 8) combine_kernel(const CombineParams p) {
  constexpr int kSlots = SLOTS, kN = Vec<F32>::kN;
  int64_t t[PIECES];
  int v[PIECES];
  if constexpr (FLAT) {
    // (a block begins at piece first - t0 * vecs of token t0, in 64 bits; the rest is in 32)
    const int64_t first = static_cast<int64_t>(blockIdx.x) * (128 * PIECES);
    const int64_t t0 = __umul64hi(first, p.vecs_magic64);
    const uint32_t from = static_cast<uint32_t>(first - t0 * p.vecs) + threadIdx.x;
#pragma unroll
    for (int q = 0; q < PIECES; ++q) {
      const uint32_t e = from + q * 128, dt = __umulhi(e, p.vecs_magic);
      t[q] = t0 + dt;
      v[q] = static_cast<int>(e - dt * p.vecs);
    }
  } else {
#pragma unroll
    for (int q = 0; q < PIECES; ++q) {
      t[q] = blockIdx.x;
      v[q] = (blockIdx.y * PIECES + q) * 128 + threadIdx.x;
    }
  }
  const uint4* y = static_cast<const uint4*>(p.y);
  float acc[PIECES][kN];
#pragma unroll
  for (int q = 0; q < PIECES; ++q)
#pragma unroll
    for (int i = 0; i < kN; ++i) acc[q][i] = 0.f;
  for (int j0 = 0; j0 < p.k; j0 += kSlots) {
    Vec<F32> x[PIECES][kSlots];
    float w[PIECES][kSlots];
    int32_t r[PIECES][kSlots];
#pragma unroll
    for (int q = 0; q < PIECES; ++q)
#pragma unroll
      for (int u = 0; u < kSlots; ++u) {
        const int j = j0 + u;
        r[q][u] = j < p.k && t[q] < p.T && v[q] < p.vecs ? p.pos[t[q] * p.k + j] : -1;
        if (r[q][u] >= p.R) r[q][u] = -1;
      }
#pragma unroll
    for (int q = 0; q < PIECES; ++q)
#pragma unroll
      for (int u = 0; u < kSlots; ++u)
        if (r[q][u] >= 0) {
          w[q][u] = p.weights ? p.weights[t[q] * p.k + j0 + u] : 1.f;
          x[q][u].r = __ldcs(y + static_cast<int64_t>(r[q][u]) * p.vecs + v[q]);
        }
#pragma unroll
    for (int q = 0; q < PIECES; ++q)
#pragma unroll
      for (int u = 0; u < kSlots; ++u)
        if (r[q][u] >= 0)
#pragma unroll
          for (int i = 0; i < kN; ++i) acc[q][i] = fmaf(w[q][u], x[q][u].get(i), acc[q][i]);
  }
#pragma unroll
  for (int q = 0; q < PIECES; ++q)
    if (t[q] < p.T && v[q] < p.vecs)
      static_cast<uint4*>(p.out)[t[q] * p.vecs + v[q]] = pack_vec<F32>(acc[q]);
}

// THREADS (a block, or a warp for short rows) per token: dY of its rows is w * dout, dw the dot
// product of dout and the row.  65536 x 1 rows of 520 FP32: 90 us with 64 threads, 277 with 256.
// The token's dout pieces are read once per SLOTS slots; with one or two slots two of them are
// in flight (16384 x 2 rows of 4096 BF16 101 us, 138 with one).  1024 threads an SM: at the 120
// registers that ptxas takes by itself 512 fit, and 8192 x 8 rows of 4096 BF16 took 197 us, not
// 170 (1.14 GB: 6.7 TB/s, DRAM 81% busy).  Under that bound five of the eight-slot kernels spill,
// 24 bytes a thread in BF16 with 64 and more threads; with a warp a token 200 in BF16, 108 in FP32.
// k of 3 and 4 take the eight slots too: 16384 x 4 rows of 1024 BF16 62 us for 302 MB.
template <bool F32, int THREADS, int SLOTS>
__global__ void __launch_bounds__(THREADS == 32 ? 256 : THREADS, THREADS == 32 ? 4 : 1024 / THREADS)
    combine_grad_kernel(const CombineParams p) {
  constexpr int kN = Vec<F32>::kN, kSlots = SLOTS, kPieces = SLOTS == 2 ? 2 : 1;
  __shared__ float part[8][kSlots];
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x / THREADS) + threadIdx.x / THREADS;
  if (t >= p.T) return;   // whole warps, or no block at all
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x % THREADS;
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
    for (int v0 = tid; v0 < p.vecs; v0 += kPieces * THREADS) {
      Vec<F32> d[kPieces], x[kPieces][kSlots];
#pragma unroll
      for (int q = 0; q < kPieces; ++q) {
        const int v = v0 + q * THREADS;
        if (v >= p.vecs) break;
        d[q].r = dout[v];
        if (p.dweights)
#pragma unroll
          for (int u = 0; u < kSlots; ++u)
            if (r[u] >= 0) x[q][u].r = __ldcs(y + static_cast<int64_t>(r[u]) * p.vecs + v);
      }
#pragma unroll
      for (int q = 0; q < kPieces; ++q) {
        const int v = v0 + q * THREADS;
        if (v >= p.vecs) break;
#pragma unroll
        for (int u = 0; u < kSlots; ++u)
          if (r[u] >= 0) {
            float o[kN];
#pragma unroll
            for (int i = 0; i < kN; ++i) o[i] = w[u] * d[q].get(i);
            __stcs(dy + static_cast<int64_t>(r[u]) * p.vecs + v, pack_vec<F32>(o));
            if (p.dweights)
#pragma unroll
              for (int i = 0; i < kN; ++i) dot[u] = fmaf(d[q].get(i), x[q][u].get(i), dot[u]);
          }
      }
    }
    if (p.dweights) {
#pragma unroll
      for (int u = 0; u < kSlots; ++u) {
        const float s = warp_sum(dot[u]);
        if constexpr (THREADS == 32) {
          if (lane == u && j0 + u < p.k) p.dweights[t * p.k + j0 + u] = s;
        } else {
          if (lane == 0) part[warp][u] = s;
        }
      }
    }
    if (THREADS > 32 && p.dweights) {
      __syncthreads();
      if (threadIdx.x < kSlots && j0 + static_cast<int>(threadIdx.x) < p.k) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < THREADS / 32; ++i) s += part[i][threadIdx.x];
        p.dweights[t * p.k + j0 + threadIdx.x] = s;
      }
      __syncthreads();
    }
  }
  // rows that no slot uses have no gradient
  for (int j = 0; j < p.k; ++j) {
    const int64_t row = t * p.k + j;
    if (p.src[row] < 0)
      for (int v = tid; v < p.vecs; v += THREADS) dy[row * p.vecs + v] = make_uint4(0, 0, 0, 0);
  }
}

// A few tokens: one warp per block, so that they spread over the SMs.  128 BF16 experts, k = 8, in
// rounds: the two are within 0.1 us up to 512 tokens; 1024 take 3.3 us with four warps a block
// and 3.5 with one, 4096 4.2 and 5.0.
int route_warps(int64_t T) { return T >= 1024 ? 4 : 1; }

template <bool F32, int V>
bsmma_status launch_route_v(const RouteParams& p, cudaStream_t stream) {
  const int warps = route_warps(p.T);
  const unsigned grid = static_cast<unsigned>((p.T + warps - 1) / warps);
  if (!F32 && !p.bias && p.groups == 1 && p.k <= 8 && p.E % 32 == 0 && p.T >= 1024 &&
      (p.sigmoid || p.renormalize)) {
    route_quad_kernel<<<static_cast<unsigned>((p.T + 31) / 32), 128, 0, stream>>>(p);
  } else if (p.k <= 8 && p.T >= 8192 && p.groups <= 8 && (p.groups & (p.groups - 1)) == 0 &&
             p.E % (8 * p.groups) == 0 && (reinterpret_cast<uintptr_t>(p.bias) & 15) == 0 && (F32 || p.bias || p.groups > 1)) {
    route_eight_kernel<F32><<<static_cast<unsigned>((p.T + 15) / 16), 128, 0, stream>>>(p);
  } else if (!F32 && !p.bias && p.groups == 1) {
    if constexpr (V >= 2) {
      if (p.E % 2 == 0)
        route_bf16_kernel<V, true><<<grid, warps * 32, 0, stream>>>(p);
      else
        route_bf16_kernel<V, false><<<grid, warps * 32, 0, stream>>>(p);
    } else {
      route_bf16_kernel<V, false><<<grid, warps * 32, 0, stream>>>(p);
    }
  } else {
    route_kernel<F32, V><<<grid, warps * 32, p.groups > 1 ? warps * p.E * 4 : 0, stream>>>(p);
  }
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

template <int BITS>
bsmma_status launch_plan_bits(const PlanParams& p, cudaStream_t stream) {
  if (p.S <= kPlanSlots) {
    plan_one_kernel<BITS><<<1, kPlanThreads, (kPlanWarps + 1) * p.E * 4, stream>>>(p);
    count_launches(1);
    return cuda_ok(cudaGetLastError());
  }
  plan_rank_kernel<BITS><<<p.blocks, kPlanThreads, kPlanWarps * p.E * 4, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) e = launch_dependent(plan_scan_kernel, (p.E + 3) / 4, 128, 0, stream, p);
  if (e == cudaSuccess) e = launch_dependent(plan_place_kernel, p.blocks, kPlanThreads, 0, stream, p);
  count_launches(3);
  return cuda_ok(e);
}

template <bool F32, int PIECES, int SLOTS>
void launch_combine_p(CombineParams p, cudaStream_t stream) {
  constexpr int kBlock = 128 * PIECES;
  if (p.vecs > 1 && p.vecs < 512 && p.vecs % kBlock != 0) {
    p.vecs_magic64 = ~uint64_t(0) / p.vecs + 1;
    p.vecs_magic = ~uint32_t(0) / p.vecs + 1;
    combine_kernel<F32, true, PIECES, SLOTS>
        <<<static_cast<unsigned>((p.T * p.vecs + kBlock - 1) / kBlock), 128, 0, stream>>>(p);
  } else {
    const dim3 grid(static_cast<unsigned>(p.T), static_cast<unsigned>((p.vecs + kBlock - 1) / kBlock));
    combine_kernel<F32, false, PIECES, SLOTS><<<grid, 128, 0, stream>>>(p);
  }
}
template <bool F32>
void launch_combine_t(const CombineParams& p, cudaStream_t stream) {
  if (p.k <= 2)
    launch_combine_p<F32, 2, 2>(p, stream);
  else if (p.k <= 4)
    launch_combine_p<F32, 1, 4>(p, stream);
  else
    launch_combine_p<F32, 1, F32 ? 8 : 4>(p, stream);
}

template <bool F32, int SLOTS>
void launch_combine_grad_s(const CombineParams& p, cudaStream_t stream) {
  const unsigned T = static_cast<unsigned>(p.T);
  if (p.vecs <= 128)
    combine_grad_kernel<F32, 32, SLOTS><<<(T + 7) / 8, 256, 0, stream>>>(p);
  else if (p.vecs <= 256)
    combine_grad_kernel<F32, 64, SLOTS><<<T, 64, 0, stream>>>(p);
  else if (p.vecs <= 512)
    combine_grad_kernel<F32, 128, SLOTS><<<T, 128, 0, stream>>>(p);
  else
    combine_grad_kernel<F32, 256, SLOTS><<<T, 256, 0, stream>>>(p);
}
template <bool F32>
void launch_combine_grad_t(const CombineParams& p, cudaStream_t stream) {
  if (p.k <= 2)
    launch_combine_grad_s<F32, 2>(p, stream);
  else
    launch_combine_grad_s<F32, 8>(p, stream);
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
  const uint64_t per = E / p.groups;
  p.per_magic = static_cast<uint32_t>(per > 1 ? ((uint64_t(1) << 32) + per - 1) / per : 0);
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
  if (f32)
    launch_route_grad<true>(p, stream);
  else
    launch_route_grad<false>(p, stream);
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
  p.blocks = static_cast<int>((S + kPlanSlots - 1) / kPlanSlots);
  p.totals = static_cast<int32_t*>(workspace);
  p.block_hist = p.totals ? p.totals + E : nullptr;
  p.m_sizes = m_sizes;
  p.src = src;
  p.pos = pos;
  // one ballot a bit of the expert's number
  if (E <= 16) return launch_plan_bits<4>(p, stream);
  if (E <= 128) return launch_plan_bits<7>(p, stream);
  return launch_plan_bits<10>(p, stream);
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
  if (f32)
    launch_combine_t<true>(p, stream);
  else
    launch_combine_t<false>(p, stream);
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
    launch_combine_grad_t<true>(p, stream);
  else
    launch_combine_grad_t<false>(p, stream);
  count_launches(1);
  return cuda_ok(cudaGetLastError());
}

}  // namespace bsmma
