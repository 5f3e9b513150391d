// branch_grad.cuh -- the gradients of branch_enter and branch_leave.
//
// With v the rows that were normed (z = n(v) * weight + bias, n = (v - m) r) and d the gradient
// of the step's result:
//   entering  dz = d                    dv = norm's gradient + dres
//   leaving   dz = y_scale * gate * keep * d,  dgate = sum_rows y_scale * d * keep * z,  dx = x_scale * d
//   norm      q = dz * weight;  dv = r (q - [layer] mean q - n mean(q n))
//   dweight = sum_rows dz n,  dbias = sum_rows dz
// r and m are taken from v again: it is read anyway, and the sums they need go through the
// same reduction as mean(q n) (one barrier a row for rms, two for a layer norm), so the forward
// pass keeps nothing but its inputs.
//
// A worker (a block, or a warp for rows of up to 1024 values) takes a run of consecutive rows
// and holds the columns' sums of its rows in registers, so that every row is read and written
// once; a second launch adds the workers' sums, in their order.  The gate's sums are taken at
// the end of each gate's rows: a gate whose rows are all one worker's is finished there, the
// others' pieces (each worker has at most a first and a last such gate) are added by the
// second launch.  Nothing depends on the order in which blocks run.
#pragma once
#include "branch.cuh"
#include "branch.h"

namespace bsmma {
namespace branch {

struct GradParams {
  BranchGradArgs a;
  int workers;
  float* part_w;   // [workers][H], or nullptr
  float* part_b;
  float* part_g;   // [workers][2][H]
};

// Rows r0(w) .. r0(w + 1) - 1 are worker w's.
__host__ __device__ inline int64_t first_row(int64_t T, int workers, int64_t w) { return T * w / workers; }

__device__ __forceinline__ void store_sums(float* to, const Vals& f) {
  *reinterpret_cast<float4*>(to) = make_float4(f.v[0].x, f.v[0].y, f.v[1].x, f.v[1].y);
  *reinterpret_cast<float4*>(to + 4) = make_float4(f.v[2].x, f.v[2].y, f.v[3].x, f.v[3].y);
}
__device__ __forceinline__ float sum_of(const float2 (&a)[2]) { return (a[0].x + a[0].y) + (a[1].x + a[1].y); }

// sum += of * z, where what was dropped (of is 0) adds nothing whatever z is.
__device__ __forceinline__ void add_gate(Vals& sum, const Vals& of, const Vals& z, bool dropping) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float2 u = z.v[j];
    if (dropping) u = make_float2(of.v[j].x == 0.f ? 0.f : u.x, of.v[j].y == 0.f ? 0.f : u.y);
    sum.v[j] = __ffma2_rn(of.v[j], u, sum.v[j]);
  }
}

// A thread's pieces of a row: with up to three sums a column the registers hold two (a warp's
// rows are short, and four of them keep it busy).
template <bool WARP>
constexpr int kGradPieces = WARP ? 4 : 2;
// Blocks of up to 14 warps (rows of 7168) keep 128 registers a thread, longer rows 64.
template <bool WARP, bool LONG>
constexpr int kGradThreads = WARP ? 128 : LONG ? 1024 : 512;

template <bool LEAVE, bool DF, bool VF, bool BIAS, bool GATE, bool WARP, bool LONG>
__global__ void __launch_bounds__(kGradThreads<WARP, LONG>, 1) grad_kernel(const GradParams p) {
  constexpr int V = kGradPieces<WARP>;
  constexpr int kPart = WARP ? 1 : 64;
  __shared__ float part[2][2][kPart];   // by the row's parity: one barrier a reduction
  grid_dependency_wait();
  grid_launch_dependents();
  const BranchGradArgs& a = p.a;
  const Place<WARP, V> at(a.H);
  const int worker = WARP ? static_cast<int>(blockIdx.x) * 4 + static_cast<int>(threadIdx.x >> 5)
                          : static_cast<int>(blockIdx.x);
  if (worker >= p.workers) return;
  const float inv_h = a.inv_h;
  const int64_t r0 = first_row(a.T, p.workers, worker), r1 = first_row(a.T, p.workers, worker + 1);
  const bool layer = a.norm.kind == BSMMA_NORM_LAYER, normed = a.norm.kind != BSMMA_NORM_NONE;
  const bool dropping = LEAVE && a.drop.threshold != 0;
  Philox gen = {};
  if (dropping) gen = philox_of(a.drop.rng);

  Vals sw[V], sb[BIAS ? V : 1], sg[GATE ? V : 1];
  const Vals none = {};
#pragma unroll
  for (int i = 0; i < V; ++i) {
    sw[i] = none;
    if constexpr (BIAS) sb[i] = none;
    if constexpr (GATE) sg[i] = none;
  }
  int64_t g = 0, g_end = 0;   // the gate in use and the row after its last
  if constexpr (GATE) {
    g = r0 / a.gate_rows;
    g_end = (g + 1) * a.gate_rows;
  }
  auto flush_gate = [&] {
    if constexpr (GATE) {
      const int64_t begin = g * a.gate_rows, end = g_end < a.T ? g_end : a.T;
      float* to = begin >= r0 && end <= r1
                      ? a.dgate + g * a.H
                      : p.part_g + (2 * static_cast<int64_t>(worker) + (begin > r0)) * a.H;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (at.in(i)) store_sums(to + 8 * (at.at(i)), sg[i]);
        sg[i] = none;
      }
    }
  };

  Raw<VF> next_v[V];
  Raw<DF> next_d[V];
  auto fetch = [&](int64_t r) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = at.at(i);
      if (at.in(i) && r < r1) {
        next_v[i] = load_raw<VF>(a.v, r * a.H + 8 * c);
        next_d[i] = load_raw<DF>(a.d, r * a.H + 8 * c);
      } else {
        next_v[i] = zero_raw<VF>();
        next_d[i] = zero_raw<DF>();
      }
    }
  };
  fetch(r0);
  for (int64_t r = r0; r < r1; ++r) {
    if constexpr (GATE) {
      if (r == g_end) {
        flush_gate();
        ++g;
        g_end += a.gate_rows;
      }
    }
    Raw<VF> rv[V], rres[LEAVE ? 1 : V];
    Vals of[V];   // leaving: y_scale * d * keep, what the gate's sum has of dz; entering: d
#pragma unroll
    for (int i = 0; i < V; ++i) {
      rv[i] = next_v[i];
      of[i] = widen<DF>(next_d[i]);
      const int c = at.at(i);
      if constexpr (LEAVE) {
        if (a.dx && at.in(i)) {
          Vals d = of[i];
#pragma unroll
          for (int j = 0; j < 4; ++j) d.v[j] = mul2(d.v[j], both(a.x_scale));
          store_raw<DF>(a.dx, r * a.H + 8 * c, narrow<DF>(d));
        }
        const float2 scale = both(a.y_scale * a.drop.scale);
#pragma unroll
        for (int j = 0; j < 4; ++j) of[i].v[j] = mul2(of[i].v[j], scale);
      } else {
        rres[i] = a.dres && at.in(i) ? load_raw<VF>(a.dres, r * a.H + 8 * c) : zero_raw<VF>();
      }
    }
    fetch(r + 1);
    if (dropping) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (at.in(i))
          drop(of[i], philox(gen, static_cast<uint64_t>(r) * at.vecs + at.at(i)), a.drop.threshold << 16);
    }
    int64_t gate_row = 0;
    if constexpr (GATE) gate_row = g * a.H;
    else if (LEAVE && a.gate)
      gate_row = static_cast<int64_t>(static_cast<uint32_t>(r) / static_cast<uint32_t>(a.gate_rows)) * a.H;
    auto dz_of = [&](int i) {
      Vals dz = of[i];
      if (LEAVE && (GATE || a.gate)) {
        const Vals w = widen<VF>(load_raw<VF>(a.gate, gate_row + 8 * (at.at(i))));
#pragma unroll
        for (int j = 0; j < 4; ++j) dz.v[j] = mul2(dz.v[j], w.v[j]);
      }
      return dz;
    };
    auto weighted = [&](int i, Vals q) {
      if (a.norm.weight) {
        const Vals w = load_columns(a.norm.weight, 8 * (at.at(i)));
#pragma unroll
        for (int j = 0; j < 4; ++j) q.v[j] = mul2(q.v[j], w.v[j]);
      }
      return q;
    };
    float mean = 0.f, qmean = 0.f, rs = 1.f, c1 = 0.f;
    if (normed) {
      float s[2];
      float (&shared)[2][kPart] = part[r & 1];
      if (layer) {
        float2 sv[2] = {both(0.f), both(0.f)}, sq[2] = {both(0.f), both(0.f)};
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (!at.in(i)) continue;
          const Vals v = widen<VF>(rv[i]), q = weighted(i, dz_of(i));
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            sv[j & 1] = add2(sv[j & 1], v.v[j]);
            sq[j & 1] = add2(sq[j & 1], q.v[j]);
          }
        }
        s[0] = sum_of(sv), s[1] = sum_of(sq);
        row_sums<WARP>(s, shared[0]);
        mean = s[0] * inv_h;
        qmean = s[1] * inv_h;
      }
      float2 sv[2] = {both(0.f), both(0.f)}, sq[2] = {both(0.f), both(0.f)};
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (!at.in(i)) continue;
        const Vals v = widen<VF>(rv[i]), q = weighted(i, dz_of(i));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 c = add2(v.v[j], both(-mean));
          sv[j & 1] = __ffma2_rn(c, c, sv[j & 1]);
          sq[j & 1] = __ffma2_rn(q.v[j], c, sq[j & 1]);
        }
      }
      s[0] = sum_of(sv), s[1] = sum_of(sq);
      row_sums<WARP>(s, shared[1]);
      rs = inv_sqrt(fmaf(s[0], inv_h, a.norm.eps));
      c1 = rs * (s[1] * inv_h);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = at.at(i);
      if (!at.in(i)) continue;
      const Vals v = widen<VF>(rv[i]), dz = dz_of(i);
      Vals o = dz;
      if (normed) {
        o = weighted(i, dz);
        Vals n;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          n.v[j] = mul2(add2(v.v[j], both(-mean)), both(rs));
          sw[i].v[j] = __ffma2_rn(dz.v[j], n.v[j], sw[i].v[j]);
          o.v[j] = mul2(__ffma2_rn(n.v[j], both(-c1), add2(o.v[j], both(-qmean))), both(rs));
        }
        if constexpr (BIAS) {
#pragma unroll
          for (int j = 0; j < 4; ++j) sb[i].v[j] = add2(sb[i].v[j], dz.v[j]);
        }
        if constexpr (GATE) {
          n = weighted(i, n);
          if (a.norm.bias) {
            const Vals b = load_columns(a.norm.bias, 8 * c);
#pragma unroll
            for (int j = 0; j < 4; ++j) n.v[j] = add2(n.v[j], b.v[j]);
          }
          add_gate(sg[i], of[i], n, dropping);
        }
      } else {
        if constexpr (GATE) add_gate(sg[i], of[i], v, dropping);
      }
      if constexpr (!LEAVE) {
        const Vals res = widen<VF>(rres[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) o.v[j] = add2(o.v[j], res.v[j]);
      }
      store_raw<VF>(a.dv, r * a.H + 8 * c, narrow<VF>(o));
    }
  }
  flush_gate();
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = at.at(i);
    if (!at.in(i)) continue;
    const int64_t to = static_cast<int64_t>(worker) * a.H + 8 * c;
    if (p.part_w) store_sums(p.part_w + to, sw[i]);
    if constexpr (BIAS) store_sums(p.part_b + to, sb[i]);
  }
}

template <bool LEAVE, bool DF, bool VF, bool BIAS, bool GATE>
bsmma_status launch_grad_kernel(const GradParams& p, cudaStream_t stream) {
  const int64_t vecs = p.a.H / 8;
  const unsigned blocks = static_cast<unsigned>(p.workers);
  cudaError_t e;
  if (vecs <= 32 * kGradPieces<true>) {
    e = launch_dependent(grad_kernel<LEAVE, DF, VF, BIAS, GATE, true, false>, dim3((blocks + 3) / 4), dim3(128), 0,
                         stream, p);
  } else {
    constexpr int kWarpVecs = 32 * kGradPieces<false>;
    const unsigned threads = static_cast<unsigned>(32 * ((vecs + kWarpVecs - 1) / kWarpVecs));
    e = launch_dependent(threads <= 512 ? grad_kernel<LEAVE, DF, VF, BIAS, GATE, false, false>
                                        : grad_kernel<LEAVE, DF, VF, BIAS, GATE, false, true>,
                         dim3(blocks), dim3(threads), 0, stream, p);
  }
  return cuda_ok(e);
}

// One translation unit each.
bsmma_status grad_enter(const GradParams& p, cudaStream_t stream);
bsmma_status grad_leave_bf16(const GradParams& p, cudaStream_t stream);
bsmma_status grad_leave_f32(const GradParams& p, cudaStream_t stream);
bsmma_status grad_leave_mixed(const GradParams& p, cudaStream_t stream);

template <bool DF, bool VF>
bsmma_status launch_leave_grad(const GradParams& p, cudaStream_t stream) {
  const bool bias = p.part_b != nullptr, gate = p.a.dgate != nullptr;
  if (bias && gate) return launch_grad_kernel<true, DF, VF, true, true>(p, stream);
  if (bias) return launch_grad_kernel<true, DF, VF, true, false>(p, stream);
  if (gate) return launch_grad_kernel<true, DF, VF, false, true>(p, stream);
  return launch_grad_kernel<true, DF, VF, false, false>(p, stream);
}

}  // namespace branch
}  // namespace bsmma
