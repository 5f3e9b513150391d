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

__device__ __forceinline__ void store_sums(float* to, const float (&f)[8]) {
  *reinterpret_cast<float4*>(to) = make_float4(f[0], f[1], f[2], f[3]);
  *reinterpret_cast<float4*>(to + 4) = make_float4(f[4], f[5], f[6], f[7]);
}

template <bool LEAVE, bool DF, bool VF, bool BIAS, bool GATE, int TPR, int V>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR, 1) grad_kernel(const GradParams p) {
  constexpr int kRows = TPR < 128 ? 128 / TPR : 1;
  constexpr int kPart = TPR < 128 ? 1 : 2 * (TPR / 32);
  __shared__ float part[2][2][kPart];   // by the row's parity: one barrier a reduction
  grid_dependency_wait();
  grid_launch_dependents();
  const BranchGradArgs& a = p.a;
  const int tid = threadIdx.x % TPR;
  const int worker = static_cast<int>(blockIdx.x) * kRows + static_cast<int>(threadIdx.x) / TPR;
  if (worker >= p.workers) return;
  const int vecs = static_cast<int>(a.H / 8);
  const float inv_h = 1.f / static_cast<float>(a.H);
  const int64_t r0 = first_row(a.T, p.workers, worker), r1 = first_row(a.T, p.workers, worker + 1);
  const bool layer = a.norm.kind == BSMMA_NORM_LAYER, normed = a.norm.kind != BSMMA_NORM_NONE;
  Philox gen = {};
  if (LEAVE && a.drop.threshold) gen = philox_of(a.drop.rng);

  float sw[V][8], sb[BIAS ? V : 1][8], sg[GATE ? V : 1][8];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sw[i][j] = 0.f;
      if constexpr (BIAS) sb[i][j] = 0.f;
      if constexpr (GATE) sg[i][j] = 0.f;
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
        if (tid + i * TPR < vecs) store_sums(to + 8 * (tid + i * TPR), sg[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) sg[i][j] = 0.f;
      }
    }
  };

  Raw<VF> next_v[V];
  Raw<DF> next_d[V];
  auto fetch = [&](int64_t r) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * TPR;
      if (c < vecs && r < r1) {
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
    Raw<DF> rd[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      rv[i] = next_v[i];
      rd[i] = next_d[i];
      if constexpr (!LEAVE)
        rres[i] = a.dres && tid + i * TPR < vecs ? load_raw<VF>(a.dres, r * a.H + 8 * (tid + i * TPR))
                                                 : zero_raw<VF>();
    }
    fetch(r + 1);
    uint32_t keep[LEAVE ? V : 1];
    if constexpr (LEAVE) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        keep[i] = a.drop.threshold && tid + i * TPR < vecs
                      ? kept8(gen, static_cast<uint64_t>(r) * vecs + tid + i * TPR, a.drop.threshold)
                      : 0xFFu;
    }
    int64_t gate_row = 0;
    if constexpr (GATE) gate_row = g * a.H;
    else if (LEAVE && a.gate)
      gate_row = static_cast<int64_t>(static_cast<uint32_t>(r) / static_cast<uint32_t>(a.gate_rows)) * a.H;
    // dz of piece i (0 past the row); of: y_scale * d * keep, what the gate's sum has of it
    auto piece = [&](int i, float (&dz)[8], float (&of)[8]) {
      widen<DF>(rd[i], of);
      if constexpr (LEAVE) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          of[j] = keep[i] >> j & 1u ? of[j] * a.y_scale * a.drop.scale : 0.f;
        if (a.gate && tid + i * TPR < vecs) {
          float w[8];
          widen<VF>(load_raw<VF>(a.gate, gate_row + 8 * (tid + i * TPR)), w);
#pragma unroll
          for (int j = 0; j < 8; ++j) dz[j] = of[j] * w[j];
          return;
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) dz[j] = of[j];
    };
    auto weights = [&](int i, float (&w)[8]) {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = 1.f;
      if (a.norm.weight && tid + i * TPR < vecs) load_columns(a.norm.weight, 8 * (tid + i * TPR), w);
    };
    float mean = 0.f, qmean = 0.f, rs = 1.f, c1 = 0.f;
    if (normed) {
      float s[2] = {0.f, 0.f};
      float (&shared)[2][kPart] = part[r & 1];
      if (layer) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float v[8], dz[8], of[8], w[8];
          widen<VF>(rv[i], v);
          piece(i, dz, of);
          weights(i, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            s[0] += v[j];
            s[1] = fmaf(dz[j], w[j], s[1]);
          }
        }
        row_sums<TPR>(s, shared[0]);
        mean = s[0] * inv_h;
        qmean = s[1] * inv_h;
        s[0] = s[1] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (tid + i * TPR >= vecs) continue;
        float v[8], dz[8], of[8], w[8];
        widen<VF>(rv[i], v);
        piece(i, dz, of);
        weights(i, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float c = v[j] - mean;
          s[0] = fmaf(c, c, s[0]);
          s[1] = fmaf(dz[j] * w[j], c, s[1]);
        }
      }
      row_sums<TPR>(s, shared[1]);
      rs = __frsqrt_rn(fmaf(s[0], inv_h, a.norm.eps));
      c1 = rs * (s[1] * inv_h);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * TPR;
      if (c >= vecs) continue;
      float v[8], dz[8], of[8], w[8], o[8], b[8];
      widen<VF>(rv[i], v);
      piece(i, dz, of);
      weights(i, w);
      if constexpr (GATE) {
#pragma unroll
        for (int j = 0; j < 8; ++j) b[j] = 0.f;
        if (a.norm.bias) load_columns(a.norm.bias, 8 * c, b);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = (v[j] - mean) * rs;
        o[j] = normed ? rs * (fmaf(dz[j], w[j], -qmean) - n * c1) : dz[j];
        sw[i][j] = fmaf(dz[j], n, sw[i][j]);
        if constexpr (BIAS) sb[i][j] += dz[j];
        if constexpr (GATE) {
          const float z = normed ? fmaf(n, w[j], b[j]) : v[j];
          if (keep[i] >> j & 1u) sg[i][j] = fmaf(of[j], z, sg[i][j]);
        }
      }
      const int64_t at = r * a.H + 8 * c;
      if constexpr (!LEAVE) {
        float res[8];
        widen<VF>(rres[i], res);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] += res[j];
      }
      store_raw<VF>(a.dv, at, narrow<VF>(o));
      if constexpr (LEAVE) {
        if (a.dx) {
          float d[8];
          widen<DF>(rd[i], d);
#pragma unroll
          for (int j = 0; j < 8; ++j) d[j] *= a.x_scale;
          store_raw<DF>(a.dx, at, narrow<DF>(d));
        }
      }
    }
  }
  flush_gate();
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = tid + i * TPR;
    if (c >= vecs) continue;
    const int64_t at = static_cast<int64_t>(worker) * a.H + 8 * c;
    if (p.part_w) store_sums(p.part_w + at, sw[i]);
    if constexpr (BIAS) store_sums(p.part_b + at, sb[i]);
  }
}

// The threads of a worker by H, as forward but with at most two pieces a thread (four in a
// warp): with up to three sums a column the registers do not hold more.
template <bool LEAVE, bool DF, bool VF, bool BIAS, bool GATE>
bsmma_status launch_grad_kernel(const GradParams& p, cudaStream_t stream) {
  const int64_t vecs = p.a.H / 8;
  const unsigned blocks = static_cast<unsigned>(p.workers);
  cudaError_t e;
  if (vecs <= 32 * 4)
    e = launch_dependent(grad_kernel<LEAVE, DF, VF, BIAS, GATE, 32, 4>, dim3((blocks + 3) / 4), dim3(128), 0, stream, p);
  else if (vecs <= 256 * 2)
    e = launch_dependent(grad_kernel<LEAVE, DF, VF, BIAS, GATE, 256, 2>, dim3(blocks), dim3(256), 0, stream, p);
  else if (vecs <= 512 * 2)
    e = launch_dependent(grad_kernel<LEAVE, DF, VF, BIAS, GATE, 512, 2>, dim3(blocks), dim3(512), 0, stream, p);
  else
    e = launch_dependent(grad_kernel<LEAVE, DF, VF, BIAS, GATE, 1024, 2>, dim3(blocks), dim3(1024), 0, stream, p);
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
