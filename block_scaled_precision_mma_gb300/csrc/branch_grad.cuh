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
#include <type_traits>

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

// What the mask drops of a piece, for rows with a NaN or an infinity.  (A call: with the ten rounds in the row
// loop once more, 39778 rows of 2520 with a bias and a gate a row take 356 us, and 344.)
static __device__ __noinline__ Vals drop_again(Vals f, Philox gen, uint64_t block, uint32_t limit) {
  drop(f, philox(gen, block), limit);
  return f;
}

// How a row is held: by a warp (rows of up to 256, 512 or 1024 values) or by a block.  A thread's
// pieces: with up to three sums a column the registers hold two; a warp's rows are short, and four of
// them keep it busy, or as many as there are (a step of 65536 rows of 256 values with dropout, a gate a row and
// two norms, both directions, 144 us, and 275 in warps that go through four).
// Blocks of up to 16 warps (rows of 8192) keep 128 registers a thread, longer rows 64.
// NORMED: there is a norm (entering: always); the two kinds of step share little but their loads.
enum RowKind { ROW_WARP_1, ROW_WARP_2, ROW_WARP, ROW_BLOCK, ROW_LONG };
template <RowKind ROW>
constexpr int kGradPieces = ROW == ROW_WARP_1 ? 1 : ROW == ROW_WARP ? 4 : 2;
template <RowKind ROW>
constexpr int kGradThreads = ROW <= ROW_WARP ? 128 : ROW == ROW_LONG ? 1024 : 512;

template <bool LEAVE, bool DF, bool VF, bool NORMED, bool BIAS, bool GATE, RowKind ROW>
__global__ void __launch_bounds__(kGradThreads<ROW>, 1) grad_kernel(const GradParams p) {
  constexpr int V = kGradPieces<ROW>;
  constexpr bool WARP = ROW <= ROW_WARP, LONG = ROW == ROW_LONG;
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
  const bool layer = a.norm.kind == BSMMA_NORM_LAYER;
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
  // dz is linear in d: its constant factor goes into the row's factors and into the sums
  const float scale = LEAVE ? a.y_scale * a.drop.scale : 1.f;
  // everything a row is read from and written to lies at these places, a row after the other
  const int64_t first = r0 * a.H + 8 * at.base;
  const char* v_at = static_cast<const char*>(a.v) + first * (VF ? 4 : 2);
  const char* d_at = static_cast<const char*>(a.d) + first * (DF ? 4 : 2);
  const int64_t v_step = a.H * (VF ? 4 : 2), d_step = a.H * (DF ? 4 : 2);
  int64_t out = 0;   // rows behind v_at's first, in bytes of v
  char* dv_at = static_cast<char*>(a.dv) + first * (VF ? 4 : 2);
  const char* res_at = !LEAVE && a.dres ? static_cast<const char*>(a.dres) + first * (VF ? 4 : 2) : nullptr;
  char* dx_at = LEAVE && a.dx ? static_cast<char*>(a.dx) + first * (DF ? 4 : 2) : nullptr;
  const float* w_at = a.norm.weight ? a.norm.weight + 8 * at.base : nullptr;
  const float* b_at = LEAVE && a.dgate && a.norm.bias ? a.norm.bias + 8 * at.base : nullptr;
  // a gate for each row (never with GATE): its gradient is a row
  float* dgate_at = LEAVE && !GATE && a.dgate ? a.dgate + first : nullptr;
  const __nv_bfloat16* gate_bf16 = nullptr;   // the gate's row, in its type
  const float* gate_f32 = nullptr;
  auto gate_piece = [&](int i) {
    if constexpr (VF) return widen<true>(load_raw<true>(gate_f32, 256 * i));
    else return widen<false>(load_raw<false>(gate_bf16, 256 * i));
  };
  auto weighted = [&](int i, Vals z) {
    if (w_at) {
      const Vals w = load_columns(w_at, 256 * i);
#pragma unroll
      for (int j = 0; j < 4; ++j) z.v[j] = mul2(z.v[j], w.v[j]);
    }
    return z;
  };

  // Where registers allow, gate * weight (a factor of 1 without either), by which d becomes q, is held for
  // a gate's rows, or for all.  With a gate's gradient sg is then the sum of d n, which over a
  // gate's rows gives dgate, times the weight, and its part of dweight, times the gate.  (Taken from the L1
  // cache for every row: 20000 rows of 5120 with dropout and a gate for 2048 of them 221 us, and 179.)
  constexpr bool HOLD = !LONG && !(BIAS && VF && !GATE);
  // With a bias there is the sum of d too, in sw's place; the parts of dweight and dbias are then added to
  // the worker's sums in memory after each gate's rows.
  constexpr bool OUT = HOLD && GATE && BIAS;
  bool fresh = true;   // nothing is there yet
  auto add_sums = [&](float* to, Vals f) {
    if (!to) return;
    to += static_cast<int64_t>(worker) * a.H;
    if (!fresh) {
      const Vals more = load_columns(to, 0);
#pragma unroll
      for (int j = 0; j < 4; ++j) f.v[j] = add2(f.v[j], more.v[j]);
    }
    store_sums(to, f);
  };
  Vals gw[HOLD ? V : 1];
  auto flush_gate = [&] {
    if constexpr (GATE) {
      const int64_t begin = g * a.gate_rows, end = g_end < a.T ? g_end : a.T;
      float* to = begin >= r0 && end <= r1
                      ? a.dgate + g * a.H
                      : p.part_g + (2 * static_cast<int64_t>(worker) + (begin > r0)) * a.H;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        // without a norm the factor is still to come (with one it came with n)
        if constexpr (!NORMED)
#pragma unroll
          for (int j = 0; j < 4; ++j) sg[i].v[j] = mul2(sg[i].v[j], both(a.y_scale * a.drop.scale));
        if (at.in(i)) {
          if constexpr (HOLD && NORMED) {
            const Vals one = gate_piece(i);
            if constexpr (OUT) {
              Vals dw, db;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                sw[i].v[j] = mul2(sw[i].v[j], both(scale));
                dw.v[j] = mul2(one.v[j], sg[i].v[j]);
                db.v[j] = mul2(one.v[j], sw[i].v[j]);
              }
              add_sums(p.part_w ? p.part_w + 8 * at.at(i) : nullptr, dw);
              add_sums(p.part_b ? p.part_b + 8 * at.at(i) : nullptr, db);
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j) sw[i].v[j] = __ffma2_rn(one.v[j], sg[i].v[j], sw[i].v[j]);
            }
            sg[i] = weighted(i, sg[i]);
            if (OUT && b_at) {
              const Vals b = load_columns(b_at, 256 * i);
#pragma unroll
              for (int j = 0; j < 4; ++j) sg[i].v[j] = __ffma2_rn(b.v[j], sw[i].v[j], sg[i].v[j]);
            }
          }
          store_sums(to + 8 * at.at(i), sg[i]);
        }
        sg[i] = none;
        if constexpr (OUT) sw[i] = none;
      }
      fresh = false;
    }
  };

  Raw<VF> next_v[V];
  Raw<DF> next_d[V];
#pragma unroll
  for (int i = 0; i < V; ++i) next_v[i] = zero_raw<VF>(), next_d[i] = zero_raw<DF>();
  // Without sums of a gate's rows the gate may be another for each: it is fetched with the row (15000 x
  // 7168, a gate a row, 275 us, and 356 when it is read at the row's turn) where registers allow.
  constexpr bool AHEAD = LEAVE && !GATE && HOLD && !VF;
  const bool each = LEAVE && !GATE && a.gate;
  Raw<VF> next_g[AHEAD ? V : 1];
  auto gate_at = [&](int64_t row) {
    if constexpr (VF) gate_f32 = static_cast<const float*>(a.gate) + row * a.H + 8 * at.base;
    else gate_bf16 = static_cast<const __nv_bfloat16*>(a.gate) + row * a.H + 8 * at.base;
  };
  auto gate_of = [&](int64_t r) {
    return static_cast<int64_t>(static_cast<uint32_t>(r) / static_cast<uint32_t>(a.gate_rows)) * a.H + 8 * at.base;
  };
  auto fetch = [&](int64_t r) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (at.in(i)) {
        next_v[i] = load_raw<VF>(v_at, 256 * i);
        next_d[i] = load_raw<DF>(d_at, 256 * i);
      }
    if constexpr (AHEAD) {
      if (each) {
        const int64_t from = gate_of(r);
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (at.in(i)) next_g[i] = load_raw<VF>(a.gate, from + 256 * i);
      }
    }
  };
  // the factors of a gate's rows, of a row with its own (fetched), or of all
  auto use_gate = [&] {
    if constexpr (HOLD) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        gw[i] = Vals{{both(1.f), both(1.f), both(1.f), both(1.f)}};
        if (!at.in(i)) continue;
        if constexpr (GATE) gw[i] = gate_piece(i);
        else if constexpr (LEAVE) {
          if constexpr (AHEAD) {
            if (each) gw[i] = widen<VF>(next_g[i]);
          } else {
            if (each) gw[i] = gate_piece(i);
          }
        }
        gw[i] = weighted(i, gw[i]);
      }
    }
  };
  if (r0 < r1) fetch(r0);
  if constexpr (GATE) gate_at(g);
  if (!each) use_gate();   // (a gate for each row: at its row's turn, when gate_at() has been there)
  for (int64_t r = r0; r < r1; ++r) {
    if constexpr (GATE) {
      if (r == g_end) {
        flush_gate();
        ++g;
        g_end += a.gate_rows;
        gate_at(g);
        use_gate();
      }
    } else if (each) {
      gate_at(static_cast<uint32_t>(r) / static_cast<uint32_t>(a.gate_rows));
      use_gate();
    }
    Vals c[V], of[V];   // the rows, later less their mean; d, without what was dropped
#pragma unroll
    for (int i = 0; i < V; ++i) {
      c[i] = widen<VF>(next_v[i]);
      of[i] = widen<DF>(next_d[i]);
    }
    v_at += v_step;
    d_at += d_step;
    if (r + 1 < r1) fetch(r + 1);
    if (LEAVE && dx_at) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        Vals d;
#pragma unroll
        for (int j = 0; j < 4; ++j) d.v[j] = mul2(of[i].v[j], both(a.x_scale));
        if (at.in(i)) store_raw<DF>(dx_at, 256 * i, narrow<DF>(d));
      }
      dx_at += d_step;
    }
    if (dropping) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const uint4 words = philox(gen, static_cast<uint64_t>(r) * at.vecs + at.at(i));
        drop(of[i], words, a.drop.threshold << 16);
        // a dropped value adds nothing to the gate's sum, whatever it is (with a norm: below)
        if constexpr (!NORMED) drop(c[i], words, a.drop.threshold << 16);
      }
    }
    // dz / scale, and times the weight (q / scale)
    auto gated = [&](int i) {
      Vals z = of[i];
      if (LEAVE && (GATE || a.gate)) {
        const Vals w = gate_piece(i);
#pragma unroll
        for (int j = 0; j < 4; ++j) z.v[j] = mul2(z.v[j], w.v[j]);
      }
      return z;
    };
    auto q_of = [&](int i) {
      if constexpr (HOLD) {
        Vals z = of[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) z.v[j] = mul2(z.v[j], gw[i].v[j]);
        return z;
      } else {
        return weighted(i, gated(i));
      }
    };
    if constexpr (!NORMED) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (!at.in(i)) continue;
        Vals z = gated(i);
        if (LEAVE && (GATE || dgate_at)) {
          if constexpr (GATE) {
#pragma unroll
            for (int j = 0; j < 4; ++j) sg[i].v[j] = __ffma2_rn(of[i].v[j], c[i].v[j], sg[i].v[j]);
          } else {
            Vals u;
#pragma unroll
            for (int j = 0; j < 4; ++j) u.v[j] = mul2(mul2(of[i].v[j], c[i].v[j]), both(scale));
            store_sums(dgate_at + 256 * i, u);
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) z.v[j] = mul2(z.v[j], both(scale));
        store_raw<VF>(dv_at + out, 256 * i, narrow<VF>(z));
      }
      out += v_step;
      if (LEAVE && !GATE && dgate_at) dgate_at += a.H;
      continue;
    }
    float (&shared)[2][kPart] = part[r & 1];
    float2 s, qmean = both(0.f);
    if (layer) {
      float2 sv = both(0.f), sq = both(0.f);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (at.in(i)) {
          const Vals z = q_of(i);
#pragma unroll
          for (int j = 0; j < 4; ++j) sv = add2(sv, c[i].v[j]), sq = add2(sq, z.v[j]);
        }
      s = row_sums2<WARP>(make_float2(sv.x + sv.y, sq.x + sq.y), shared[0]);
      const float2 minus_mean = both(-s.x * inv_h);
      qmean = both(s.y * inv_h);
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) c[i].v[j] = add2(c[i].v[j], minus_mean);
    }
    float2 sv = both(0.f), sq = both(0.f);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (at.in(i)) {
        const Vals z = q_of(i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sv = __ffma2_rn(c[i].v[j], c[i].v[j], sv);
          sq = __ffma2_rn(z.v[j], c[i].v[j], sq);
        }
      }
    Raw<VF> res[LEAVE ? 1 : V];   // on its way during the reduction
    if constexpr (!LEAVE) {
      if (res_at) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (at.in(i)) res[i] = load_raw<VF>(res_at + out, 256 * i);
      }
    }
    s = row_sums2<WARP>(make_float2(sv.x + sv.y, sq.x + sq.y), shared[1]);
    // dv = scale * (rs (q - mean q) - c rs^3 mean(q c)); n = c rs
    const float rs = inv_sqrt(fmaf(s.x, inv_h, a.norm.eps)), rss = rs * scale;
    float2 fq = both(rss);
    const float2 fc = both(-(rs * (s.y * inv_h)) * rs * rss), f0 = both(-rss * qmean.x);
    if (dropping && fc.x != fc.x) {
      // A row with a NaN or an infinity: dv is NaN, by fc, and so may every n be, but what was dropped adds
      // nothing to the sums all the same.  c becomes n, without it.
#pragma unroll
      for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) c[i].v[j] = mul2(c[i].v[j], fq);
        c[i] = drop_again(c[i], gen, static_cast<uint64_t>(r) * at.vecs + at.at(i), a.drop.threshold << 16);
      }
      fq = both(1.f);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (!at.in(i)) continue;
      Vals o = q_of(i), z;
      if constexpr (!(HOLD && GATE)) z = gated(i);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 n = mul2(c[i].v[j], fq);   // n scale
        o.v[j] = __ffma2_rn(c[i].v[j], fc, __ffma2_rn(o.v[j], fq, f0));
        if constexpr (HOLD && GATE) sg[i].v[j] = __ffma2_rn(of[i].v[j], n, sg[i].v[j]);
        else sw[i].v[j] = __ffma2_rn(z.v[j], n, sw[i].v[j]);
        if constexpr (OUT) sw[i].v[j] = add2(sw[i].v[j], of[i].v[j]);
        else if constexpr (BIAS) sb[i].v[j] = add2(sb[i].v[j], z.v[j]);
        if constexpr (!HOLD && GATE) c[i].v[j] = n;
      }
      if constexpr (!HOLD && GATE) {
        Vals n = weighted(i, c[i]);
        if (b_at) {
          const Vals b = load_columns(b_at, 256 * i);
#pragma unroll
          for (int j = 0; j < 4; ++j) n.v[j] = __ffma2_rn(b.v[j], both(scale), n.v[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) sg[i].v[j] = __ffma2_rn(of[i].v[j], n.v[j], sg[i].v[j]);
      }
      if (LEAVE && !GATE && dgate_at) {
        Vals n;
#pragma unroll
        for (int j = 0; j < 4; ++j) n.v[j] = mul2(c[i].v[j], fq);
        n = weighted(i, n);
        if (b_at) {
          const Vals b = load_columns(b_at, 256 * i);
#pragma unroll
          for (int j = 0; j < 4; ++j) n.v[j] = __ffma2_rn(b.v[j], both(scale), n.v[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) n.v[j] = mul2(of[i].v[j], n.v[j]);
        store_sums(dgate_at + 256 * i, n);
      }
      if constexpr (!LEAVE) {
        if (res_at) {
          const Vals more = widen<VF>(res[i]);
#pragma unroll
          for (int j = 0; j < 4; ++j) o.v[j] = add2(o.v[j], more.v[j]);
        }
      }
      store_raw<VF>(dv_at + out, 256 * i, narrow<VF>(o));
    }
    out += v_step;
    if (LEAVE && !GATE && dgate_at) dgate_at += a.H;
  }
  flush_gate();
  if constexpr (OUT) return;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (!at.in(i)) continue;
    const int64_t to = static_cast<int64_t>(worker) * a.H + 8 * at.at(i);
    if (p.part_w) store_sums(p.part_w + to, sw[i]);
    if constexpr (BIAS) {
#pragma unroll
      for (int j = 0; j < 4; ++j) sb[i].v[j] = mul2(sb[i].v[j], both(scale));
      if (p.part_b) store_sums(p.part_b + to, sb[i]);
    }
  }
}

template <bool LEAVE, bool DF, bool VF, bool NORMED, bool BIAS, bool GATE>
bsmma_status launch_grad_kernel(const GradParams& p, cudaStream_t stream) {
  const int64_t vecs = p.a.H / 8;
  const unsigned workers = static_cast<unsigned>(p.workers);
  auto launch = [&](auto kind) {
    constexpr RowKind ROW = decltype(kind)::value;
    constexpr int kWarpVecs = 32 * kGradPieces<ROW>;
    const unsigned threads = static_cast<unsigned>(32 * ((vecs + kWarpVecs - 1) / kWarpVecs));
    return ROW <= ROW_WARP ? launch_dependent(grad_kernel<LEAVE, DF, VF, NORMED, BIAS, GATE, ROW>, dim3((workers + 3) / 4),
                                              dim3(128), 0, stream, p)
                           : launch_dependent(grad_kernel<LEAVE, DF, VF, NORMED, BIAS, GATE, ROW>, dim3(workers),
                                              dim3(threads), 0, stream, p);
  };
  const cudaError_t e = vecs <= 32     ? launch(std::integral_constant<RowKind, ROW_WARP_1>{})
                        : vecs <= 64   ? launch(std::integral_constant<RowKind, ROW_WARP_2>{})
                        : vecs <= 128  ? launch(std::integral_constant<RowKind, ROW_WARP>{})
                        : vecs <= 1024 ? launch(std::integral_constant<RowKind, ROW_BLOCK>{})
                                       : launch(std::integral_constant<RowKind, ROW_LONG>{});
  return cuda_ok(e);
}

// One translation unit each.
bsmma_status grad_enter(const GradParams& p, cudaStream_t stream);
bsmma_status grad_leave_bf16(const GradParams& p, cudaStream_t stream);
bsmma_status grad_leave_f32(const GradParams& p, cudaStream_t stream);
bsmma_status grad_leave_mixed(const GradParams& p, cudaStream_t stream);

template <bool DF, bool VF>
bsmma_status launch_leave_grad(const GradParams& p, cudaStream_t stream) {
  // a gate for each row has no sums; where it has, a bias is part of them
  const bool gate = p.a.dgate != nullptr && p.a.gate_rows > 1, bias = p.part_b != nullptr || (gate && p.a.norm.bias);
  if (p.a.norm.kind == BSMMA_NORM_NONE)   // (no bias either)
    return gate ? launch_grad_kernel<true, DF, VF, false, false, true>(p, stream)
                : launch_grad_kernel<true, DF, VF, false, false, false>(p, stream);
  if (bias && gate) return launch_grad_kernel<true, DF, VF, true, true, true>(p, stream);
  if (bias) return launch_grad_kernel<true, DF, VF, true, true, false>(p, stream);
  if (gate) return launch_grad_kernel<true, DF, VF, true, false, true>(p, stream);
  return launch_grad_kernel<true, DF, VF, true, false, false>(p, stream);
}

}  // namespace branch
}  // namespace bsmma
