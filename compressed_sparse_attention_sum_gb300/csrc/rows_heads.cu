// Rows of up to 512 channels: norm, rotary positions, or both in one pass
// (csa_rope, csa_norm_rope and csa_norm of narrow rows).
//
// y = (x - m) r weight + bias with r = 1 / sqrt(mean((x - m)^2) + eps), then pairs
// (u, v) of y become scale (u cos a - v sin a, u sin a + v cos a).
//
// A row lies on 1 to 32 neighbouring lanes, 16 channels on each (see Unit), so
// that means are a few shuffles and both members of a pair are on one lane.  The
// lanes go through consecutive rows: a token's heads share their sines and cosines,
// all rows the weights, and the next kStages batches of rows are on their way.
#include <algorithm>

#include "csa_kernels.h"
#include "rows.cuh"
#include "smem_once.h"

namespace csa {
namespace {

constexpr int kThreads = 256;

// Rows that are used together (their sums are shuffled side by side), and batches
// under way: 256 bytes a thread, 128 KB an SM.
template <typename T>
struct Depth {
  static constexpr int kBatch = sizeof(T) == 2 ? 2 : 1, kStages = 4;
};

template <typename TI, typename TO, int ROPE, int V, int KIND>
__global__ void __launch_bounds__(kThreads, 2) rows_fwd_kernel(RowsFwd a, int lanes, int per) {
  constexpr int NU = 8 / V, kBatch = Depth<TI>::kBatch, kStages = Depth<TI>::kStages;
  constexpr bool NORM = KIND != kNormNone;
  using Vec = Pack<TI, V>;
  extern __shared__ __align__(16) unsigned char s_raw[];
  using Slot = VecSlot<Vec, kThreads>;                  // [stage][row][NU][2] of s_raw
  using PosSlot = VecSlot<Word, kThreads>;              // [stage][row] of s_pos
  unsigned char* s_pos = s_raw + sizeof(Vec) * kStages * kBatch * NU * 2 * kThreads;
  __shared__ int64_t s_turns[ROPE == kRopeNone ? 1 : kMaxHeadWidth / 2];
  const int lane = threadIdx.x & (lanes - 1);
  const int rows = a.b * a.s * a.H;
  const long long r0 = ((long long)blockIdx.x * kThreads + threadIdx.x) / lanes * per;
  const int n_rows = (int)max(0ll, min((long long)per, rows - r0));   // rows of these lanes
  RowCursor in = {0, 0, 0, 0};
  if (n_rows > 0) in.start(a.xs, (int)r0, a.s, a.H);
  RowCursor to = {in.h, in.t, in.bi, in.bi * a.os.b + in.t * a.os.t + in.h * a.os.h};
  int at[NU][2];
  uint32_t turns[NU];                                   // pairs of this lane that turn
#pragma unroll
  for (int k = 0; k < NU; ++k) {
    const Unit<ROPE, V> u(lane + k * lanes, a.d, a.rope.first, a.rope.dim);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      at[k][i] = !NORM && a.in_place && !u.turned(i, a.rope.first, a.rope.dim) ? -1 : u.c[i];
    turns[k] = 0;
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (u.index(e, a.rope.first, a.rope.dim) >= 0) turns[k] |= 1u << e;
  }
  int asked = 0;                                        // rows whose copies have begun
  const auto ask = [&](int stage) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (asked < n_rows) {
        const TI* x = (const TI*)a.x + in.off;
#pragma unroll
        for (int k = 0; k < NU; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (at[k][i] >= 0)
              Slot::ask(s_raw, ((stage * kBatch + u) * NU + k) * 2 + i, x + at[k][i]);
        if (ROPE != kRopeNone && a.pos != nullptr && (in.h == 0 || asked == 0))
          PosSlot::ask(s_pos, stage * kBatch + u, a.pos + in.bi * a.pos_stride + in.t);
        in.next(a.xs, a.s, a.H);
      }
      ++asked;
    }
    copies_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages; ++i) ask(i);
  float2 w[NU][2][V / 2], c[NU][2][V / 2];              // weight; bias (layer norm)
  float cs[NU][V], sn[NU][V];
#pragma unroll
  for (int k = 0; k < NU; ++k) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (NORM) {
        Pack<float, V> pw, pc;
#pragma unroll
        for (int e = 0; e < V; ++e) pw.w[e] = __float_as_uint(1.f), pc.w[e] = 0;
        if (at[k][i] >= 0 && a.weight != nullptr) pw.load(a.weight + at[k][i]);
        if (KIND == kNormLayer && at[k][i] >= 0 && a.bias != nullptr) pc.load(a.bias + at[k][i]);
#pragma unroll
        for (int e = 0; e < V / 2; ++e) w[k][i][e] = pw.two(e), c[k][i][e] = pc.two(e);
      }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) cs[k][e] = 1.f, sn[k][e] = 0.f;
  }
  if constexpr (ROPE != kRopeNone) {
    for (int i = threadIdx.x; i < a.rope.dim / 2; i += kThreads) s_turns[i] = a.rope.turns[i];
    __syncthreads();
  }
  const float inv_n = 1.f / a.d;
  int stage = 0;
  for (int k0 = 0; k0 < per; k0 += kBatch) {
    copies_wait<kStages - 1>();
    Vec raw[kBatch][NU][2];
    int pos[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      pos[u] = 0;
#pragma unroll
      for (int k = 0; k < NU; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          raw[u][k][i].clear();
          if (k0 + u < n_rows && at[k][i] >= 0)
            Slot::take(s_raw, ((stage * kBatch + u) * NU + k) * 2 + i, raw[u][k][i]);
        }
      if (ROPE != kRopeNone && a.pos != nullptr) {
        Word p;
        PosSlot::take(s_pos, stage * kBatch + u, p);
        pos[u] = (int)p.w[0];
      }
    }
    ask(stage);
    stage = stage + 1 == kStages ? 0 : stage + 1;
    float mean[kBatch], rstd[kBatch];
    if constexpr (NORM) {
      if constexpr (KIND == kNormLayer) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          float2 q = make_float2(0.f, 0.f);
#pragma unroll
          for (int k = 0; k < NU; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int e = 0; e < V / 2; ++e) q = add2(q, raw[u][k][i].two(e));
          mean[u] = q.x + q.y;
        }
        group_sums(mean, lanes);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) mean[u] *= inv_n;
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        float2 q = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < NU; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (KIND == kNormLayer && at[k][i] < 0) continue;
#pragma unroll
            for (int e = 0; e < V / 2; ++e) {
              float2 v = raw[u][k][i].two(e);
              if (KIND == kNormLayer) v = add2(v, make_float2(-mean[u], -mean[u]));
              q = fma2(v, v, q);
            }
          }
        rstd[u] = q.x + q.y;
      }
      group_sums(rstd, lanes);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) rstd[u] = rsqrtf(fmaf(rstd[u], inv_n, a.eps));
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (k0 + u >= n_rows) break;
      if constexpr (ROPE != kRopeNone) {
        if (to.h == 0 || k0 + u == 0) {                 // a token's first row here
          const int p = a.pos != nullptr ? pos[u] : to.t;
#pragma unroll
          for (int k = 0; k < NU; ++k) {
            const Unit<ROPE, V> un(lane + k * lanes, a.d, a.rope.first, a.rope.dim);
            unit_cos_sin<ROPE, V>(un, turns[k], s_turns, a.rope, p, cs[k], sn[k]);
          }
        }
      }
      TO* out = (TO*)a.out + to.off;
      to.next(a.os, a.s, a.H);
#pragma unroll
      for (int k = 0; k < NU; ++k) {
        float2 v[2][V / 2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < V / 2; ++e) {
            float2 y = raw[u][k][i].two(e);
            if constexpr (NORM) {
              if (KIND == kNormLayer) y = add2(y, make_float2(-mean[u], -mean[u]));
              y = mul2(y, make_float2(rstd[u], rstd[u]));
              y = KIND == kNormLayer ? fma2(y, w[k][i][e], c[k][i][e]) : mul2(y, w[k][i][e]);
            }
            v[i][e] = y;
          }
        if constexpr (KIND == kNormRms) {
          if (a.bias != nullptr) {                      // rare: not kept in registers
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (at[k][i] < 0) continue;
              Pack<float, V> pc;
              pc.load(a.bias + at[k][i]);
#pragma unroll
              for (int e = 0; e < V / 2; ++e) v[i][e] = add2(v[i][e], pc.two(e));
            }
          }
        }
        turn_unit<ROPE, V>(v, cs[k], sn[k], turns[k]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (at[k][i] < 0) continue;
          Pack<TO, V> o;
#pragma unroll
          for (int e = 0; e < V / 2; ++e) o.set(e, v[i][e]);
          o.store(out + at[k][i]);
        }
      }
    }
  }
}

template <typename TI, typename TO, int ROPE, int V, int KIND>
cudaError_t fwd(const RowsFwd& a, cudaStream_t st) {
  constexpr size_t smem = (size_t)Depth<TI>::kStages * Depth<TI>::kBatch * kThreads *
                          (16 * sizeof(TI) + (ROPE != kRopeNone ? sizeof(int) : 0));
  static SmemOnce once;
  const auto k = rows_fwd_kernel<TI, TO, ROPE, V, KIND>;
  const cudaError_t e = once(k, smem);
  if (e != cudaSuccess) return e;
  const int lanes = row_lanes<V>(a.d), groups = kThreads / lanes;
  const long long rows = (long long)a.b * a.s * a.H;
  // two CTAs an SM, of which each goes through a share of the rows
  const long long ctas = std::min((rows + groups - 1) / groups, 2ll * 152);
  const int per = (int)((rows + ctas * groups - 1) / (ctas * groups));
  k<<<(unsigned)ctas, kThreads, smem, st>>>(a, lanes, per);
  count_launches(1);
  return cudaGetLastError();
}

// Vectors of 16 bytes; the half layout's pairs on smaller ones where dim or first ask for it.
template <typename TI, typename TO, int KIND>
cudaError_t fwd_rope(const RowsFwd& a, cudaStream_t st) {
  constexpr int V = 16 / sizeof(TI);
  if (a.rope.turns == nullptr) {
    if constexpr (KIND != kNormNone) return fwd<TI, TO, kRopeNone, V, KIND>(a, st);
    return cudaErrorInvalidValue;
  }
  if (!a.rope.half) return fwd<TI, TO, kRopeInter, V, KIND>(a, st);
  if (half_by(V, a.rope)) return fwd<TI, TO, kRopeHalf, V, KIND>(a, st);
  return fwd<TI, TO, kRopeHalf, 2, KIND>(a, st);
}

}  // namespace

cudaError_t launch_rows_fwd(const RowsFwd& a, cudaStream_t st) {
  using bf = __nv_bfloat16;
  if (a.kind == kNormRms)
    return a.x_bf16 ? fwd_rope<bf, bf, kNormRms>(a, st) : fwd_rope<float, float, kNormRms>(a, st);
  if (a.kind == kNormLayer)
    return a.x_bf16 ? fwd_rope<bf, bf, kNormLayer>(a, st)
                    : fwd_rope<float, float, kNormLayer>(a, st);
  if (a.x_bf16)
    return a.out_bf16 ? fwd_rope<bf, bf, kNormNone>(a, st) : fwd_rope<bf, float, kNormNone>(a, st);
  return a.out_bf16 ? fwd_rope<float, bf, kNormNone>(a, st)
                    : fwd_rope<float, float, kNormNone>(a, st);
}

}  // namespace csa
