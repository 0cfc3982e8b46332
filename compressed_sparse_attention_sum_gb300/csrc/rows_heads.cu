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

// Rows that are used together, their sums shuffled side by side: two bf16 rows of a norm
// alone (1M x 512: 337 us, one at a time 354); a rotation has as much to do meanwhile.
template <typename T, int ROPE, int KIND>
constexpr int batch_rows() {
  return sizeof(T) == 2 && KIND != kNormNone && ROPE == kRopeNone ? 2 : 1;
}
constexpr int kStages = 4;                              // batches under way

// PER_SM: CTAs an SM; with three the weight stays in shared memory.
template <typename TI, typename TO, int ROPE, int V, int KIND, int PER_SM>
__global__ void __launch_bounds__(kThreads, PER_SM)
rows_fwd_kernel(RowsFwd a, int lanes, Walk walk) {
  constexpr int NU = 8 / V, kBatch = batch_rows<TI, ROPE, KIND>();
  constexpr bool kKeep = PER_SM < 3;
  constexpr bool NORM = KIND != kNormNone;
  using Vec = Pack<TI, V>;
  extern __shared__ __align__(16) unsigned char s_raw[];
  using Slot = VecSlot<Vec, kThreads>;                  // [stage][row][NU][2] of s_raw
  using PosSlot = VecSlot<Word, kThreads>;              // [stage][row] of s_pos
  unsigned char* s_pos = s_raw + sizeof(Vec) * kStages * kBatch * NU * 2 * kThreads;
  __shared__ int64_t s_turns[ROPE == kRopeNone ? 1 : kMaxHeadWidth / 2];
  __shared__ __align__(16) float s_w[NORM && !kKeep ? kMaxHeadWidth : 1];
  const int lane = threadIdx.x & (lanes - 1);
  const int step = (int)gridDim.x * (kThreads / lanes);
  const long long x_step = (walk.tokens ? a.xs.t : a.xs.h) * (int)sizeof(TI);
  const long long o_step = (walk.tokens ? a.os.t : a.os.h) * (int)sizeof(TO);
  Walk::At in, to;
  in.run = to.run = (int)((blockIdx.x * kThreads + threadIdx.x) / lanes);
  walk.open(in, a.s, a.H, a.xs, a.x, sizeof(TI));
  walk.open(to, a.s, a.H, a.os, a.out, sizeof(TO));
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
  const auto ask = [&](int stage) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (in.slot + u < in.len) {
        const TI* x = reinterpret_cast<const TI*>(in.p + u * x_step);
#pragma unroll
        for (int k = 0; k < NU; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (at[k][i] >= 0)
              Slot::ask(s_raw, ((stage * kBatch + u) * NU + k) * 2 + i, x + at[k][i]);
        if (ROPE != kRopeNone && a.pos != nullptr && (walk.tokens || in.slot + u == 0))
          PosSlot::ask(s_pos, stage * kBatch + u, a.pos + in.bi * a.pos_stride + in.t + in.slot + u);
      }
    }
    copies_commit();
    in.p += kBatch * x_step;
    in.slot += kBatch;
    if (in.slot >= walk.run) {
      in.run += step;
      walk.open(in, a.s, a.H, a.xs, a.x, sizeof(TI));
    }
  };
#pragma unroll 1
  for (int i = 0; i < kStages; ++i) ask(i);
  float2 w[NU][2][V / 2], c[NU][2][V / 2];              // weight; bias (layer norm)
  float cs[NU][V], sn[NU][V];
#pragma unroll
  for (int k = 0; k < NU; ++k) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (NORM && kKeep) {
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
  static_assert(kKeep || (KIND == kNormRms && ROPE != kRopeNone), "");
  if constexpr (!kKeep)
    for (int i = threadIdx.x; i < a.d; i += kThreads) s_w[i] = a.weight != nullptr ? a.weight[i] : 1.f;
  if constexpr (ROPE != kRopeNone) {
    for (int i = threadIdx.x; i < a.rope.dim / 2; i += kThreads) s_turns[i] = a.rope.turns[i];
    __syncthreads();
  }
  const float inv_n = 1.f / a.d;
  const auto use = [&](int stage) {
    copies_wait<kStages - 1>();
    float2 v[kBatch][NU][2][V / 2];
    int pos[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      pos[u] = 0;
      // where nothing was asked for, whatever the place holds: it is neither counted nor stored
#pragma unroll
      for (int k = 0; k < NU; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          Vec raw;
          Slot::take(s_raw, ((stage * kBatch + u) * NU + k) * 2 + i, raw);
#pragma unroll
          for (int e = 0; e < V / 2; ++e) v[u][k][i][e] = raw.two(e);
        }
      if (ROPE != kRopeNone && a.pos != nullptr) {
        Word p;
        PosSlot::take(s_pos, stage * kBatch + u, p);
        pos[u] = (int)p.w[0];
      }
    }
    ask(stage);
    if constexpr (NORM) {
      float sum[kBatch];
      if constexpr (KIND == kNormLayer) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          sum[u] = 0.f;
#pragma unroll
          for (int k = 0; k < NU; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float2 q = v[u][k][i][0];
#pragma unroll
              for (int e = 1; e < V / 2; ++e) q = add2(q, v[u][k][i][e]);
              sum[u] += at[k][i] >= 0 ? q.x + q.y : 0.f;
            }
        }
        group_sums(sum, lanes);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const float m = -sum[u] * inv_n;
#pragma unroll
          for (int k = 0; k < NU; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int e = 0; e < V / 2; ++e) v[u][k][i][e] = add2(v[u][k][i][e], make_float2(m, m));
        }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        sum[u] = 0.f;
#pragma unroll
        for (int k = 0; k < NU; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float2 q = mul2(v[u][k][i][0], v[u][k][i][0]);
#pragma unroll
            for (int e = 1; e < V / 2; ++e) q = fma2(v[u][k][i][e], v[u][k][i][e], q);
            sum[u] += at[k][i] >= 0 ? q.x + q.y : 0.f;
          }
      }
      group_sums(sum, lanes);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const float r = rsqrtf(fmaf(sum[u], inv_n, a.eps));
#pragma unroll
        for (int k = 0; k < NU; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            Pack<float, V> pw;
            if constexpr (!kKeep) pw.load(s_w + max(at[k][i], 0));
#pragma unroll
            for (int e = 0; e < V / 2; ++e) {
              const float2 y = mul2(v[u][k][i][e], make_float2(r, r));
              const float2 we = kKeep ? w[k][i][e] : pw.two(e);
              v[u][k][i][e] = KIND == kNormLayer ? fma2(y, we, c[k][i][e]) : mul2(y, we);
            }
          }
      }
      if (KIND == kNormRms && a.bias != nullptr) {      // rare: not kept in registers
#pragma unroll
        for (int k = 0; k < NU; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (at[k][i] < 0) continue;
            Pack<float, V> pc;
            pc.load(a.bias + at[k][i]);
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
#pragma unroll
              for (int e = 0; e < V / 2; ++e) v[u][k][i][e] = add2(v[u][k][i][e], pc.two(e));
          }
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if constexpr (ROPE != kRopeNone) {
        if (walk.tokens || to.slot + u == 0) {          // another token
          const int p = a.pos != nullptr ? pos[u] : to.t + to.slot + u;
#pragma unroll
          for (int k = 0; k < NU; ++k) {
            const Unit<ROPE, V> un(lane + k * lanes, a.d, a.rope.first, a.rope.dim);
            unit_cos_sin<ROPE, V>(un, turns[k], s_turns, a.rope, p, cs[k], sn[k]);
          }
        }
      }
      TO* out = reinterpret_cast<TO*>(to.p + u * o_step);
      const bool live = to.slot + u < to.len;
#pragma unroll
      for (int k = 0; k < NU; ++k) {
        turn_unit<ROPE, V>(v[u][k], cs[k], sn[k], turns[k]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (at[k][i] < 0 || !live) continue;
          Pack<TO, V> o;
#pragma unroll
          for (int e = 0; e < V / 2; ++e) o.set(e, v[u][k][i][e]);
          o.store(out + at[k][i]);
        }
      }
    }
    to.p += kBatch * o_step;
    to.slot += kBatch;
    if (to.slot >= walk.run) {
      to.run += step;
      walk.open(to, a.s, a.H, a.os, a.out, sizeof(TO));
    }
  };
  int stage = 0;
#pragma unroll 1
  for (int left = walk.rounds * walk.run; left > 0; left -= kBatch) {
    use(stage);
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }
}

template <typename TI, typename TO, int ROPE, int V, int KIND, int PER_SM = 2>
cudaError_t fwd(const RowsFwd& a, cudaStream_t st) {
  constexpr int kBatch = batch_rows<TI, ROPE, KIND>();
  constexpr size_t smem = (size_t)kStages * kBatch * kThreads *
                          (16 * sizeof(TI) + (ROPE != kRopeNone ? sizeof(int) : 0));
  static SmemOnce once;
  const auto k = rows_fwd_kernel<TI, TO, ROPE, V, KIND, PER_SM>;
  const cudaError_t e = once(k, smem);
  if (e != cudaSuccess) return e;
  const int lanes = row_lanes<V>(a.d);
  int ctas = PER_SM * 152;
  const Walk w = make_walk(a.b, a.s, a.H, ROPE != kRopeNone, kThreads / lanes, kBatch, &ctas);
  k<<<(unsigned)ctas, kThreads, smem, st>>>(a, lanes, w);
  count_launches(1);
  return cudaGetLastError();
}

// Whether three CTAs an SM go through bf16 rows that are normed and turned, RMS, interleaved.  They
// hide more latency but read the weight from shared memory and share an SM's issue, and are faster
// only for long calls whose runs are 16 heads of a token, on all lanes, half of them turned at most
// (us, two CTAs / three; 64 of 512 channels turned): 64 heads, 2^26 channels 44.2 / 52.4, 1.5 x 2^26
// 80.8 / 77.6, 2^28 198 / 175, 2^29 377 / 343; 64 of 128 at 2^28 196 / 182.  Others, at 2^28 channels: 8
// heads 180 / 190, 5 heads 176 / 209, 16 x 192 183 / 227, all 512 turned 183 / 191, half layout 198 / 195
// (at 2^29 378 / 383); 16 x 2 tokens of 32 x 128 2.9 / 3.2.
bool three_ctas(const RowsFwd& a, int lanes) {
  return !a.rope.half && a.H % 16 == 0 && a.d == 16 * lanes && 2 * a.rope.dim <= a.d &&
         (long long)a.b * a.s * a.H * a.d > 1ll << 26;
}

// Vectors of 16 bytes; the half layout's pairs on smaller ones where dim or first ask for it.
template <typename TI, typename TO, int KIND>
cudaError_t fwd_rope(const RowsFwd& a, cudaStream_t st) {
  constexpr int V = 16 / sizeof(TI);
  if (a.rope.turns == nullptr) {
    if constexpr (KIND != kNormNone) return fwd<TI, TO, kRopeNone, V, KIND>(a, st);
    return cudaErrorInvalidValue;
  }
  if (a.rope.half && !half_by(V, a.rope))
    return V == 8 && half_by(4, a.rope) ? fwd<TI, TO, kRopeHalf, 4, KIND>(a, st)
                                        : fwd<TI, TO, kRopeHalf, 2, KIND>(a, st);
  if constexpr (KIND == kNormRms && sizeof(TI) == 2) {
    if (three_ctas(a, row_lanes<V>(a.d))) return fwd<TI, TO, kRopeInter, V, KIND, 3>(a, st);
  }
  return a.rope.half ? fwd<TI, TO, kRopeHalf, V, KIND>(a, st)
                     : fwd<TI, TO, kRopeInter, V, KIND>(a, st);
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
