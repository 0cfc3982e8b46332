// The gradient of the norms of rows of up to 512 channels, and of a norm followed by
// rotary positions (csa_norm_rope_bwd, csa_norm_bwd of narrow rows).
//
// With dy the gradient turned back by the row's angle, xc = x - mean, r = 1 / sqrt(mean(xc^2)
// + eps) and g = dy weight: dx = r g - r mean(g) - xc r^3 mean(g xc), dweight = sum dy xc r,
// dbias = sum dy (RMS: mean = 0 and no mean(g)).  Rows lie on lanes and come as in
// rows_heads.cu; a lane keeps its channels' sums of dweight and dbias in registers to the end.
#include "csa_kernels.h"
#include "rows.cuh"
#include "smem_once.h"

namespace csa {
namespace {

constexpr int kThreads = 256, kStages = 3;

// DB: whether dbias may be wanted and the norm may be a layer norm; RMS norms without a bias
// have a kernel of their own, with fewer sums.
template <typename TX, typename TG, int ROPE, int V, bool DB>
__global__ void __launch_bounds__(kThreads, 2) rows_bwd_kernel(RowsBwd a, int lanes, Walk walk) {
  constexpr int NU = 8 / V;
  using VecX = Pack<TX, V>;
  using VecG = Pack<TG, V>;
  using SlotX = VecSlot<VecX, kThreads>;                // [stage][NU][2]
  using SlotG = VecSlot<VecG, kThreads>;
  using PosSlot = VecSlot<Word, kThreads>;              // [stage]
  extern __shared__ __align__(16) unsigned char s_raw[];
  unsigned char* s_g = s_raw + sizeof(VecX) * kStages * NU * 2 * kThreads;
  unsigned char* s_pos = s_g + sizeof(VecG) * kStages * NU * 2 * kThreads;
  __shared__ int64_t s_turns[ROPE == kRopeNone ? 1 : kMaxHeadWidth / 2];
  const int lane = threadIdx.x & (lanes - 1);
  const int step = (int)gridDim.x * (kThreads / lanes);
  const int dx_size = a.dx_bf16 ? 2 : 4;
  const long long x_step = (walk.tokens ? a.xs.t : a.xs.h) * (int)sizeof(TX);
  const long long g_step = (walk.tokens ? a.gs.t : a.gs.h) * (int)sizeof(TG);
  const long long o_step = (walk.tokens ? a.ds.t : a.ds.h) * dx_size;
  Walk::At in, in_g, to;
  in.run = in_g.run = to.run = (int)((blockIdx.x * kThreads + threadIdx.x) / lanes);
  walk.open(in, a.s, a.H, a.xs, a.x, sizeof(TX));
  walk.open(in_g, a.s, a.H, a.gs, a.dout, sizeof(TG));
  walk.open(to, a.s, a.H, a.ds, a.dx, dx_size);
  int at[NU][2];
  uint32_t turns[NU];                                   // pairs of this lane that turn
#pragma unroll
  for (int k = 0; k < NU; ++k) {
    const Unit<ROPE, V> u(lane + k * lanes, a.d, a.rope.first, a.rope.dim);
#pragma unroll
    for (int i = 0; i < 2; ++i) at[k][i] = u.c[i];
    turns[k] = 0;
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (u.index(e, a.rope.first, a.rope.dim) >= 0) turns[k] |= 1u << e;
  }
  const auto ask = [&](int stage) {
    if (in.slot < in.len) {
#pragma unroll
      for (int k = 0; k < NU; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (at[k][i] >= 0) {
            SlotX::ask(s_raw, (stage * NU + k) * 2 + i, (const TX*)in.p + at[k][i]);
            SlotG::ask(s_g, (stage * NU + k) * 2 + i, (const TG*)in_g.p + at[k][i]);
          }
      if (ROPE != kRopeNone && a.pos != nullptr && (walk.tokens || in.slot == 0))
        PosSlot::ask(s_pos, stage, a.pos + in.bi * a.pos_stride + in.t + in.slot);
    }
    copies_commit();
    in.p += x_step;
    in_g.p += g_step;
    if (++in.slot >= walk.run) {
      in.run += step;
      in_g.run = in.run;
      walk.open(in, a.s, a.H, a.xs, a.x, sizeof(TX));
      walk.open(in_g, a.s, a.H, a.gs, a.dout, sizeof(TG));
    }
  };
#pragma unroll 1
  for (int i = 0; i < kStages; ++i) ask(i);
#pragma unroll
  for (int k = 0; k < NU; ++k)
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (at[k][i] < 0)
        for (int q = 0; q < kStages; ++q)
          SlotX::zero(s_raw, (q * NU + k) * 2 + i), SlotG::zero(s_g, (q * NU + k) * 2 + i);
  float2 w[NU][2][V / 2], dw[NU][2][V / 2], db[DB ? NU : 1][2][V / 2];
  float cs[NU][V], sn[NU][V];
#pragma unroll
  for (int k = 0; k < NU; ++k) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      Pack<float, V> pw;
#pragma unroll
      for (int e = 0; e < V; ++e) pw.w[e] = __float_as_uint(1.f);
      if (at[k][i] >= 0 && a.weight != nullptr) pw.load(a.weight + at[k][i]);
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        w[k][i][e] = pw.two(e);
        dw[k][i][e] = make_float2(0.f, 0.f);
        if (DB) db[k][i][e] = make_float2(0.f, 0.f);
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
  const bool layer = DB && a.kind == kNormLayer;
  int stage = 0;
#pragma unroll 1
  for (int left = walk.rounds * walk.run; left > 0; --left) {
    copies_wait<kStages - 1>();
    const bool live = to.slot < to.len;
    VecX x[NU][2];
    float2 dy[NU][2][V / 2];
#pragma unroll
    for (int k = 0; k < NU; ++k)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        VecG g;
        SlotX::take(s_raw, (stage * NU + k) * 2 + i, x[k][i]);
        SlotG::take(s_g, (stage * NU + k) * 2 + i, g);
#pragma unroll
        for (int e = 0; e < V / 2; ++e) dy[k][i][e] = g.two(e);
      }
    if constexpr (ROPE != kRopeNone) {
      if (walk.tokens || to.slot == 0) {                // another token
        int p = to.t + to.slot;
        if (a.pos != nullptr) {
          Word v;
          PosSlot::take(s_pos, stage, v);
          p = (int)v.w[0];
        }
#pragma unroll
        for (int k = 0; k < NU; ++k) {
          const Unit<ROPE, V> un(lane + k * lanes, a.d, a.rope.first, a.rope.dim);
          unit_cos_sin<ROPE, V>(un, turns[k], s_turns, a.rope, p, cs[k], sn[k]);
        }
      }
#pragma unroll
      for (int k = 0; k < NU; ++k) turn_unit<ROPE, V>(dy[k], cs[k], sn[k], turns[k]);
    }
    ask(stage);
    stage = stage + 1 == kStages ? 0 : stage + 1;
    float mean[1] = {0.f};
    if (DB && layer) {
      float2 t = make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < NU; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < V / 2; ++e) t = add2(t, x[k][i].two(e));
      mean[0] = t.x + t.y;
      group_sums(mean, lanes);
      mean[0] *= -inv_n;
    }
    constexpr int kSums = DB ? 3 : 2;                   // squares, g xc, g
    float sums[kSums];
    {
      float2 q = make_float2(0.f, 0.f), gx = q, gs = q;
#pragma unroll
      for (int k = 0; k < NU; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < V / 2; ++e) {
            float2 y = x[k][i].two(e);
            if (DB) y = add2(y, make_float2(mean[0], mean[0]));
            const float2 g = mul2(dy[k][i][e], w[k][i][e]);
            if (!DB || at[k][i] >= 0) q = fma2(y, y, q);
            gx = fma2(g, y, gx);
            if (DB) gs = add2(gs, g);
          }
      sums[0] = q.x + q.y;
      sums[1] = gx.x + gx.y;
      if (DB) sums[kSums - 1] = gs.x + gs.y;
    }
    group_sums(sums, lanes);
    const float r = rsqrtf(fmaf(sums[0], inv_n, a.eps));
    const float cx = -r * (r * (r * (sums[1] * inv_n)));   // (r^3 alone may overflow)
    const float c0 = DB && layer ? -r * (sums[kSums - 1] * inv_n) : 0.f;
#pragma unroll
    for (int k = 0; k < NU; ++k)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float2 o[V / 2];
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
          float2 y = x[k][i].two(e);
          if (DB) y = add2(y, make_float2(mean[0], mean[0]));
          const float2 rdy = mul2(dy[k][i][e], make_float2(r, r));
          if (live) {                                   // (behind the last row: what the places held)
            dw[k][i][e] = fma2(rdy, y, dw[k][i][e]);
            if (DB) db[k][i][e] = add2(db[k][i][e], dy[k][i][e]);
          }
          const float2 t = DB ? fma2(y, make_float2(cx, cx), make_float2(c0, c0))
                              : mul2(y, make_float2(cx, cx));
          o[e] = fma2(rdy, w[k][i][e], t);
        }
        if (at[k][i] < 0 || !live) continue;
        if (a.dx_bf16) {
          Pack<__nv_bfloat16, V> p;
#pragma unroll
          for (int e = 0; e < V / 2; ++e) p.set(e, o[e]);
          p.store((__nv_bfloat16*)to.p + at[k][i]);
        } else {
          Pack<float, V> p;
#pragma unroll
          for (int e = 0; e < V / 2; ++e) p.set(e, o[e]);
          p.store((float*)to.p + at[k][i]);
        }
      }
    to.p += o_step;
    if (++to.slot >= walk.run) {
      to.run += step;
      walk.open(to, a.s, a.H, a.ds, a.dx, dx_size);
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int wanted = (a.dweight != nullptr) + (DB && a.dbias != nullptr);
  if (wanted == 0) return;
  copies_wait<0>();
  __syncthreads();                                      // the rows' places become the sums'
  float* s_sum = reinterpret_cast<float*>(s_raw);       // [warps][wanted][d]
  const int warp = threadIdx.x >> 5;
  const auto put = [&](float v, int c, int which, bool on) {
    for (int o = lanes; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) < lanes && on) s_sum[(warp * wanted + which) * a.d + c] = v;
  };
#pragma unroll
  for (int k = 0; k < NU; ++k)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const bool on = at[k][i] >= 0;
        const float2 x = dw[k][i][e / 2];
        if (a.dweight != nullptr) put(e % 2 ? x.y : x.x, at[k][i] + e, 0, on);
        if constexpr (DB) {
          const float2 y = db[k][i][e / 2];
          if (a.dbias != nullptr) put(e % 2 ? y.y : y.x, at[k][i] + e, wanted - 1, on);
        }
      }
  __syncthreads();
  for (int c = threadIdx.x; c < wanted * a.d; c += kThreads) {
    float x = 0.f;
#pragma unroll
    for (int v = 0; v < kThreads / 32; ++v) x += s_sum[v * wanted * a.d + c];
    a.parts[(size_t)blockIdx.x * wanted * a.d + c] = x;
  }
}

template <typename TX, typename TG, int ROPE, int V, bool DB>
cudaError_t bwd(const RowsBwd& a, int ctas, cudaStream_t st) {
  constexpr size_t smem = (size_t)kStages * kThreads *
                          (16 * (sizeof(TX) + sizeof(TG)) + (ROPE != kRopeNone ? sizeof(int) : 0));
  static_assert(smem >= kThreads / 32 * 2 * kMaxHeadWidth * sizeof(float), "the sums take the rows' places");
  static SmemOnce once;
  const auto k = rows_bwd_kernel<TX, TG, ROPE, V, DB>;
  const cudaError_t e = once(k, smem);
  if (e != cudaSuccess) return e;
  const int lanes = row_lanes<V>(a.d);
  int used = ctas;
  const Walk w = make_walk(a.b, a.s, a.H, ROPE != kRopeNone, kThreads / lanes, 1, &used);
  k<<<(unsigned)ctas, kThreads, smem, st>>>(a, lanes, w);   // (a CTA without rows has sums of zero)
  count_launches(1);
  return cudaGetLastError();
}

template <typename TX, typename TG, bool DB>
cudaError_t bwd_rope(const RowsBwd& a, int ctas, cudaStream_t st) {
  constexpr int V = sizeof(TX) == 2 && sizeof(TG) == 2 ? 8 : 4;
  if (a.rope.turns == nullptr) return bwd<TX, TG, kRopeNone, V, DB>(a, ctas, st);
  if (!a.rope.half) return bwd<TX, TG, kRopeInter, V, DB>(a, ctas, st);
  if (half_by(V, a.rope)) return bwd<TX, TG, kRopeHalf, V, DB>(a, ctas, st);
  if (half_by(4, a.rope)) return bwd<TX, TG, kRopeHalf, 4, DB>(a, ctas, st);
  return bwd<TX, TG, kRopeHalf, 2, DB>(a, ctas, st);
}

template <typename TX, typename TG>
cudaError_t bwd_kind(const RowsBwd& a, int ctas, cudaStream_t st) {
  return a.kind == kNormRms && a.dbias == nullptr ? bwd_rope<TX, TG, false>(a, ctas, st)
                                                  : bwd_rope<TX, TG, true>(a, ctas, st);
}

}  // namespace

cudaError_t launch_rows_bwd(const RowsBwd& a, int ctas, cudaStream_t st) {
  using bf = __nv_bfloat16;
  if (a.x_bf16) return a.g_bf16 ? bwd_kind<bf, bf>(a, ctas, st) : bwd_kind<bf, float>(a, ctas, st);
  return a.g_bf16 ? bwd_kind<float, bf>(a, ctas, st) : bwd_kind<float, float>(a, ctas, st);
}

}  // namespace csa
