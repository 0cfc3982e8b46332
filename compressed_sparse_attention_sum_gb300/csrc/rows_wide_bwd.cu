// The gradient of the norms of rows of up to 32768 channels.
//
// With xc = x - mean, r = 1 / sqrt(mean(xc^2) + eps), xh = xc r and g = dout weight:
//   dx = r g - r mean(g) - xc r^3 mean(g xc),  dweight = sum dout xh,  dbias = sum dout
// (RMS: mean = 0 and no mean(g)).
//
// A CTA goes through rows; its threads keep their channels' sums of dweight and dbias in
// registers to the end.  The next rows of x and dout are on their way into the threads' own
// places of shared memory.  A row takes one barrier: of a warp's share of it, its mean, its
// squares and its sum of g xc about that mean and its sum of g go to shared memory, from
// which every thread joins the row's (exactly, at any mean: sum g (x - mean) = sum g (x - m_w)
// + (m_w - mean) sum g).
#include <algorithm>

#include "csa_kernels.h"
#include "rows.cuh"
#include "smem_once.h"

namespace csa {
namespace {

// DB: whether dbias may be wanted and the norm may be a layer norm; RMS norms without a bias
// have a kernel of their own, with fewer sums.
template <typename TX, typename TG, int C, bool DB, int STAGES, int THREADS, int PER_SM>
__global__ void __launch_bounds__(THREADS, PER_SM) norm_wide_bwd_kernel(RowsBwd a) {
  constexpr int V = sizeof(TX) == 2 && sizeof(TG) == 2 ? 8 : 4, NV = C / V;
  constexpr bool kKeep = C <= 16;
  static_assert(THREADS <= 512, "a warp's share for each of 16 lanes");
  using VecX = Pack<TX, V>;
  using VecG = Pack<TG, V>;
  using SlotX = VecSlot<VecX, 0>;                       // [stage][NV]
  using SlotG = VecSlot<VecG, 0>;
  extern __shared__ __align__(16) unsigned char s_raw[];
  __shared__ __align__(16) float4 s_part[2][THREADS / 32];
  __shared__ float s_count[THREADS / 32];               // elements of each warp
  const int nv = a.d / V, threads = blockDim.x, warps = threads / 32, v0 = threadIdx.x;
  unsigned char* s_g = s_raw + (size_t)STAGES * C * sizeof(TX) * threads;
  const int rows = a.H, row_step = gridDim.x;
  const bool layer = DB && a.kind == kNormLayer;
  const auto has = [&](int k) { return v0 + k * threads < nv; };
  long long asked = blockIdx.x;                         // the next row to ask for
  const auto ask = [&](int stage) {
    const TX* x = (const TX*)a.x + asked * a.xs.h;
    const TG* g = (const TG*)a.dout + asked * a.gs.h;
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (asked < rows && has(k)) {
        SlotX::ask(s_raw, stage * NV + k, x + (v0 + k * threads) * V);
        SlotG::ask(s_g, stage * NV + k, g + (v0 + k * threads) * V);
      }
    asked += row_step;
    copies_commit();
  };
#pragma unroll
  for (int i = 0; i < STAGES; ++i) ask(i);
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (!has(k))
      for (int i = 0; i < STAGES; ++i) SlotX::zero(s_raw, i * NV + k), SlotG::zero(s_g, i * NV + k);
  const auto weight = [&](int k, Pack<float, V>& w) {
#pragma unroll
    for (int e = 0; e < V; ++e) w.w[e] = __float_as_uint(1.f);
    if (has(k) && a.weight != nullptr) w.load(a.weight + (v0 + k * threads) * V);
  };
  Pack<float, V> w[kKeep ? NV : 1];
  if constexpr (kKeep) {
#pragma unroll
    for (int k = 0; k < NV; ++k) weight(k, w[k]);
  }
  float2 dw[NV][V / 2], db[DB ? NV : 1][V / 2];
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int e = 0; e < V / 2; ++e) {
      dw[k][e] = make_float2(0.f, 0.f);
      if (DB) db[k][e] = make_float2(0.f, 0.f);
    }
  if (threadIdx.x < warps) {
    int n = 0;
#pragma unroll
    for (int k = 0; k < NV; ++k) n += min(32, max(0, nv - k * threads - (int)threadIdx.x * 32));
    s_count[threadIdx.x] = (float)(n * V);
  }
  __syncthreads();
  const float inv_n = 1.f / a.d, mine = s_count[threadIdx.x / 32];
  const float inv_mine = mine > 0.f ? 1.f / mine : 0.f;
  int stage = 0, turn = 0;
#pragma unroll 1
  for (long long row = blockIdx.x; row < rows; row += row_step) {
    if constexpr (STAGES > 0) copies_wait<STAGES - 1>();
    VecX x[NV];
    VecG g[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if constexpr (STAGES > 0) {
        SlotX::take(s_raw, stage * NV + k, x[k]);
        SlotG::take(s_g, stage * NV + k, g[k]);
      } else if (has(k)) {
        x[k].load((const TX*)a.x + row * a.xs.h + (v0 + k * threads) * V);
        g[k].load((const TG*)a.dout + row * a.gs.h + (v0 + k * threads) * V);
      } else {
        x[k].clear(), g[k].clear();
      }
    }
    if constexpr (STAGES > 0) {
      ask(stage);
      stage = stage + 1 == STAGES ? 0 : stage + 1;
    }
    float m[1] = {0.f};
    if (DB && layer) {
      float2 t = make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < V / 2; ++e) t = add2(t, x[k].two(e));
      m[0] = t.x + t.y;
      group_sums(m, 32);
      m[0] *= inv_mine;
    }
    constexpr int kSums = DB ? 3 : 2;                   // squares, g xc, g
    float sums[kSums];
    float2 xc[NV][V / 2];                               // x less the warp's mean
    {
      float2 q = make_float2(0.f, 0.f), gx = q, gs = q;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        Pack<float, V> pw;
        if constexpr (kKeep)
          pw = w[k];
        else
          weight(k, pw);
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
          float2 y = x[k].two(e);
          if (DB) y = add2(y, make_float2(-m[0], -m[0]));
          xc[k][e] = y;
          const float2 gw = mul2(g[k].two(e), pw.two(e));
          if (!DB || has(k)) q = fma2(y, y, q);
          gx = fma2(gw, y, gx);
          if (DB) gs = add2(gs, gw);
        }
      }
      sums[0] = q.x + q.y;
      sums[1] = gx.x + gx.y;
      if (DB) sums[kSums - 1] = gs.x + gs.y;
    }
    group_sums(sums, 32);
    if ((threadIdx.x & 31) == 0)
      s_part[turn][threadIdx.x >> 5] =
          make_float4(m[0], sums[0], sums[1], DB ? sums[kSums - 1] : 0.f);
    __syncthreads();
    // lanes i and 16 + i have warp i's share; the row's sums are those over 16 lanes
    const int lane = threadIdx.x & 15;
    const float cnt = lane < warps ? s_count[lane] : 0.f;
    const float4 p = lane < warps ? s_part[turn][lane] : make_float4(0.f, 0.f, 0.f, 0.f);
    float mean[1] = {p.x * cnt}, all[kSums];
    if (DB && layer) group_sums(mean, 16);
    mean[0] = DB && layer ? mean[0] * inv_n : 0.f;
    const float off = DB ? p.x - mean[0] : 0.f;
    all[0] = DB ? fmaf(off * off, cnt, p.y) : p.y;
    all[1] = DB ? fmaf(off, p.w, p.z) : p.z;
    if (DB) all[kSums - 1] = layer ? p.w : 0.f;
    group_sums(all, 16);
    turn ^= 1;
    const float r = rsqrtf(fmaf(all[0], inv_n, a.eps));
    const float cx = -r * (r * (r * (all[1] * inv_n)));   // (r^3 alone may overflow)
    const float c0 = DB ? -r * (all[kSums - 1] * inv_n) : 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      Pack<float, V> pw;
      if constexpr (kKeep)
        pw = w[k];
      else
        weight(k, pw);
      float2 o[V / 2];
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        float2 y = xc[k][e];
        if (DB) y = add2(y, make_float2(m[0] - mean[0], m[0] - mean[0]));
        const float2 dy = g[k].two(e), rdy = mul2(dy, make_float2(r, r));
        dw[k][e] = fma2(rdy, y, dw[k][e]);
        if (DB) db[k][e] = add2(db[k][e], dy);
        const float2 t = DB ? fma2(y, make_float2(cx, cx), make_float2(c0, c0))
                            : mul2(y, make_float2(cx, cx));
        o[e] = fma2(rdy, pw.two(e), t);
      }
      if (!has(k)) continue;
      if (a.dx_bf16) {
        Pack<__nv_bfloat16, V> p;
#pragma unroll
        for (int e = 0; e < V / 2; ++e) p.set(e, o[e]);
        p.store((__nv_bfloat16*)a.dx + row * a.ds.h + (v0 + k * threads) * V);
      } else {
        Pack<float, V> p;
#pragma unroll
        for (int e = 0; e < V / 2; ++e) p.set(e, o[e]);
        p.store((float*)a.dx + row * a.ds.h + (v0 + k * threads) * V);
      }
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int wanted = (a.dweight != nullptr) + (DB && a.dbias != nullptr);
  float* to = a.parts + (size_t)blockIdx.x * wanted * a.d;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    if (!has(k)) continue;
    Pack<float, V> p;
    if (a.dweight != nullptr) {
#pragma unroll
      for (int e = 0; e < V / 2; ++e) p.set(e, dw[k][e]);
      p.store(to + (v0 + k * threads) * V);
    }
    if (DB && a.dbias != nullptr) {
#pragma unroll
      for (int e = 0; e < V / 2; ++e) p.set(e, db[k][e]);
      p.store(to + (size_t)(wanted - 1) * a.d + (v0 + k * threads) * V);
    }
  }
}

// Channels a thread, and the most threads and CTAs an SM, by the width.  16384 x 4096 bf16
// (floor 59 us), RMS / layer norm with a bias: 66 / 78 us; 8 channels a thread 66 / 115 (twice
// the warps, whose joins cost as much as their channels), 32 channels 80 / 143 (the layer norm's
// sums no longer fit the registers), two rows a barrier 88 / 98.  Other widths of 64M channels:
// 2048 68 / 78, 8192 68 / 82, 16384 77 / 133 (layer norms and biases spill 200 to 264 bytes a thread),
// 32768 149 / 251 (all spill); fp32 (floor 119) 2048 to 8192 130 / 141 to 145, 16384 130 / 211, 32768 295 / 444.
struct WideShape { int c, threads, per_sm; };
WideShape wide_shape(int n) {
  if (n <= 2048) return {16, 128, 4};
  if (n <= 4096) return {16, 256, 2};
  if (n <= 8192) return {16, 512, 1};
  if (n <= 16384) return {32, 512, 1};
  return {64, 512, 1};
}
int wide_threads(int n) {
  const int c = wide_shape(n).c;
  return (n + c * 32 - 1) / (c * 32) * 32;
}

template <typename TX, typename TG, int C, bool DB, int STAGES, int THREADS, int PER_SM>
cudaError_t bwd(const RowsBwd& a, int ctas, cudaStream_t st) {
  constexpr size_t a_thread = (size_t)STAGES * C * (sizeof(TX) + sizeof(TG));
  static SmemOnce once;
  const auto k = norm_wide_bwd_kernel<TX, TG, C, DB, STAGES, THREADS, PER_SM>;
  const cudaError_t e = once(k, a_thread * THREADS);
  if (e != cudaSuccess) return e;
  const int threads = wide_threads(a.d);
  k<<<(unsigned)ctas, threads, a_thread * threads, st>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

template <typename TX, typename TG, bool DB>
cudaError_t bwd_width(const RowsBwd& a, int ctas, cudaStream_t st) {
  constexpr int bytes = sizeof(TX) + sizeof(TG);        // a channel: 4, 6 or 8
  if (a.d <= 2048) return bwd<TX, TG, 16, DB, 3, 128, 4>(a, ctas, st);
  if (a.d <= 4096) return bwd<TX, TG, 16, DB, 3, 256, 2>(a, ctas, st);
  if (a.d <= 8192) return bwd<TX, TG, 16, DB, bytes == 4 ? 4 : 3, 512, 1>(a, ctas, st);
  if (a.d <= 16384) return bwd<TX, TG, 32, DB, bytes == 8 ? 1 : 2, 512, 1>(a, ctas, st);
  // two fp32 rows of 32768 channels are more than shared memory: read where they are used
  return bwd<TX, TG, 64, DB, bytes == 8 ? 0 : 1, 512, 1>(a, ctas, st);
}

template <typename TX, typename TG>
cudaError_t bwd_kind(const RowsBwd& a, int ctas, cudaStream_t st) {
  return a.kind == kNormRms && a.dbias == nullptr ? bwd_width<TX, TG, false>(a, ctas, st)
                                                  : bwd_width<TX, TG, true>(a, ctas, st);
}

}  // namespace

int rows_bwd_ctas(long long rows, int n) {
  if (n <= kMaxHeadWidth) {                             // 256 threads, 16 channels on each
    int lanes = 1;
    while (lanes * 16 < n) lanes *= 2;
    const long long at_once = 256 / lanes;
    return (int)std::max(1ll, std::min<long long>((rows + at_once - 1) / at_once, 2 * 152));
  }
  // with four rows a CTA or more its sums are a small part of what it moves
  const WideShape w = wide_shape(n);
  const long long most = w.threads * w.per_sm / wide_threads(n) * 152;
  return (int)std::min({rows, most, std::max(152ll, (rows + 3) / 4)});
}

cudaError_t launch_norm_wide_bwd(const RowsBwd& a, int ctas, cudaStream_t st) {
  using bf = __nv_bfloat16;
  if (a.x_bf16) return a.g_bf16 ? bwd_kind<bf, bf>(a, ctas, st) : bwd_kind<bf, float>(a, ctas, st);
  return a.g_bf16 ? bwd_kind<float, bf>(a, ctas, st) : bwd_kind<float, float>(a, ctas, st);
}

}  // namespace csa
