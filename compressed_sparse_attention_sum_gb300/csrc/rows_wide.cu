// Layer and RMS norm of rows of up to 32768 channels, one CTA a row (the formulas stand
// in rows_heads.cu), and the sums of the CTAs' shares of the weight's and the bias's
// gradient.
#include <algorithm>

#include "csa_kernels.h"
#include "rows.cuh"
#include "smem_once.h"

namespace csa {
namespace {

// Forward.  A thread has NV vectors of 16 bytes of every row of its CTA, the next rows on
// their way in its own places of shared memory, weight and bias in registers (beyond 32
// channels a thread they are read again for each row).  BATCH rows share a barrier: a warp's
// mean and its squares about that mean go to shared memory, and every thread joins the warps'
// (squares about means, with the count of each: no cancellation at any mean).
template <typename T, int NV, int KIND, int BATCH, int STAGES, int THREADS, int PER_SM>
__global__ void __launch_bounds__(THREADS, PER_SM) norm_wide_kernel(RowsFwd a) {
  constexpr int V = 16 / sizeof(T);
  static_assert(THREADS <= 512, "a warp's share for each of 16 lanes");
  using Vec = Pack<T, V>;
  using Slot = VecSlot<Vec, 0>;                         // [stage][row][NV]
  extern __shared__ __align__(16) unsigned char s_raw[];
  constexpr bool kKeep = NV * V <= 32;
  __shared__ __align__(16) float2 s_part[2][BATCH][THREADS / 32];
  __shared__ float s_count[THREADS / 32];               // elements of each warp
  const int nv = a.d / V, threads = blockDim.x, warps = threads / 32;
  const int v0 = threadIdx.x;                           // this thread's first vector
  const int rows = a.H, row_step = gridDim.x;
  const auto has = [&](int k) { return v0 + k * threads < nv; };
  long long asked = blockIdx.x;                         // the next row to ask for
  const auto ask = [&](int stage) {
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const T* x = (const T*)a.x + asked * a.xs.h;
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (asked < rows && has(k))
          Slot::ask(s_raw, (stage * BATCH + u) * NV + k, x + (v0 + k * threads) * V);
      asked += row_step;
    }
    copies_commit();
  };
#pragma unroll
  for (int i = 0; i < STAGES; ++i) ask(i);
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (!has(k))
      for (int i = 0; i < STAGES * BATCH; ++i) Slot::zero(s_raw, i * NV + k);
  const auto affine = [&](int k, Pack<float, V>& w, Pack<float, V>& c) {
#pragma unroll
    for (int e = 0; e < V; ++e) w.w[e] = __float_as_uint(1.f), c.w[e] = 0;
    if (has(k) && a.weight != nullptr) w.load(a.weight + (v0 + k * threads) * V);
    if (has(k) && a.bias != nullptr) c.load(a.bias + (v0 + k * threads) * V);
  };
  Pack<float, V> w[kKeep ? NV : 1], c[kKeep ? NV : 1];
  if constexpr (kKeep) {
#pragma unroll
    for (int k = 0; k < NV; ++k) affine(k, w[k], c[k]);
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
  for (long long row = blockIdx.x; row < rows; row += (long long)BATCH * row_step) {
    copies_wait<STAGES - 1>();
    Vec raw[BATCH][NV];
#pragma unroll
    for (int u = 0; u < BATCH; ++u)
#pragma unroll
      for (int k = 0; k < NV; ++k) Slot::take(s_raw, (stage * BATCH + u) * NV + k, raw[u][k]);
    ask(stage);
    stage = stage + 1 == STAGES ? 0 : stage + 1;
    float m[BATCH], q[BATCH];
    if constexpr (KIND == kNormLayer) {
#pragma unroll
      for (int u = 0; u < BATCH; ++u) {
        float2 t = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int e = 0; e < V / 2; ++e) t = add2(t, raw[u][k].two(e));
        m[u] = t.x + t.y;
      }
      group_sums(m, 32);
#pragma unroll
      for (int u = 0; u < BATCH; ++u) m[u] *= inv_mine;
    }
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      float2 t = make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (KIND == kNormLayer && !has(k)) continue;
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
          float2 y = raw[u][k].two(e);
          if (KIND == kNormLayer) y = add2(y, make_float2(-m[u], -m[u]));
          t = fma2(y, y, t);
        }
      }
      q[u] = t.x + t.y;
    }
    group_sums(q, 32);
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int u = 0; u < BATCH; ++u)
        s_part[turn][u][threadIdx.x >> 5] = make_float2(KIND == kNormLayer ? m[u] : 0.f, q[u]);
    }
    __syncthreads();
    // lanes i and 16 + i have warp i's share; the row's sums are those over 16 lanes
    float mean[BATCH], sq[BATCH];
    const int lane = threadIdx.x & 15;
    const float cnt = lane < warps ? s_count[lane] : 0.f;
    float2 p[BATCH];
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      p[u] = lane < warps ? s_part[turn][u][lane] : make_float2(0.f, 0.f);
      mean[u] = p[u].x * cnt;
      sq[u] = p[u].y;
    }
    if constexpr (KIND == kNormLayer) {
      group_sums(mean, 16);
#pragma unroll
      for (int u = 0; u < BATCH; ++u) {
        mean[u] *= inv_n;
        sq[u] = fmaf((p[u].x - mean[u]) * (p[u].x - mean[u]), cnt, sq[u]);
      }
    }
    group_sums(sq, 16);
    turn ^= 1;
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const float r = rsqrtf(fmaf(sq[u], inv_n, a.eps));
      const long long at = row + (long long)u * row_step;
      T* out = (T*)a.out + at * a.os.h;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        Vec o;
        Pack<float, V> pw, pc;
        if constexpr (kKeep)
          pw = w[k], pc = c[k];
        else
          affine(k, pw, pc);
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
          float2 y = raw[u][k].two(e);
          if (KIND == kNormLayer) y = add2(y, make_float2(-mean[u], -mean[u]));
          y = mul2(y, make_float2(r, r));
          o.set(e, fma2(y, pw.two(e), pc.two(e)));
        }
        if (has(k) && at < rows) o.store(out + (v0 + k * threads) * V);
      }
    }
  }
}

// A programmatic dependent of the kernel that wrote the parts: 32 columns a CTA, the parts
// dealt to its WARPS warps and joined in a fixed order.  (No __restrict__: parts are written
// while this kernel already runs, so they may not be read as constant data.)
template <int WARPS>
__global__ void __launch_bounds__(32 * WARPS) sum_parts_kernel(const float* parts, int ctas,
                                                               float* dweight, float* dbias, int n) {
  __shared__ float s[WARPS][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cols = n * ((dweight != nullptr) + (dbias != nullptr)), c = blockIdx.x * 32 + lane;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float x = 0.f;
  if (c < cols) {
    constexpr int kAtOnce = 10;                  // loads under way
    for (int p0 = warp; p0 < ctas; p0 += kAtOnce * WARPS) {
      float v[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k)
        v[k] = p0 + k * WARPS < ctas ? parts[(size_t)(p0 + k * WARPS) * cols + c] : 0.f;
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) x += v[k];
    }
  }
  s[warp][lane] = x;
  __syncthreads();
  // warp w joins the columns w, w + WARPS, ...
#pragma unroll
  for (int k = 0; k < 32; k += WARPS) {
    const int col = blockIdx.x * 32 + warp + k;
    x = warp_sum(lane < WARPS ? s[lane][warp + k] : 0.f);
    if (lane != 0 || col >= cols) continue;
    if (dweight == nullptr)
      dbias[col] = x;
    else if (col < n)
      dweight[col] = x;
    else
      dbias[col - n] = x;
  }
}

// C channels a thread, BATCH rows together, STAGES batches under way, at most THREADS threads
// a CTA and PER_SM of these an SM.
template <typename T, int C, int KIND, int BATCH, int STAGES, int THREADS, int PER_SM>
cudaError_t wide_fwd(const RowsFwd& a, cudaStream_t st) {
  constexpr size_t a_thread = (size_t)STAGES * BATCH * C * sizeof(T);
  static SmemOnce once;
  const auto k = norm_wide_kernel<T, C * (int)sizeof(T) / 16, KIND, BATCH, STAGES, THREADS, PER_SM>;
  const cudaError_t e = once(k, a_thread * THREADS);
  if (e != cudaSuccess) return e;
  const int threads = (a.d + C * 32 - 1) / (C * 32) * 32;
  const int ctas = std::min(a.H, THREADS * PER_SM / threads * 152);
  k<<<(unsigned)ctas, threads, a_thread * threads, st>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

// Channels a thread by the width, measured for 64M bf16 channels (floor 39.6 us): more of them
// mean fewer warps to join, fewer mean more CTAs that do not wait for one another's barriers.
// 1024: 48.6 us (16 channels 48.8, one warp a row 57); 2048: 44.6 (8: 51, 32: 48);
// 4096: 42.8 (16: 47, 8: 88); 8192: 42.8 (32: 44 to 50); 16384: 41.9 (16 with 1024 threads
// 88, two CTAs of a cluster a row 114); 32768: RMS 56.5, layer 75.5.  fp32 in the same shapes
// (floor 79.1), RMS / layer: 1024 to 16384 channels 88 to 92 / 90 to 95, 32768 104 / 118.
template <typename T, int KIND>
cudaError_t wide_fwd_width(const RowsFwd& a, cudaStream_t st) {
  constexpr bool half = sizeof(T) == 2;
  // rows for one CTA an SM, or two: nothing to overlap with, so as many threads as there are
  // (16 x 4096: 1.9 us, without this rule 2.5; 304 x 4096: 2.9 and 3.5; 152 x 1024: 1.9 and 2.0)
  if (a.H <= 2 * 152 && a.d <= 4096) return wide_fwd<T, 8, KIND, 1, 1, 512, 1>(a, st);
  if (a.d <= 1024) return wide_fwd<T, 8, KIND, 2, 3, 128, 6>(a, st);
  if (a.d <= 2048) return wide_fwd<T, 16, KIND, 2, 3, 128, 4>(a, st);
  if (a.d <= 4096) return wide_fwd<T, 32, KIND, 2, 2, 128, 3>(a, st);
  if (a.d <= 8192) return wide_fwd<T, 16, KIND, 2, half ? 3 : 2, 512, 1>(a, st);
  if (a.d <= 16384) return wide_fwd<T, 32, KIND, 1, 3, 512, 1>(a, st);
  return wide_fwd<T, 64, KIND, 1, half ? 2 : 1, 512, 1>(a, st);
}

}  // namespace

cudaError_t launch_norm_wide(const RowsFwd& a, cudaStream_t st) {
  using bf = __nv_bfloat16;
  if (a.kind == kNormRms)
    return a.x_bf16 ? wide_fwd_width<bf, kNormRms>(a, st) : wide_fwd_width<float, kNormRms>(a, st);
  return a.x_bf16 ? wide_fwd_width<bf, kNormLayer>(a, st)
                  : wide_fwd_width<float, kNormLayer>(a, st);
}

cudaError_t launch_sum_parts(const float* parts, int ctas, float* dweight, float* dbias, int n,
                             cudaStream_t st) {
  const int cols = n * ((dweight != nullptr) + (dbias != nullptr));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((cols + 31) / 32));
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  count_launches(1);
  // as many warps as run at once: of few columns all of a CTA's (4 x 32 columns of 304 parts),
  // of many eight (448 x 32 of 152 parts: 5.2 us, with 32 warps 9)
  if (cols >= 4096) {
    cfg.blockDim = dim3(32 * 8);
    return cudaLaunchKernelEx(&cfg, sum_parts_kernel<8>, parts, ctas, dweight, dbias, n);
  }
  cfg.blockDim = dim3(32 * 32);
  return cudaLaunchKernelEx(&cfg, sum_parts_kernel<32>, parts, ctas, dweight, dbias, n);
}

}  // namespace csa
