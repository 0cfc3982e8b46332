// Indexer scores of csa_indexer_topk_decode on CUDA cores: fp32 queries, and
// widths the tensor-core kernel does not take.
//
// A CTA takes 128 keys of one sequence; a thread owns a key, dequantises it
// eight channels at a time and adds its dot products with 16 heads of q
// (shared memory, read by all threads at the same address).  Bound by the FMA
// pipe: H_I d_I per (query, key).
#include <cuda_bf16.h>

#include "indexer_decode.h"

namespace csa {
namespace {

constexpr int kScoreThreads = kIdxTile;
constexpr int kHeadChunk = 16;

template <typename T, int BITS>
__global__ void __launch_bounds__(kScoreThreads) index_scores_simt_kernel(
    const IndexDecodeArgs a) {
  extern __shared__ __align__(16) float q_s[];   // [kHeadChunk][d]
  __shared__ int s_scale[kScoreThreads / 32];
  __shared__ float2 s_range[kScoreThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tile = blockIdx.x, bi = blockIdx.y, tid = threadIdx.x;
  const int d = a.d, j = tile * kIdxTile + tid;
  int most = 0;
  for (int i = 0; i < a.s_q; ++i) most = max(most, index_vis(a, bi, i));
  if (tile * kIdxTile >= most) return;           // CTA-uniform

  long long code = 0, scale = 0;
  const bool live = j < most && cache_row(a.cs, a.table + (long long)bi * a.P, j, &code, &scale,
                                          a.status);
  int big = 0;
  if (live)
    for (int g = 0; g < d / 32; ++g) big = max(big, (int)a.cache[scale + g]);
  big = __reduce_max_sync(0xffffffffu, big);
  if ((tid & 31) == 0) s_scale[tid >> 5] = big;

  for (int i = 0; i < a.s_q; ++i) {
    const int vis = index_vis(a, bi, i);
    if (vis <= a.topk || vis <= tile * kIdxTile) continue;   // CTA-uniform: no score is read
    const long long row = (long long)bi * a.s_q + i;
    float total = 0.f;
    for (int h0 = 0; h0 < a.H; h0 += kHeadChunk) {
      const int nh = min(kHeadChunk, a.H - h0);
      __syncthreads();
      for (int e = tid; e < kHeadChunk * d; e += kScoreThreads)
        q_s[e] = e < nh * d ? to_f(((const T*)a.q)[(row * a.H + h0) * d + e]) : 0.f;
      __syncthreads();
      if (!live) continue;
      float dot[kHeadChunk];
#pragma unroll
      for (int h = 0; h < kHeadChunk; ++h) dot[h] = 0.f;
      for (int c0 = 0; c0 < d; c0 += 8) {
        float k[8];
        cache_load8<BITS>(a.cache + code, scale_value(a.cache[scale + c0 / 32]), c0, k);
#pragma unroll
        for (int h = 0; h < kHeadChunk; ++h) {
          const float4 q0 = *reinterpret_cast<const float4*>(q_s + h * d + c0);
          const float4 q1 = *reinterpret_cast<const float4*>(q_s + h * d + c0 + 4);
          dot[h] = fmaf(q0.x, k[0], dot[h]);
          dot[h] = fmaf(q0.y, k[1], dot[h]);
          dot[h] = fmaf(q0.z, k[2], dot[h]);
          dot[h] = fmaf(q0.w, k[3], dot[h]);
          dot[h] = fmaf(q1.x, k[4], dot[h]);
          dot[h] = fmaf(q1.y, k[5], dot[h]);
          dot[h] = fmaf(q1.z, k[6], dot[h]);
          dot[h] = fmaf(q1.w, k[7], dot[h]);
        }
      }
#pragma unroll
      for (int h = 0; h < kHeadChunk; ++h)
        if (h < nh) total = fmaf(a.w[row * a.H + h0 + h], fmaxf(dot[h], 0.f), total);
    }
    if (total != total) total = -INFINITY;               // the select's order has no NaN
    if (j < vis) a.scores[row * a.slots + j] = total;
    float mn = j < vis ? total : INFINITY, mx = j < vis ? total : -INFINITY;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mx = warp_max(mx);
    if ((tid & 31) == 0) s_range[tid >> 5] = make_float2(mn, mx);
    __syncthreads();
    if (tid == 0) {
      int scale_byte = 0;
      for (int k = 0; k < kScoreThreads / 32; ++k) {
        mn = fminf(mn, s_range[k].x);
        mx = fmaxf(mx, s_range[k].y);
        scale_byte = max(scale_byte, s_scale[k]);
      }
      const float top = scale_value((uint32_t)scale_byte) * (BITS == 4 ? 6.f : 448.f);
      a.tile_info[row * a.tiles + tile] = make_float4(top * sqrtf((float)d) * 1.000001f, mn, mx, 0.f);
    }
  }
}

}  // namespace

cudaError_t launch_index_scores_simt(const IndexDecodeArgs& a, bool bf16, int bits,
                                     cudaStream_t st) {
  const dim3 grid(a.tiles, a.b);
  const size_t smem = (size_t)kHeadChunk * a.d * sizeof(float);
  if (bf16) {
    if (bits == 4) index_scores_simt_kernel<__nv_bfloat16, 4><<<grid, kScoreThreads, smem, st>>>(a);
    else index_scores_simt_kernel<__nv_bfloat16, 8><<<grid, kScoreThreads, smem, st>>>(a);
  } else {
    if (bits == 4) index_scores_simt_kernel<float, 4><<<grid, kScoreThreads, smem, st>>>(a);
    else index_scores_simt_kernel<float, 8><<<grid, kScoreThreads, smem, st>>>(a);
  }
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace csa
