// csa_attn_decode on CUDA cores, for any head count and width, and the
// kernel that joins the parts of a query.
//
// A CTA takes one (query, group of 8 heads, split of the query's slots).  Tile
// by tile, the slots' rows are dequantised into shared memory as fp32 (one
// conversion serves the CTA's heads, and the row serves as key and as value),
// and each warp runs the online softmax of its head: lanes split the channels.
// The arithmetic is fp32 throughout, which is what fp32 queries need; it is
// bound by the FMA pipe (4 H d flops a slot) and shared-memory reads.
#include <cuda_bf16.h>

#include "attn_decode.h"
#include "smem_once.h"
#include "tcgen05.cuh"

namespace csa {
namespace {

constexpr int kWarps = 8;            // heads of a CTA
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 32;            // slots of a shared-memory tile

template <typename T, int BITS, int ND>   // ND = 32-channel groups held per warp (d <= 32 ND)
__global__ void __launch_bounds__(kThreads) attn_decode_simt_kernel(const AttnDecodeArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ __align__(16) float kv_s[];   // [kTile][d]
  __shared__ long long s_code[kTile], s_scale[kTile];
  __shared__ int s_ok[kTile];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int d = a.d, ng = d / 32;
  const long long row = blockIdx.x;
  const int bi = (int)(row / a.s_q), i = (int)(row - (long long)bi * a.s_q);
  const int split = blockIdx.y, h = blockIdx.z * kWarps + warp;
  const bool has_head = h < a.H;
  const DecodeRow r = decode_row(a, bi, i);
  const int tiles = (r.slots + kDecodeTile - 1) / kDecodeTile;
  const int s_begin = (int)((long long)tiles * split / a.parts) * kDecodeTile;
  const int s_end = min((int)((long long)tiles * (split + 1) / a.parts) * kDecodeTile, r.slots);

  float qv[ND], acc[ND];
#pragma unroll
  for (int k = 0; k < ND; ++k) {
    qv[k] = has_head && k < ng
                ? to_f(((const T*)a.q)[(row * a.H + h) * d + k * 32 + lane]) * (a.scale * kLog2e)
                : 0.f;
    acc[k] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int s0 = s_begin; s0 < s_end; s0 += kTile) {
    const int n = min(kTile, s_end - s0);
    __syncthreads();
    if (tid < n) {
      long long c = 0, sc = 0;
      s_ok[tid] = decode_slot(a, r, bi, row, s0 + tid, &c, &sc);
      s_code[tid] = c;
      s_scale[tid] = sc;
    }
    __syncthreads();
    for (int e = tid; e < n * (d / 8); e += kThreads) {
      const int s = e / (d / 8), c0 = (e - s * (d / 8)) * 8;
      float v[8];
      if (s_ok[s]) {
        cache_load8<BITS>(a.cache + s_code[s], scale_value(a.cache[s_scale[s] + c0 / 32]), c0, v);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = 0.f;
      }
      store8(kv_s + s * d + c0, v);
    }
    __syncthreads();
    if (!has_head) continue;
    for (int s = 0; s < n; ++s) {
      if (!s_ok[s]) continue;
      float x = 0.f;
#pragma unroll
      for (int k = 0; k < ND; ++k)
        if (k < ng) x = fmaf(qv[k], kv_s[s * d + k * 32 + lane], x);
      x = warp_sum(x);
      const float m2 = fmaxf(m, x);
      const float f = exp2f(m - m2), p = exp2f(x - m2);   // m = -inf: f = 0
      l = fmaf(l, f, p);
#pragma unroll
      for (int k = 0; k < ND; ++k)
        if (k < ng) acc[k] = fmaf(p, kv_s[s * d + k * 32 + lane], acc[k] * f);
      m = m2;
    }
  }
  if (!has_head) return;
  if (a.parts > 1) {
    const long long at = (row * a.parts + split) * a.H + h;
#pragma unroll
    for (int k = 0; k < ND; ++k)
      if (k < ng) a.part_o[at * d + k * 32 + lane] = acc[k];
    if (lane == 0) a.part_ml[at] = make_float2(m, l);
    return;
  }
  const float sink2 = a.sink != nullptr ? sink_log2(a.sink[h]) : -INFINITY;
  const float mm = fmaxf(m, sink2);
  float f = 0.f, out_l = -INFINITY;
  if (mm > -INFINITY) {
    const float fm = exp2f(m - mm), total = fmaf(l, fm, exp2f(sink2 - mm));
    f = fm / total;
    out_l = sink2 > -INFINITY && l * fm == 0.f ? a.sink[h] : (mm + log2f(total)) * kLn2;
  }
#pragma unroll
  for (int k = 0; k < ND; ++k)
    if (k < ng) ((T*)a.o)[(row * a.H + h) * d + k * 32 + lane] = from_f<T>(acc[k] * f);
  if (lane == 0) a.lse[row * a.H + h] = out_l;
}

// One warp per (row, head): the parts' (m, l) give each part's weight, then the
// lanes add the parts' O, four channels each.  Launched as a programmatic
// dependent of the kernel that writes the parts.
template <typename T>
__global__ void __launch_bounds__(128) attn_decode_combine_kernel(const AttnDecodeArgs a) {
  const int lane = threadIdx.x & 31;
  const long long rh = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (rh >= (long long)a.b * a.s_q * a.H) return;
  const long long row = rh / a.H;
  const int h = (int)(rh - row * a.H);
  const float sink2 = a.sink != nullptr ? sink_log2(a.sink[h]) : -INFINITY;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const float2* ml = a.part_ml + row * a.parts * a.H + h;
  float m = sink2;
  for (int s = lane; s < a.parts; s += 32) m = fmaxf(m, ml[(long long)s * a.H].x);
  m = warp_max(m);
  float total = 0.f;
  for (int s = lane; s < a.parts; s += 32) {
    const float2 v = ml[(long long)s * a.H];
    if (v.y > 0.f) total = fmaf(v.y, exp2f(v.x - m), total);
  }
  total = warp_sum(total);
  const bool rows = total > 0.f;
  if (sink2 > -INFINITY) total += exp2f(sink2 - m);
  const float inv = total > 0.f ? 1.f / total : 0.f;
  for (int c = lane * 4; c < a.d; c += 128) {
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < a.parts; s0 += 4) {            // four parts' reads in flight
      float f[4];
      float4 o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int s = min(s0 + k, a.parts - 1);
        const float2 v = ml[(long long)s * a.H];
        f[k] = s0 + k < a.parts && v.y > 0.f ? exp2f(v.x - m) * inv : 0.f;
        o[k] = *reinterpret_cast<const float4*>(a.part_o + ((row * a.parts + s) * a.H + h) * a.d + c);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (f[k] > 0.f) {                                // an empty part's O was never written
          acc.x = fmaf(f[k], o[k].x, acc.x);
          acc.y = fmaf(f[k], o[k].y, acc.y);
          acc.z = fmaf(f[k], o[k].z, acc.z);
          acc.w = fmaf(f[k], o[k].w, acc.w);
        }
      }
    }
    T* dst = (T*)a.o + (row * a.H + h) * a.d + c;
    if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<uint2*>(dst) = make_uint2(umma::pack_bf16x2(acc.x, acc.y),
                                                  umma::pack_bf16x2(acc.z, acc.w));
    } else {
      *reinterpret_cast<float4*>(dst) = acc;
    }
  }
  if (lane == 0)
    a.lse[rh] = rows ? (m + log2f(total)) * kLn2 : sink2 > -INFINITY ? a.sink[h] : -INFINITY;
}

template <typename T, int BITS>
cudaError_t launch_simt(const AttnDecodeArgs& a, cudaStream_t st) {
  const dim3 grid((unsigned)(a.b * a.s_q), a.parts, (a.H + kWarps - 1) / kWarps);
  const size_t smem = (size_t)kTile * a.d * sizeof(float);
#define CSA_DEC(ND)                                                                              \
  do {                                                                                           \
    static SmemOnce once;                                                                        \
    const cudaError_t e = once(attn_decode_simt_kernel<T, BITS, ND>, kTile * 32 * ND * 4);        \
    if (e != cudaSuccess) return e;                                                              \
    attn_decode_simt_kernel<T, BITS, ND><<<grid, kThreads, smem, st>>>(a);                       \
  } while (0)
  if (a.d <= 64) CSA_DEC(2);
  else if (a.d <= 128) CSA_DEC(4);
  else if (a.d <= 256) CSA_DEC(8);
  else CSA_DEC(16);
#undef CSA_DEC
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_decode_combine(const AttnDecodeArgs& a, bool bf16, cudaStream_t st) {
  const long long rh = (long long)a.b * a.s_q * a.H;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((rh + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  count_launches(1);
  return bf16 ? cudaLaunchKernelEx(&cfg, attn_decode_combine_kernel<__nv_bfloat16>, a)
              : cudaLaunchKernelEx(&cfg, attn_decode_combine_kernel<float>, a);
}

cudaError_t launch_attn_decode_simt(const AttnDecodeArgs& a, bool bf16, int bits,
                                    cudaStream_t st) {
  const cudaError_t e = bf16 ? (bits == 4 ? launch_simt<__nv_bfloat16, 4>(a, st)
                                          : launch_simt<__nv_bfloat16, 8>(a, st))
                             : (bits == 4 ? launch_simt<float, 4>(a, st)
                                          : launch_simt<float, 8>(a, st));
  if (e != cudaSuccess || a.parts == 1) return e;
  return launch_attn_decode_combine(a, bf16, st);
}

}  // namespace csa
