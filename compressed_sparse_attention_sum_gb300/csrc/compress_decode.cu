// csa_compress_decode: the compressor for the newest tokens of each sequence.
//
// Block j of a sequence is pooled from the positions [lo, (j + 1) ratio) of its
// window, those before the new tokens from the rings and the others from the
// call's rows: per channel the softmax of the scores weighs the rows.  The pooled
// row is cast once, normalised, turned by its position and cast again.
//
// One CTA a block: d / 8 threads have 8 channels each of one token at a time, the
// other threads other tokens, each with a running maximum and sum; they are joined
// through shared memory.
#include "cache_format.cuh"
#include "compress_decode.h"
#include "csa_kernels.h"
#include "rows.cuh"

namespace csa {
namespace {

constexpr int kThreads = 256;

struct Place {        // of a CTA's sequence
  int n, t0;          // its tokens; the first new position (may be negative)
  int first, count;   // blocks complete before the call, blocks that it completes
};

__device__ __forceinline__ Place place_of(const CompressDecodeArgs& a, int i, bool tell) {
  Place p;
  const int n = a.seq_lens[i];
  if (n < 0 && tell) set_status(a.status, kDevCheck, kSiteCacheRange);
  p.n = max(n, 0);
  p.t0 = p.n - a.s_q;
  p.first = max(p.t0, 0) / a.ratio;
  p.count = p.n / a.ratio - p.first;
  return p;
}

// New rows k in [k0, k1) of sequence i into the rings.
template <typename T>
__device__ __forceinline__ void store_ring(const CompressDecodeArgs& a, int i, int t0, int k0,
                                           int k1) {
  const T* kv = (const T*)a.kv + i * a.kv_bs;
  const T* sc = (const T*)a.score + i * a.sc_bs;
  T* kr = (T*)a.kv_ring + (long long)i * a.R * a.d;
  T* sr = (T*)a.score_ring + (long long)i * a.R * a.sw;
  k0 = max(k0, a.s_q - a.R);                    // of more than R tokens the last
  const int per = a.d / 8;
  for (int x = (int)threadIdx.x; x < (k1 - k0) * per; x += kThreads) {
    // Padding is skipped here and not by a bound max(k0, -t0): nvcc 13.0 was seen to take
    // that maximum of t0 instead of -t0 (next to max(t0, 0)), and no token was stored.
    const int k = k0 + x / per, c = x % per * 8, t = t0 + k;
    if (t < 0) continue;
    const int slot = t % a.R;
    float v[8];
    load8(kv + k * a.kv_rs + c, v);
    store8(kr + (long long)slot * a.d + c, v);
    if (a.sw != 1) {
      load8(sc + k * a.sc_rs + c, v);
      store8(sr + (long long)slot * a.d + c, v);
    } else if (c == 0) {
      sr[slot] = sc[k * a.sc_rs];
    }
  }
}

// Sum over the CTA, of a value of every thread; s has room for the warps.
__device__ __forceinline__ float cta_sum(float v, float* s) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  float x = 0.f;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) x += s[w];
  return x;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) compress_decode_kernel(CompressDecodeArgs a) {
  __shared__ float s_m[kThreads * 8], s_l[kThreads * 8], s_o[kThreads * 8];
  __shared__ float s_y[kMaxHeadWidth], s_r[2][kThreads / 32];
  const int i = blockIdx.y, tid = threadIdx.x, d = a.d;
  const Place p = place_of(a, i, blockIdx.x == 0 && tid == 0);
  if (blockIdx.x == 0 && tid == 0) {
    a.first[i] = p.first;
    a.counts[i] = p.count;
  }
  if (a.store_here)
    store_ring<T>(a, i, p.t0, (int)blockIdx.x * a.ratio,
                  min(a.s_q, ((int)blockIdx.x + 1) * a.ratio));
  if ((int)blockIdx.x >= p.count) return;
  const int j = p.first + (int)blockIdx.x;
  const int lo = max(0, (j + 1 - a.coff) * a.ratio), hi = (j + 1) * a.ratio;
  const int per = d / 8, slices = kThreads / per, slice = tid / per, c0 = (tid - slice * per) * 8;
  const T* kv = (const T*)a.kv + i * a.kv_bs;
  const T* sc = (const T*)a.score + i * a.sc_bs;
  const T* kr = (const T*)a.kv_ring + (long long)i * a.R * d;
  const T* sr = (const T*)a.score_ring + (long long)i * a.R * a.sw;
  if (slice < slices) {
    float m[8], l[8], o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) { m[e] = -INFINITY; l[e] = o[e] = 0.f; }
    for (int t = lo + slice; t < hi; t += slices) {
      const bool fresh = t >= p.t0;
      const int slot = fresh ? 0 : t % a.R;
      const T* row = fresh ? kv + (t - p.t0) * a.kv_rs : kr + (long long)slot * d;
      const T* srow = fresh ? sc + (t - p.t0) * a.sc_rs : sr + (long long)slot * a.sw;
      float v[8], z[8];
      load8(row + c0, v);
      if (a.sw == 1) {
        const float z1 = to_f(srow[0]);
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] = z1;
      } else {
        load8(srow + c0, z);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float mn = fmaxf(m[e], z[e]);
        // a score of -inf has no weight, also in front of the first finite one
        const float w = z[e] == -INFINITY ? 0.f : expf(z[e] - mn);
        const float old = m[e] == -INFINITY ? 0.f : expf(m[e] - mn);
        l[e] = fmaf(l[e], old, w);
        o[e] = fmaf(o[e], old, w * v[e]);
        m[e] = mn;
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      s_m[slice * d + c0 + e] = m[e];
      s_l[slice * d + c0 + e] = l[e];
      s_o[slice * d + c0 + e] = o[e];
    }
  }
  __syncthreads();
  constexpr int kPer = kMaxHeadWidth / kThreads;
  float y[kPer];
  float sum = 0.f;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int c = tid + k * kThreads;
    y[k] = 0.f;
    if (c >= d) continue;
    float m = -INFINITY, l = 0.f, o = 0.f;
    for (int s = 0; s < slices; ++s) m = fmaxf(m, s_m[s * d + c]);
    for (int s = 0; s < slices; ++s) {
      const float ms = s_m[s * d + c];
      const float w = ms == -INFINITY ? 0.f : expf(ms - m);
      l = fmaf(s_l[s * d + c], w, l);
      o = fmaf(s_o[s * d + c], w, o);
    }
    y[k] = to_f(from_f<T>(o / l));               // the pooled row's one cast
    sum += y[k];
  }
  if (a.kind != kNormNone) {
    const float mean = a.kind == kNormLayer ? cta_sum(sum, s_r[0]) / d : 0.f;
    float q = 0.f;
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (tid + k * kThreads < d) q = fmaf(y[k] - mean, y[k] - mean, q);
    const float rstd = 1.f / sqrtf(cta_sum(q, s_r[1]) / d + a.eps);
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int c = tid + k * kThreads;
      if (c >= d) continue;
      y[k] = (y[k] - mean) * rstd;
      if (a.weight != nullptr) y[k] *= a.weight[c];
      if (a.bias != nullptr) y[k] += a.bias[c];
    }
  }
  T* out = (T*)a.out + i * a.out_bs + (long long)blockIdx.x * d;
  const RopeArgs& r = a.rope;
  if (r.turns != nullptr) {
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (tid + k * kThreads < d) s_y[tid + k * kThreads] = y[k];
    __syncthreads();
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int c = tid + k * kThreads, at = c - r.first;
    if (c >= d) continue;
    float v = y[k];
    if (r.turns != nullptr && at >= 0 && at < r.dim) {
      const int half = r.dim / 2;
      const bool second = r.half ? at >= half : (at & 1) != 0;
      const int pair = r.half ? (second ? at - half : at) : at / 2;
      const int apart = r.half ? half : 1;
      const long long turn[2] = {r.turns[pair], 0};
      float2 c2, s2;
      turn_cos_sin(turn, hi - 1, &c2, &s2);
      const float cs = c2.x * r.scale, sn = s2.x * r.scale;
      v = second ? s_y[c - apart] * sn + v * cs : v * cs - s_y[c + apart] * sn;
    }
    out[c] = from_f<T>(v);
  }
}

// The rings' new rows, behind a pooling kernel that still read what they overwrite.
template <typename T>
__global__ void __launch_bounds__(kThreads) compress_decode_store_kernel(CompressDecodeArgs a,
                                                                         int rows) {
  const Place p = place_of(a, (int)blockIdx.y, false);
  const int k0 = max(0, a.s_q - a.R) + (int)blockIdx.x * rows;
  store_ring<T>(a, (int)blockIdx.y, p.t0, k0, min(a.s_q, k0 + rows));
}

template <typename T>
cudaError_t launch(CompressDecodeArgs a, cudaStream_t st) {
  // no slot that a pooled block reads is one that the new rows take
  a.store_here = a.R >= (long long)a.coff * a.ratio - 1 + a.s_q;
  const unsigned blocks = (unsigned)((a.s_q - 1) / a.ratio + 1);
  compress_decode_kernel<T><<<dim3(blocks, (unsigned)a.b), kThreads, 0, st>>>(a);
  count_launches(1);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.store_here) return e;
  const int rows = 16, n = a.s_q < a.R ? a.s_q : a.R;
  compress_decode_store_kernel<T>
      <<<dim3((unsigned)((n + rows - 1) / rows), (unsigned)a.b), kThreads, 0, st>>>(a, rows);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_compress_decode(const CompressDecodeArgs& a, bool bf16, cudaStream_t st) {
  return bf16 ? launch<__nv_bfloat16>(a, st) : launch<float>(a, st);
}

}  // namespace csa
