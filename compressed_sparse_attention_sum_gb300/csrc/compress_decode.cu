// csa_compress_decode: the compressor for the newest tokens of each sequence.
//
// Block j of a sequence is pooled from the positions [lo, (j + 1) ratio) of its
// window, those before the new tokens from the rings and the others from the
// call's rows: per channel the softmax of the scores weighs the rows.  The pooled
// row is cast once, normalised, turned by its position and cast again.
//
// Pooling: a thread has 8 channels and every `slices`-th token of a block, kTokens of them
// read together, with a running maximum, sum and weighted sum; the slices are joined through
// shared memory.  Blocks of few tokens have one slice, several of them share a CTA; long ones
// have as many slices as 512 threads allow (a block of 128 tokens x 512 channels is 256 KB:
// 8 slices of 16 tokens).  How a block is cut depends on ratio, coff and d alone, so its row
// does not depend on the calls that its tokens came in.  Then a warp takes a row.
#include "cache_format.cuh"
#include "compress_decode.h"
#include "csa_kernels.h"
#include "rows.cuh"
#include "smem_once.h"

namespace csa {
namespace {

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

// `rows` new rows from row k0 of sequence i on into the rings.
template <typename T>
__device__ __forceinline__ void store_ring(const CompressDecodeArgs& a, int i, int t0, int k0,
                                           int rows) {
  const T* kv = (const T*)a.kv + i * a.kv_bs;
  const T* sc = (const T*)a.score + i * a.sc_bs;
  T* kr = (T*)a.kv_ring + (long long)i * a.R * a.d;
  T* sr = (T*)a.score_ring + (long long)i * a.R * a.sw;
  const int per = a.d / 8;
  const int vecs = a.sw == 1 ? per + 1 : 2 * per;        // of a row (a score of width 1: one)
  constexpr int kAtOnce = 4;
  for (int x0 = (int)threadIdx.x; x0 < rows * vecs; x0 += kAtOnce * (int)blockDim.x) {
    Pack<T, 8> v[kAtOnce];
    T* to[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      // (rows of padding, before the sequence's first token, are skipped one by one)
      const int x = x0 + u * (int)blockDim.x, row = x / vecs, e = x - row * vecs;
      const int k = k0 + row, t = t0 + k;
      to[u] = nullptr;
      if (x >= rows * vecs || t < 0) continue;
      const long long slot = t % a.R;
      if (e >= per && a.sw == 1) {
        sr[slot] = sc[k * a.sc_rs];
        continue;
      }
      const T* from = e < per ? kv + k * a.kv_rs + e * 8 : sc + k * a.sc_rs + (e - per) * 8;
      to[u] = e < per ? kr + slot * a.d + e * 8 : sr + slot * a.d + (e - per) * 8;
      v[u].load(from);
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u)
      if (to[u] != nullptr) v[u].store(to[u]);
  }
}

// e^(z - m) of two channels' scores z under maxima m: the difference is formed first, so that a
// token at the maximum has weight 1 whatever the scores' common offset, also at the lowest values of
// the type (z log2 e - m log2 e leaves a residue of m's rounding, and infinity where that overflows).
// m = -inf (nothing but scores of -inf so far) counts as 0, so that such scores have no weight.
// (ex2.approx is within 2^-22 of itself; weights below 2^-126 are 0)
__device__ __forceinline__ float minus_max(float m) { return m == -INFINITY ? 0.f : -m; }
__device__ __forceinline__ float2 weight_of(float2 z, float2 minus_m) {
  const float2 x = mul2(add2(z, minus_m), make_float2(kLog2e, kLog2e));
  float2 w;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w.x) : "f"(x.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w.y) : "f"(x.y));
  return w;
}

template <typename T, int kTokens, int THREADS>
__global__ void __launch_bounds__(THREADS) compress_decode_kernel(CompressDecodeArgs a, int slices,
                                                                  int groups, int pool_ctas, int rows) {
  extern __shared__ __align__(16) float s_mem[];
  const int i = blockIdx.y, tid = threadIdx.x, d = a.d, per = d / 8, size = per * slices;
  if ((int)blockIdx.x >= pool_ctas) {            // the rings' new rows, beside the pooling
    const Place p = place_of(a, i, false);
    const int k0 = ((int)blockIdx.x - pool_ctas) * rows;
    store_ring<T>(a, i, p.t0, k0, min(rows, a.s_q - k0));
    return;
  }
  const RopeArgs& r = a.rope;
  const int dim = r.turns != nullptr ? r.dim : 0;
  const bool norm = a.kind != kNormNone;
  float* s_w = s_mem;                            // [d] weight, [d] bias
  int64_t* s_turns = reinterpret_cast<int64_t*>(s_mem + 2 * d);   // [d / 2]
  float* s_row = s_mem + 3 * d;                  // [groups][d]
  float* s_part = s_row + groups * d;            // [3][groups][slices][d]
  const int part = groups * slices * d;
  // what the end needs is under way while the lengths and the rows are read
  const auto fetch = [&](void* to, const void* from, int bytes) {
    for (int x = tid * 16; x < bytes; x += (int)blockDim.x * 16)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                       (uint32_t)__cvta_generic_to_shared((char*)to + x)),
                   "l"((const char*)from + x)
                   : "memory");
  };
  if (norm && a.weight != nullptr) fetch(s_w, a.weight, d * 4);
  if (norm && a.bias != nullptr) fetch(s_w + d, a.bias, d * 4);
  if (dim > 0) fetch(s_turns, r.turns, dim / 2 * 8 & ~15);
  copies_commit();
  if (tid == 0 && dim % 4 != 0) s_turns[dim / 2 - 1] = r.turns[dim / 2 - 1];
  const Place p = place_of(a, i, blockIdx.x == 0 && tid == 0);
  if (blockIdx.x == 0 && tid == 0) {
    a.first[i] = p.first;
    a.counts[i] = p.count;
  }
  const int b0 = (int)blockIdx.x * groups;       // this CTA's blocks of the call
  if (b0 >= p.count) return;
  const int g = tid / size, in_g = tid - g * size, slice = in_g / per, c0 = (in_g - slice * per) * 8;
  const bool live = g < groups && b0 + g < p.count;
  if (live) {
    const int j = p.first + b0 + g;
    // tokens counted from the window's start: a sequence may end at 2^31 - 1, where the step
    // past the last token would leave 32 bits
    const int lo = max(0, (j + 1 - a.coff) * a.ratio), len = (j + 1) * a.ratio - lo;
    const int held = p.t0 - lo;                  // tokens of the rings
    const T* kv = (const T*)a.kv + i * a.kv_bs;
    const T* sc = (const T*)a.score + i * a.sc_bs;
    const T* kr = (const T*)a.kv_ring + (long long)i * a.R * d;
    const T* sr = (const T*)a.score_ring + (long long)i * a.R * a.sw;
    float m[8], l[8], o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) { m[e] = -INFINITY; l[e] = o[e] = 0.f; }
    int slot = (lo + slice) % a.R;
#pragma unroll 1
    for (int t0 = slice; t0 < len; t0 += slices * kTokens) {
      Pack<T, 8> v[kTokens], z[kTokens];
#pragma unroll
      for (int k = 0; k < kTokens; ++k) {
        const int t = t0 + k * slices;
        if (t >= len) continue;
        const bool fresh = t >= held;
        const T* row = fresh ? kv + (t - held) * a.kv_rs : kr + (long long)slot * d;
        const T* srow = fresh ? sc + (t - held) * a.sc_rs : sr + (long long)slot * a.sw;
        v[k].load(row + c0);
        if (a.sw == 1) {
          const float z1 = to_f(srow[0]);
#pragma unroll
          for (int e = 0; e < 4; ++e) z[k].set(e, make_float2(z1, z1));
        } else {
          z[k].load(srow + c0);
        }
        slot += slices;                          // (slices <= coff * ratio / 8 < R)
        if (slot >= a.R) slot -= a.R;
      }
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        float2 top = make_float2(m[e], m[e + 1]);
#pragma unroll
        for (int k = 0; k < kTokens; ++k)
          if (t0 + k * slices < len) {
            const float2 x = z[k].two(e / 2);
            top.x = fmaxf(top.x, x.x);
            top.y = fmaxf(top.y, x.y);
          }
        const float2 minus = make_float2(minus_max(top.x), minus_max(top.y));
        const float2 old = weight_of(make_float2(m[e], m[e + 1]), minus);
        l[e] *= old.x, l[e + 1] *= old.y;
        o[e] *= old.x, o[e + 1] *= old.y;
        m[e] = top.x, m[e + 1] = top.y;
#pragma unroll
        for (int k = 0; k < kTokens; ++k)
          if (t0 + k * slices < len) {
            const float2 y = v[k].two(e / 2), w = weight_of(z[k].two(e / 2), minus);
            l[e] += w.x, l[e + 1] += w.y;
            o[e] = fmaf(w.x, y.x, o[e]), o[e + 1] = fmaf(w.y, y.y, o[e + 1]);
          }
      }
    }
    if (slices == 1) {
      float4* to = reinterpret_cast<float4*>(s_row + g * d + c0);
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = to_f(from_f<T>(o[e] / l[e]));   // the pooled row's one cast
      to[0] = make_float4(y[0], y[1], y[2], y[3]);
      to[1] = make_float4(y[4], y[5], y[6], y[7]);
    } else {
      float4* to = reinterpret_cast<float4*>(s_part + (g * slices + slice) * d + c0);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        to[h] = make_float4(m[4 * h], m[4 * h + 1], m[4 * h + 2], m[4 * h + 3]);
        to[h + part / 4] = make_float4(l[4 * h], l[4 * h + 1], l[4 * h + 2], l[4 * h + 3]);
        to[h + part / 2] = make_float4(o[4 * h], o[4 * h + 1], o[4 * h + 2], o[4 * h + 3]);
      }
    }
  }
  copies_wait<0>();
  __syncthreads();
  if (slices > 1) {
    for (int x = tid; x < groups * d; x += (int)blockDim.x) {
      const int gr = x / d, c = x - gr * d;
      if (b0 + gr >= p.count) break;
      const float* from = s_part + gr * slices * d + c;
      float top = -INFINITY, l = 0.f, o = 0.f;
#pragma unroll 8
      for (int s = 0; s < slices; ++s) top = fmaxf(top, from[s * d]);
      const float2 minus = make_float2(minus_max(top), minus_max(top));
#pragma unroll 4
      for (int s = 0; s < slices; s += 2) {      // (2 slices or more are an even number)
        const float2 w = weight_of(make_float2(from[s * d], from[(s + 1) * d]), minus);
        l = fmaf(from[part + s * d], w.x, l);
        o = fmaf(from[2 * part + s * d], w.x, o);
        l = fmaf(from[part + (s + 1) * d], w.y, l);
        o = fmaf(from[2 * part + (s + 1) * d], w.y, o);
      }
      s_row[x] = to_f(from_f<T>(o / l));         // the pooled row's one cast
    }
    __syncthreads();
  }
  const int lane = tid & 31;
  constexpr int kQuads = kMaxHeadWidth / 128;    // float4 of a lane
  for (int gr = tid >> 5; gr < groups && b0 + gr < p.count; gr += (int)blockDim.x / 32) {
    float4* y = reinterpret_cast<float4*>(s_row + gr * d);
    if (norm) {
      float4 v[kQuads];
      float mean = 0.f, q = 0.f;
#pragma unroll
      for (int k = 0; k < kQuads; ++k) {
        v[k] = lane + 32 * k < d / 4 ? y[lane + 32 * k] : make_float4(0.f, 0.f, 0.f, 0.f);
        mean += v[k].x + v[k].y + v[k].z + v[k].w;
      }
      mean = a.kind == kNormLayer ? warp_sum(mean) / d : 0.f;
#pragma unroll
      for (int k = 0; k < kQuads; ++k) {
        v[k].x -= mean, v[k].y -= mean, v[k].z -= mean, v[k].w -= mean;
        if (lane + 32 * k < d / 4)
          q += v[k].x * v[k].x + v[k].y * v[k].y + v[k].z * v[k].z + v[k].w * v[k].w;
      }
      const float rstd = rsqrtf(warp_sum(q) / d + a.eps);
#pragma unroll
      for (int k = 0; k < kQuads; ++k) {
        if (lane + 32 * k >= d / 4) continue;
        float4 w = make_float4(1.f, 1.f, 1.f, 1.f), c = make_float4(0.f, 0.f, 0.f, 0.f);
        if (a.weight != nullptr) w = reinterpret_cast<const float4*>(s_w)[lane + 32 * k];
        if (a.bias != nullptr) c = reinterpret_cast<const float4*>(s_w + d)[lane + 32 * k];
        y[lane + 32 * k] = make_float4(fmaf(v[k].x * rstd, w.x, c.x), fmaf(v[k].y * rstd, w.y, c.y),
                                       fmaf(v[k].z * rstd, w.z, c.z), fmaf(v[k].w * rstd, w.w, c.w));
      }
      __syncwarp();
    }
    if (dim > 0) {
      const int pos = (p.first + b0 + gr + 1) * a.ratio - 1;
      float* x = s_row + gr * d + r.first;
      for (int e = lane; e < dim / 2; e += 32) {
        const long long turn[2] = {s_turns[e], 0};
        float2 c2, s2;
        turn_cos_sin(turn, pos, &c2, &s2);
        const float cs = c2.x * r.scale, sn = s2.x * r.scale;
        float &u = x[r.half ? e : 2 * e], &v = x[r.half ? e + dim / 2 : 2 * e + 1];
        const float u0 = u, v0 = v;
        u = u0 * cs - v0 * sn;
        v = u0 * sn + v0 * cs;
      }
      __syncwarp();
    }
    T* out = (T*)a.out + i * a.out_bs + (long long)(b0 + gr) * d;
#pragma unroll
    for (int k = 0; k < kQuads; ++k) {
      const int c = lane + 32 * k;
      if (c >= d / 4) continue;
      const float4 v = y[c];
      Pack<T, 4> o;
      o.set(0, make_float2(v.x, v.y));
      o.set(1, make_float2(v.z, v.w));
      o.store(out + 4 * c);
    }
  }
}

// The rings' new rows, of more than a ring has the last, behind a pooling kernel that still
// read what they overwrite.
template <typename T>
__global__ void __launch_bounds__(256) compress_decode_store_kernel(CompressDecodeArgs a, int rows) {
  const Place p = place_of(a, (int)blockIdx.y, false);
  const int k0 = max(0, a.s_q - a.R) + (int)blockIdx.x * rows;
  store_ring<T>(a, (int)blockIdx.y, p.t0, k0, min(rows, a.s_q - k0));
}

// Rows of a CTA that stores: 8 vectors for each of 256 threads.
int store_rows(int d) { return std::max(1, 2048 / (d / 4)); }

template <typename T, int kTokens, int THREADS>
cudaError_t launch_pool(const CompressDecodeArgs& a, int slices, cudaStream_t st) {
  const int size = a.d / 8 * slices, blocks = (a.s_q - 1) / a.ratio + 1;
  const int groups = std::max(1, std::min(blocks, THREADS / size));
  const int threads = (groups * size + 31) / 32 * 32;
  const size_t smem = (size_t)a.d * sizeof(float) * (3 + groups * (slices > 1 ? 1 + 3 * slices : 1));
  static SmemOnce once;
  const auto k = compress_decode_kernel<T, kTokens, THREADS>;
  const cudaError_t e = once(k, (size_t)(3 * kMaxHeadWidth + THREADS * (8 + 24)) * sizeof(float));
  if (e != cudaSuccess) return e;
  const int pool = (blocks - 1) / groups + 1, rows = store_rows(a.d);   // (blocks may be 2^31 - 1)
  const int store = a.store_here ? (a.s_q + rows - 1) / rows : 0;
  k<<<dim3((unsigned)(pool + store), (unsigned)a.b), threads, smem, st>>>(a, slices, groups, pool, rows);
  count_launches(1);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch(CompressDecodeArgs a, cudaStream_t st) {
  // no slot that a pooled block reads is one that the new rows take
  a.store_here = a.R >= (long long)a.coff * a.ratio - 1 + a.s_q;
  constexpr int kTokens = sizeof(T) == 2 ? 8 : 4;
  int slices = 1;
  while (slices * 2 * 8 <= a.coff * a.ratio && a.d / 8 * slices * 2 <= 512 && slices < 32) slices *= 2;
  const cudaError_t e = a.d / 8 * slices <= 256 ? launch_pool<T, kTokens, 256>(a, slices, st)
                                                : launch_pool<T, kTokens, 512>(a, slices, st);
  if (e != cudaSuccess || a.store_here) return e;
  const int rows = store_rows(a.d), n = a.s_q < a.R ? a.s_q : a.R;
  compress_decode_store_kernel<T>
      <<<dim3((unsigned)((n + rows - 1) / rows), (unsigned)a.b), 256, 0, st>>>(a, rows);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_compress_decode(const CompressDecodeArgs& a, bool bf16, cudaStream_t st) {
  return bf16 ? launch<__nv_bfloat16>(a, st) : launch<float>(a, st);
}

}  // namespace csa
