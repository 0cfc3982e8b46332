// csa_indexer_topk_decode on CUDA cores: fp32 scores of the newest tokens
// against the cached index keys, and the exact top-k of each row.
//
// Scores.  A CTA takes 128 keys of one sequence; a thread owns a key,
// dequantises it 32 channels at a time and adds its dot products with 16 heads
// of q (shared memory, read by all threads at the same address).  Bound by the
// FMA pipe: H_I d_I per (query, key).
//
// Select.  One CTA per query.  A radix select over the fp32 scores gives the
// K-th largest, T.  The set has to be that of the exact scores, so the blocks
// whose score lies within the possible error of T are scored again.  With eps
// a bound on the error of every fp32 score, a block above T + 2 eps belongs to
// the exact top-k and one below T - 2 eps does not; those between are close.
// eps follows from the rounding of a sum of products: a dot over d_I channels
// and a weighted sum over H_I heads err by less than (d_I + H_I + 16) 2^-24 of
// sum_h |w_h| |q_h| |k_j|.  |k_j| is bounded first through the largest group
// scale of the visible keys (6 or 448 times 2^e per channel), then, for the
// few blocks this leaves, by their actual norms.  A close block's dot products
// are then accumulated as fp32 pairs (the rounding error of each sum is itself
// summed; 2^-40 relative and better), one (block, head) per thread, and added
// over the heads in fp64.  The best of them fill the places that the blocks
// above T + 2 eps leave, ties to the lower block.
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
    if (j < vis) a.scores[row * a.slots + j] = total;
  }
  __syncthreads();
  if (tid == 0) {
    for (int k = 1; k < kScoreThreads / 32; ++k) s_scale[0] = max(s_scale[0], s_scale[k]);
    a.tile_scale[bi * a.tiles + tile] = s_scale[0];
  }
}

// ---------------------------------------------------------------------------
// select
// ---------------------------------------------------------------------------
constexpr int kSel = 512;            // threads
constexpr int kSelWarps = kSel / 32;

// Unsigned keys in the order of the floats they come from (-0 as +0).
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float order_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ unsigned long long order_key(double x) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(x + 0.0);
  return (u >> 63) ? ~u : u | 0x8000000000000000ull;
}

struct SelShared {
  int hist[256];
  int warp_n[kSelWarps];
  int digit, above;
  float part[kSelWarps];
};

// The k-th largest of the keys key(0) .. key(n - 1) (1 <= k <= n), and in
// *equal how many keys equal to it belong to the k largest.  Called by the
// whole CTA; 8 bits a pass, ended early when the chosen bin is taken whole.
template <typename Key, typename F>
__device__ Key radix_select(SelShared& sh, int n, int k, F key, int* equal) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Key prefix = 0, mask = 0;
  for (int shift = (int)sizeof(Key) * 8 - 8; shift >= 0; shift -= 8) {
    for (int e = tid; e < 256; e += kSel) sh.hist[e] = 0;
    __syncthreads();
    for (int j = tid; j < n; j += kSel) {
      const Key x = key(j);
      if ((x & mask) == prefix) atomicAdd(&sh.hist[(int)(x >> shift) & 255], 1);
    }
    __syncthreads();
    if (warp == 0) {
      // lane l holds bins 255 - 8l .. 248 - 8l, so that counts run from the top
      int c[8], sum = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        c[e] = sh.hist[255 - lane * 8 - e];
        sum += c[e];
      }
      int before = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
      }
      before -= sum;
      if (before < k && before + sum >= k) {     // exactly one lane
        int at = before;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (at < k && at + c[e] >= k) {
            sh.digit = 255 - lane * 8 - e;
            sh.above = at;
          }
          at += c[e];
        }
      }
    }
    __syncthreads();
    prefix |= (Key)sh.digit << shift;
    mask |= (Key)255 << shift;
    k -= sh.above;
    __syncthreads();
  }
  *equal = k;
  return prefix;
}

// Ordered compaction: emit(j, rank) for every j < n with pred(j), ranks in
// ascending j.  Returns the number of them.  Called by the whole CTA; warp v
// owns the v-th contiguous part.
template <typename P, typename E>
__device__ int compact(SelShared& sh, int n, P pred, E emit) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = ((n + kSel - 1) / kSel) * 32;
  const int j0 = min(warp * part, n), j1 = min(j0 + part, n);
  int c = 0;
  for (int j = j0 + lane; j - lane < j1; j += 32)
    c += __popc(__ballot_sync(0xffffffffu, j < j1 && pred(j)));
  if (lane == 0) sh.warp_n[warp] = c;
  __syncthreads();
  int before = 0, total = 0;
  for (int v = 0; v < kSelWarps; ++v) {
    if (v < warp) before += sh.warp_n[v];
    total += sh.warp_n[v];
  }
  for (int j = j0 + lane; j - lane < j1; j += 32) {
    const bool p = j < j1 && pred(j);
    const unsigned m = __ballot_sync(0xffffffffu, p);
    if (p) emit(j, before + __popc(m & ((1u << lane) - 1u)));
    before += __popc(m);
  }
  __syncthreads();
  return total;
}

__device__ __forceinline__ float block_sum(SelShared& sh, float v) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) sh.part[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.f;
  for (int k = 0; k < kSelWarps; ++k) t += sh.part[k];
  __syncthreads();
  return t;
}
__device__ __forceinline__ int block_count(SelShared& sh, int c) {
  c = __reduce_add_sync(0xffffffffu, c);
  if ((threadIdx.x & 31) == 0) sh.warp_n[threadIdx.x >> 5] = c;
  __syncthreads();
  int t = 0;
  for (int k = 0; k < kSelWarps; ++k) t += sh.warp_n[k];
  __syncthreads();
  return t;
}
__device__ __forceinline__ float block_max(SelShared& sh, float v) {
  v = warp_max(v);
  if ((threadIdx.x & 31) == 0) sh.part[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = sh.part[0];
  for (int k = 1; k < kSelWarps; ++k) t = fmaxf(t, sh.part[k]);
  __syncthreads();
  return t;
}

// The dot product of q and k over d channels as hi + lo: the products are
// split by an fma, the sums by the exact error of an addition.
template <typename T>
__device__ __forceinline__ double dot_pair(const T* q, const float* k, int d) {
  float hi = 0.f, lo = 0.f;
  for (int c0 = 0; c0 < d; c0 += 8) {
    float qv[8];
    load8(q + c0, qv);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float p = __fmul_rn(qv[e], k[c0 + e]);
      if (sizeof(T) == 4) lo += __fmaf_rn(qv[e], k[c0 + e], -p);   // bf16: the product is exact
      const float s = __fadd_rn(hi, p), bb = __fsub_rn(s, hi);
      lo += __fadd_rn(__fsub_rn(hi, __fsub_rn(s, bb)), __fsub_rn(p, bb));
      hi = s;
    }
  }
  return (double)hi + (double)lo;
}

template <typename T, int BITS>
__global__ void __launch_bounds__(kSel) index_select_kernel(const IndexDecodeArgs a) {
  extern __shared__ __align__(16) unsigned char dyn[];
  __shared__ SelShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long row = blockIdx.x;
  const int bi = (int)(row / a.s_q), i = (int)(row - (long long)bi * a.s_q);
  const int vis = index_vis(a, bi, i), K = a.topk;
  int32_t* out = a.out + row * K;
  if (vis <= K) {
    for (int k = tid; k < K; k += kSel) out[k] = k < vis ? k : -1;
    return;
  }
  float* score = a.scores + row * a.slots;
  int equal = 0;
  const uint32_t tkey = radix_select<uint32_t>(
      sh, vis, K, [&](int j) { return order_key(score[j]); }, &equal);
  const float tval = order_value(tkey);

  // error scale of a score per unit of |k_j|: delta * sum_h |w_h| |q_h|
  const T* q = (const T*)a.q + row * a.H * a.d;
  float aw = 0.f;
  for (int h = warp; h < a.H; h += kSelWarps) {
    float n2 = 0.f;
    for (int c = lane; c < a.d; c += 32) {
      const float v = to_f(q[h * a.d + c]);
      n2 = fmaf(v, v, n2);
    }
    n2 = warp_sum(n2);
    aw += fabsf(a.w[row * a.H + h]) * sqrtf(n2);
  }
  aw = block_sum(sh, lane == 0 ? aw : 0.f);
  const float delta = (float)(a.d + a.H + 16) * 5.9604645e-8f * aw;
  int big = 0;
  for (int t = tid; t * kIdxTile < vis; t += kSel) big = max(big, a.tile_scale[bi * a.tiles + t]);
  const float kmax = block_max(sh, (float)big);
  const float top = BITS == 4 ? 6.f : 448.f;
  float eps = delta * (scale_value((uint32_t)kmax) * top * sqrtf((float)a.d));

  // close blocks, first by the bound on |k_j|, then by the largest norm among them
  uint32_t lo = 0, hi = 0;
  auto bounds = [&](float e) {
    lo = min(tkey, order_key(tval - 2.f * e));
    hi = max(tkey, order_key(tval + 2.f * e));
  };
  bounds(eps);
  int32_t* list = a.list + row * a.slots;
  auto is_close = [&](int j) {
    const uint32_t k = order_key(score[j]);
    return k >= lo && k <= hi;
  };
  auto collect = [&]() {
    return compact(sh, vis, is_close, [&](int j, int at) { list[at] = j; });
  };
  int m = collect();
  if (eps > 0.f) {
    const int32_t* pages = a.table + (long long)bi * a.P;
    float norm = 0.f;
    for (int e = warp; e < m; e += kSelWarps) {
      long long code, scale;
      float n2 = 0.f;
      if (cache_row(a.cs, pages, list[e], &code, &scale, a.status)) {
        for (int c0 = lane * 8; c0 < a.d; c0 += 256) {
          float v[8];
          cache_load8<BITS>(a.cache + code, scale_value(a.cache[scale + c0 / 32]), c0, v);
#pragma unroll
          for (int k = 0; k < 8; ++k) n2 = fmaf(v[k], v[k], n2);
        }
      }
      norm = fmaxf(norm, sqrtf(warp_sum(n2)));
    }
    norm = block_max(sh, norm);
    const float tight = delta * norm * 1.0001f;
    if (tight < eps) {
      eps = tight;
      bounds(eps);
      m = collect();
    }
  }
  // places left by the blocks above the close ones
  int c = 0;
  for (int j = tid; j < vis; j += kSel) c += order_key(score[j]) > hi;
  const int need = K - block_count(sh, c);

  if (need < m && eps > 0.f) {
    // exact scores of the close blocks: HP threads a block, one per head
    double* ex = a.exact + row * a.slots;
    const int HP = (a.H + 31) / 32 * 32, per = kSel / HP;
    float* k_s = reinterpret_cast<float*>(dyn);                  // [per][d]
    double* part = reinterpret_cast<double*>(dyn + (size_t)per * a.d * sizeof(float));
    const int32_t* pages = a.table + (long long)bi * a.P;
    const int mine = tid / HP, h = tid - mine * HP;
    for (int e0 = 0; e0 < m; e0 += per) {
      const int n = min(per, m - e0);
      for (int e = tid; e < n * (a.d / 8); e += kSel) {
        const int s = e / (a.d / 8), c0 = (e - s * (a.d / 8)) * 8;
        long long code, scale;
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (cache_row(a.cs, pages, list[e0 + s], &code, &scale, a.status))
          cache_load8<BITS>(a.cache + code, scale_value(a.cache[scale + c0 / 32]), c0, v);
        store8(k_s + s * a.d + c0, v);
      }
      __syncthreads();
      if (mine < n) {
        double x = 0.0;
        if (h < a.H) {
          const double dot = dot_pair(q + h * a.d, k_s + mine * a.d, a.d);
          x = dot > 0.0 ? (double)a.w[row * a.H + h] * dot : 0.0;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (lane == 0) part[warp] = x;
      }
      __syncthreads();
      if (tid < n) {
        double x = 0.0;
        for (int k = 0; k < HP / 32; ++k) x += part[tid * (HP / 32) + k];
        ex[e0 + tid] = x;
      }
      __syncthreads();
    }
    // the `need` best of the m, ties to the lower block: their scores become
    // +inf, the others' -inf
    int eq = 0;
    const unsigned long long bar = radix_select<unsigned long long>(
        sh, m, need, [&](int e) { return order_key(ex[e]); }, &eq);
    compact(sh, m, [&](int e) { return order_key(ex[e]) == bar; },
            [&](int e, int rank) { score[list[e]] = rank < eq ? INFINITY : -INFINITY; });
    for (int e = tid; e < m; e += kSel) {
      const unsigned long long k = order_key(ex[e]);
      if (k != bar) score[list[e]] = k > bar ? INFINITY : -INFINITY;
    }
    __syncthreads();
    compact(sh, vis, [&](int j) { return order_key(score[j]) > hi; },
            [&](int j, int at) { if (at < K) out[at] = j; });
    return;
  }
  // every close block belongs to the set, or only ties are close: the first `need`
  compact(sh, m, [&](int) { return true; },
          [&](int e, int rank) { score[list[e]] = rank < need ? INFINITY : -INFINITY; });
  compact(sh, vis, [&](int j) { return order_key(score[j]) > hi; },
          [&](int j, int at) { if (at < K) out[at] = j; });
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

cudaError_t launch_index_select(const IndexDecodeArgs& a, bool bf16, int bits, cudaStream_t st) {
  const int HP = (a.H + 31) / 32 * 32, per = kSel / HP;
  const size_t smem = (size_t)per * a.d * sizeof(float) + kSelWarps * sizeof(double);
  const unsigned grid = (unsigned)(a.b * a.s_q);
  if (bf16) {
    if (bits == 4) index_select_kernel<__nv_bfloat16, 4><<<grid, kSel, smem, st>>>(a);
    else index_select_kernel<__nv_bfloat16, 8><<<grid, kSel, smem, st>>>(a);
  } else {
    if (bits == 4) index_select_kernel<float, 4><<<grid, kSel, smem, st>>>(a);
    else index_select_kernel<float, 8><<<grid, kSel, smem, st>>>(a);
  }
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace csa
