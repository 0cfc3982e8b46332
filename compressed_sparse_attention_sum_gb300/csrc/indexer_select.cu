// The exact top-k of csa_indexer_topk_decode from its fp32 scores.
//
// The set has to be that of the exact scores, so blocks whose score lies
// within the possible error of the K-th largest, T, are scored again.  With
// eps a bound on the error of every fp32 score of the row, a block above
// T + 2 eps belongs to the exact top-k and one below T - 2 eps does not; those
// between are close.  eps = err * sum_h |w_h| |q_h| * max |k_j|, with |k_j|
// bounded by the keys' group scales and err by the roundings of the sums:
//   CUDA cores: d_I products and H_I heads added one by one, each addition
//     rounding by 2^-24 of the sum so far: (d_I + H_I + 16) 2^-24;
//   tensor cores: d_I / 16 steps, each of which adds 16 products to the sum so
//     far, all 17 cut at 2^-25 of the largest of them, and cuts their sum at
//     2^-23; H_I / 4 heads one by one in each of four chains:
//     (11 d_I / 16 + H_I / 4 + 8) 2^-24.  The cuts are measured, not documented:
//     next to a product of 1, products of 2^-25 count and 1.99 2^-26 do not, and
//     2^-23 is the step of the sum.  One product of 1 and 126 of 1.99 2^-26
//     lose 63 2^-24 of the 96 2^-24 at one head of 128 channels; N(0, 1) inputs
//     0.1 2^-24.
// Underflow adds less than 2^-149 to each of these roundings; a head's |q_h| is
// taken as at least 2^-84 for it (keys count as 2^-35 at least), and 2^-140 is
// added for the sum over the heads.  The product is formed with its exponent
// apart, as its factors may leave fp32 where it does not.  Where it does, and
// for keys above 2^60, the fp32 scores decide.
//
// A close block's dot products are accumulated as pairs of fp32 (the rounding
// error of every addition is itself summed, which leaves about 2^-40), as is
// their sum over the heads; the best fill the places that the blocks above
// T + 2 eps leave, ties to the lower block.
//
// A CTA takes a row and keeps its scores in shared memory as ordered integers;
// long rows take a cluster of up to eight CTAs, each a contiguous part of the
// scores.  A histogram of 1024 bins over the range of scores (the tiles'
// ranges come with them), whose counts the CTAs read from each other, gives
// the bin that T lies in (where outliers leave more than 512 scores in it,
// histograms over the bits of the keys, four rounds at most, narrow it down).
// The keys of that bin and of 2 eps around it are gathered in every CTA; T and
// the close blocks follow from ranks among them.  The heads of the close
// blocks' exact scores are dealt over the CTAs.  The blocks above set bits of a
// map as they are passed, the close ones that are chosen theirs; the map gives
// the ascending list.  A row with more than 512 keys around T (ties) is
// finished by the first CTA alone, by radix selects over global lists.
// Latency bounds it: barriers, dependent reads, reads of the other CTAs' shared
// memory (all of a step are in flight at once) and the chain of dependent
// additions of a dot product (d_I / 4 long: four threads share a head).  They are
// formed of q, k and w scaled by powers of two to about 1, where no error term
// underflows.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "indexer_decode.h"
#include "smem_once.h"

namespace csa {
namespace {

namespace cg = cooperative_groups;

constexpr int kSel = 1024;           // threads of a CTA
constexpr int kSelWarps = kSel / 32;
constexpr int kBins = kSel;          // one a thread
constexpr int kBinBits = 10;
constexpr int kNarrow = 256;         // keys of the bin around T
constexpr int kList = 512;           // keys around T that are ranked directly
constexpr int kMaxCluster = 8;
constexpr int kMaxStaged = 32768;    // scores a CTA keeps in shared memory

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

// x = mantissa * 2^exponent for a normal x, the mantissa in [1, 2); a mantissa of 0 for 0
// and NaN for NaN and the infinities.
constexpr int kNoExp = -100000;      // below every exponent
__device__ __forceinline__ int exponent(float x) { return (int)(__float_as_uint(x) >> 23 & 255u) - 127; }
__device__ __forceinline__ float mantissa(float x) {
  if (!(fabsf(x) < INFINITY)) return NAN;
  return x == 0.f ? 0.f : __uint_as_float((__float_as_uint(x) & 0x807fffffu) | 0x3f800000u);
}

struct __align__(16) SelShared {
  // read by the other CTAs of the cluster
  int hist[2][kBins];                // a round's counts; two, so that a round needs one barrier
  uint32_t list_key[kList];
  int list_j[kList];
  float2 exact[kList];               // close blocks' exact scores over this CTA's heads
  int n[2];                          // keys in the list, keys above it
  // this CTA's own
  alignas(16) uint32_t all_key[kList];   // read four at a time
  int all_j[kList];
  int close_j[kList];
  int close_page[kList];
  unsigned long long all_exact[kList];
  int warp_n[kSelWarps];
  int warp_m[kSelWarps];
  float part[kSelWarps];
  float2 pair[kSelWarps];
  int head_e[kMaxDecodeHI];          // exponents of |q_h|
  int bin, above, in_bin;
  uint32_t tkey;
  int digit, radix_above;            // the lone CTA's radix select
};

template <int CS>
__device__ __forceinline__ void cluster_sync() {
  if constexpr (CS > 1) cg::this_cluster().sync();
  else __syncthreads();
}
template <int CS, typename V>
__device__ __forceinline__ const V* peer(V* p, int rank) {
  if constexpr (CS > 1) return cg::this_cluster().map_shared_rank(p, rank);
  else return p;
}

static_assert(kSelWarps == 32, "a warp's lanes hold the warps' counts");

__device__ __forceinline__ int block_count(SelShared& sh, int c) {
  c = __reduce_add_sync(0xffffffffu, c);
  if ((threadIdx.x & 31) == 0) sh.warp_n[threadIdx.x >> 5] = c;
  __syncthreads();
  const int t = __reduce_add_sync(0xffffffffu, sh.warp_n[threadIdx.x & 31]);
  __syncthreads();
  return t;
}

// Ordered compaction: emit(j, rank) for every j in [0, n) with pred(j), ranks
// in ascending j.  Returns their number.  Warp v owns the v-th contiguous part.
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

// Numbers held as an unevaluated sum hi + lo of two fp32, about 2^-46.
__device__ __forceinline__ float2 pair_add(float2 a, float2 b) {
  const float s = __fadd_rn(a.x, b.x), t = __fsub_rn(s, a.x);
  const float e = __fadd_rn(__fsub_rn(a.x, __fsub_rn(s, t)), __fsub_rn(b.x, t));
  const float lo = __fadd_rn(e, __fadd_rn(a.y, b.y)), hi = __fadd_rn(s, lo);
  return make_float2(hi, __fsub_rn(lo, __fsub_rn(hi, s)));
}
__device__ __forceinline__ float2 pair_mul(float2 a, float w) {
  const float p = __fmul_rn(a.x, w);
  const float e = __fmaf_rn(a.y, w, __fmaf_rn(a.x, w, -p));
  const float hi = __fadd_rn(p, e);
  return make_float2(hi, __fsub_rn(e, __fsub_rn(hi, p)));
}
__device__ __forceinline__ float2 pair_shfl(float2 a, int o) {
  return make_float2(__shfl_xor_sync(0xffffffffu, a.x, o), __shfl_xor_sync(0xffffffffu, a.y, o));
}
__device__ __forceinline__ unsigned long long pair_key(float2 a) {
  return order_key((double)a.x + (double)a.y);
}

// The dot product of n channels of q, times qf (a power of two), and k: a product
// is split by an fma (exact already for bf16 q), a sum by the exact error of an
// addition.  Eight channels a step and no more unrolling: the code runs once a
// row, and fetching instructions would take longer than the loop.
template <typename T>
__device__ __forceinline__ float2 dot_pair(const T* q, float qf, const float* k, int n) {
  float hi = 0.f, lo = 0.f;
#pragma unroll 1
  for (int c = 0; c < n; c += 8) {
    float qv[8], kv[8];
    load8(q + c, qv);
    load8(k + c, kv);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = qv[e] * qf, p = __fmul_rn(x, kv[e]);
      if (sizeof(T) == 4) lo += __fmaf_rn(x, kv[e], -p);
      const float s = __fadd_rn(hi, p), t = __fsub_rn(s, hi);
      lo += __fadd_rn(__fsub_rn(hi, __fsub_rn(s, t)), __fsub_rn(p, t));
      hi = s;
    }
  }
  return pair_add(make_float2(hi, 0.f), make_float2(lo, 0.f));
}

// Sums over the heads [h0, h0 + nh) of the exact scores of blocks block(0) ..
// block(m - 1) on pages page(0) .. page(m - 1), each given to store(e, sum), all
// times the same power of two: |w_h| |q_h| is at most about 2^we, |k| 2^ke.
// Four threads a (block, head); scratch k_s holds the dequantised keys of a
// round (up to 32 of them).  Called by the whole CTA.
template <typename T, int BITS, typename B, typename P, typename S>
__device__ void score_exact(SelShared& sh, const IndexDecodeArgs& a, long long row, float* k_s,
                            int m, int h0, int nh, int we, int ke, B block, P page, S store) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int wpb = max(1, (nh + 7) / 8);                  // warps of a block
  const int per = kSelWarps / wpb;
  const int mine = warp / wpb, h = (warp - mine * wpb) * 8 + (lane >> 2), part = lane & 3;
  const int n4 = a.d / 4, pitch = a.d + 16;
  const T* qh = (const T*)a.q + (row * a.H + h0 + min(h, max(nh - 1, 0))) * a.d + part * n4;
  const int he = h < nh ? min(sh.head_e[h0 + h], 126) : 0;
  const float w = h < nh ? ldexpf(a.w[row * a.H + h0 + h], he - we) : 0.f;
  const float qf = pow2f(-he);
  for (int e0 = 0; e0 < m; e0 += per) {
    const int n = min(per, m - e0);
    // eight channels a thread: at most 32 keys of 256
    const int s = tid / (a.d / 8), c0 = (tid - s * (a.d / 8)) * 8;
    uint2 code = make_uint2(0u, 0u);
    uint32_t scale = 0;
    if (s < n) {
      const int j = block(e0 + s), pg = page(e0 + s);
      if ((unsigned)pg < (unsigned)a.cs.n_pages) {       // recorded by the score kernel
        const int r = j - page_index(a.cs, j) * a.cs.page_size;
        const uint8_t* base = a.cache + page_base(a.cs, pg);
        const uint8_t* src = base + row_code(a.cs, r) + c0 * BITS / 8;
        if constexpr (BITS == 4) code.x = __ldg(reinterpret_cast<const uint32_t*>(src));
        else code = __ldg(reinterpret_cast<const uint2*>(src));
        scale = __ldg(base + row_scale(a.cs, r) + c0 / 32);
      }
    }
    if (s < n) {
      const int se = (int)scale - ke;                    // below 1: nothing next to 2^ke
      const float f = scale_value(se < 1 ? 0u : (uint32_t)min(se, 254));
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if constexpr (BITS == 4) v[k] = code_e2m1(code.x >> (4 * k)) * f;
        else v[k] = code_e4m3((k < 4 ? code.x : code.y) >> (8 * (k & 3))) * f;
      }
      // quarters four banks apart: the lanes of a head read all four at once
      store8(k_s + s * pitch + c0 + c0 / n4 * 4, v);
    }
    __syncthreads();
    if (mine < n) {                                      // warp-uniform
      float2 x = make_float2(0.f, 0.f);
      if (h < nh) x = dot_pair(qh, qf, k_s + mine * pitch + part * (n4 + 4), n4);
#pragma unroll 1
      for (int o = 1; o < 32; o <<= 1) {                 // the quarters, then the heads
        x = pair_add(x, pair_shfl(x, o));
        if (o == 2) x = x.x > 0.f ? pair_mul(x, w) : make_float2(0.f, 0.f);   // hi has the sum's sign
      }
      if (lane == 0) sh.pair[warp] = x;
    }
    __syncthreads();
    if (warp < n) {                                      // block `warp` of the round
      float2 x = lane < wpb ? sh.pair[warp * wpb + lane] : make_float2(0.f, 0.f);
#pragma unroll 1
      for (int o = 1; o < 16; o <<= 1) x = pair_add(x, pair_shfl(x, o));
      if (lane == 0) store(e0 + warp, x);
    }
    __syncthreads();
  }
}

// The k-th largest of the keys key(0) .. key(n - 1) (1 <= k <= n), and in
// *equal how many keys equal to it belong to the k largest.  One CTA.
template <typename F>
__device__ unsigned long long radix_select(SelShared& sh, int n, int k, F key, int* equal) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unsigned long long prefix = 0, mask = 0;
  for (int shift = 56; shift >= 0; shift -= 8) {
    for (int e = tid; e < 256; e += kSel) sh.hist[0][e] = 0;
    __syncthreads();
    for (int j = tid; j < n; j += kSel) {
      const unsigned long long x = key(j);
      if ((x & mask) == prefix) atomicAdd(&sh.hist[0][(int)(x >> shift) & 255], 1);
    }
    __syncthreads();
    if (warp == 0) {
      int c[8], sum = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        c[e] = sh.hist[0][255 - lane * 8 - e];
        sum += c[e];
      }
      int before = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
      }
      before -= sum;
      if (before < k && before + sum >= k) {             // exactly one lane
        int at = before;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (at < k && at + c[e] >= k) {
            sh.digit = 255 - lane * 8 - e;
            sh.radix_above = at;
          }
          at += c[e];
        }
      }
    }
    __syncthreads();
    prefix |= (unsigned long long)sh.digit << shift;
    mask |= 255ull << shift;
    k -= sh.radix_above;
    __syncthreads();
  }
  *equal = k;
  return prefix;
}

// How many of all_key[0, m) are above x and equal to it (the entries up to the
// next multiple of four are 0, below every key but -NaN's).
__device__ __forceinline__ void count_keys(const SelShared& sh, int m, uint32_t x, int* above,
                                           int* equal) {
  int g = 0, q = 0;
#pragma unroll 4
  for (int e = 0; e < m; e += 4) {
    const uint4 y = *reinterpret_cast<const uint4*>(sh.all_key + e);
    g += (y.x > x) + (y.y > x) + (y.z > x) + (y.w > x);
    q += (y.x == x) + (y.y == x) + (y.z == x) + (y.w == x);
  }
  *above = g;
  *equal = q;
}

template <typename T, int BITS, int CS>
__global__ void __launch_bounds__(kSel) index_select_kernel(const IndexDecodeArgs a,
                                                            int staged_cap) {
  extern __shared__ __align__(16) unsigned char dyn[];
  __shared__ SelShared sh;
  uint32_t* staged = reinterpret_cast<uint32_t*>(dyn);
  uint32_t* bitmap = staged + staged_cap;
  float* k_s = reinterpret_cast<float*>(bitmap + staged_cap / 32);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = CS > 1 ? (int)cg::this_cluster().block_rank() : 0;
  const long long row = blockIdx.x / CS;
  const int bi = (int)(row / a.s_q), i = (int)(row - (long long)bi * a.s_q);
  const int vis = index_vis(a, bi, i), K = a.topk;
  const int32_t* pages = a.table + (long long)bi * a.P;
  int32_t* out = a.out + row * K;
  if (vis <= K) {                                        // every block, whatever the scores
    for (int k = rank * kSel + tid; k < K; k += CS * kSel) out[k] = k < vis ? k : -1;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }

  // sum_h |w_h| |q_h| = aw * 2^ae, from the row's own q and w: eight lanes a head
  static_assert(kSelWarps * 4 >= kMaxDecodeHI, "a head for every eight lanes");
  float aw = 0.f;
  int ae = kNoExp;
  {
    const int h = warp * 4 + (lane >> 3);
    float n2 = 0.f, small = 0.f, big = 0.f;              // |q_h|^2, and times 2^160, 2^-160
    if (h < a.H) {
      const T* q = (const T*)a.q + (row * a.H + h) * a.d;
#pragma unroll 2
      for (int c = (lane & 7) * 8; c < a.d; c += 64) {
        float v[8];
        load8(q + c, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float s = v[e] * 0x1p80f, g = v[e] * 0x1p-80f;
          n2 = fmaf(v[e], v[e], n2);
          small = fmaf(s, s, small);
          big = fmaf(g, g, big);
        }
      }
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {
      n2 += __shfl_xor_sync(0xffffffffu, n2, o);
      small += __shfl_xor_sync(0xffffffffu, small, o);
      big += __shfl_xor_sync(0xffffffffu, big, o);
    }
    if (h < a.H && (lane & 7) == 0) {
      int e = 0;
      if (!(n2 < 0x1p100f)) {
        n2 = big;
        e = 80;
      } else if (n2 < 0x1p-80f) {
        n2 = small > 0.f ? fmaxf(small, 0x1p-8f) : 0.f;
        e = -80;
      }
      const float x = sqrtf(n2);                         // 0, or a normal number
      e += exponent(x);
      sh.head_e[h] = x > 0.f ? e : 0;
      float w = fabsf(a.w[row * a.H + h]);
      if (w < 0x1p-100f) {
        w *= 0x1p49f;
        e -= 49;
      }
      aw = mantissa(x) * mantissa(w);                    // NaN and infinite inputs: NaN
      if (aw != 0.f) ae = e + exponent(w);
    }
  }
  auto align = [&]() {                                   // to the warp's largest exponent
    const int top = __reduce_max_sync(0xffffffffu, ae);
    aw *= ae - top < -126 ? 0.f : pow2f(ae - top);
    aw = warp_sum(aw);
    ae = top;
  };
  align();
  if (lane == 0) {
    sh.part[warp] = aw;
    sh.warp_m[warp] = ae;
  }
  for (int e = tid; e < kBins; e += kSel) sh.hist[0][e] = 0;
  if (tid == 0) {
    sh.bin = sh.above = sh.in_bin = 0;
    sh.tkey = 0u;
  }
  __syncthreads();
  aw = sh.part[lane];
  ae = sh.warp_m[lane];
  align();
  __syncthreads();

  asm volatile("griddepcontrol.wait;" ::: "memory");     // the scores

  const int seg = ((vis + CS - 1) / CS + 31) / 32 * 32;  // whole words of the bitmap
  const int j0 = min(rank * seg, vis), n = min(seg, vis - j0);
  float* score = a.scores + row * a.slots;
  const bool is_staged = seg <= staged_cap;              // the same in every CTA
  // chosen blocks of this part, a bit each
  uint32_t* bits = is_staged ? bitmap : reinterpret_cast<uint32_t*>(a.list + row * a.slots) + j0 / 32;
  float v0[8];                                           // the first scores, in flight with the tiles' data
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int j = e * kSel + tid;
    v0[e] = j < n ? score[j0 + j] : 0.f;
  }
  float kmax = 0.f, mn = INFINITY, mx = -INFINITY;
  for (int t = tid; t * kIdxTile < vis; t += kSel) {
    const float4 v = a.tile_info[row * a.tiles + t];
    kmax = fmaxf(kmax, v.x);
    mn = fminf(mn, v.y);
    mx = fmaxf(mx, v.z);
  }
  kmax = warp_max(kmax);
  mn = -warp_max(-mn);
  mx = warp_max(mx);
  if (lane == 0) {
    sh.part[warp] = kmax;
    sh.pair[warp] = make_float2(mn, mx);
  }
  __syncthreads();
  kmax = fmaxf(warp_max(sh.part[lane]), 0x1p-35f);
  mn = -warp_max(-sh.pair[lane].x);
  mx = warp_max(sh.pair[lane].y);
  const uint32_t lo0 = order_key(mn), hi0 = order_key(mx);
  uint32_t lo = lo0, hi = hi0;
  auto key = [&](int j) { return is_staged ? staged[j] : order_key(score[j0 + j]); };
  // Inputs beyond fp32 (their row's blocks are unspecified) leave the fp32 scores.
  float eps2 = aw > 0.f ? ldexpf(2.f * a.err * aw * kmax, ae) + 0x1p-140f : 0.f;
  if (!(eps2 < 3e38f)) eps2 = 0.f;
  const int ke = exponent(kmax);

  // ---- narrow [lo, hi] to a bin that holds the k-th largest key ------------------
  // Counts of the other CTAs' bins and this one's; returns the bin of the k-th
  // largest (from the top), how many lie above it and in it.
  int buf = 0;
  auto find_bin = [&](int k) {
    cluster_sync<CS>();
    // bins from the top: thread t holds one, of all CTAs
    const int bin = kBins - 1 - tid;
    int c = 0, pc[CS];
#pragma unroll
    for (int r = 0; r < CS; ++r) pc[r] = peer<CS>(sh.hist[buf], r)[bin];
#pragma unroll
    for (int r = 0; r < CS; ++r) c += pc[r];
    sh.hist[buf ^ 1][bin] = 0;         // last read before this barrier
    int before = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += v;
    }
    if (lane == 31) sh.warp_n[warp] = before;
    __syncthreads();
    int base = lane < warp ? sh.warp_n[lane] : 0;
    base = __reduce_add_sync(0xffffffffu, base);
    before += base - c;
    if (before < k && before + c >= k) {                 // exactly one thread
      sh.bin = bin;
      sh.above = before;
      sh.in_bin = c;
    }
    __syncthreads();
    buf ^= 1;
  };
  // First by value, 1024 bins between the smallest and largest score, counted
  // as the scores are read.  The bin is then widened by what rounding may have
  // moved a score across its edge.
  const float range = mx - mn, inv = (float)kBins / range;
  const bool by_range = vis > kNarrow && range < 3e38f && inv < 3e38f && inv > 0.f;   // finite, not NaN
  bool by_value = by_range;
  for (int jb = 0; jb < n; jb += 8 * kSel) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int j = jb + e * kSel + tid;
      v[e] = jb == 0 ? v0[e] : j < n ? score[j0 + j] : 0.f;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int j = jb + e * kSel + tid;
      if (j < n) {
        if (is_staged) staged[j] = order_key(v[e]);
        if (by_range) atomicAdd(&sh.hist[0][max(0, min((int)((v[e] - mn) * inv), kBins - 1))], 1);
      }
    }
  }
  if (by_value) {
    find_bin(K);
    const float w = range / (float)kBins, slack = 0.01f * w + fmaxf(fabsf(mn), fabsf(mx)) * 0x1p-21f;
    if (sh.bin > 0) lo = max(lo0, order_key(mn + (float)sh.bin * w - slack));
    if (sh.bin < kBins - 1) hi = min(hi0, order_key(mn + (float)(sh.bin + 1) * w + slack));
  } else {
    __syncthreads();
  }
  int k = K, in_range = vis;
  int m = 0, above = 0, before_me = 0;
  uint32_t list_hi = 0;
  // One round by value, four by bits and the last list: whatever the scores' memory
  // holds (a score kernel that gave up), the rounds end, and alike in all CTAs.
  constexpr int kRounds = 16;
  int rounds = 0;
  for (int limit = by_value ? vis : kNarrow;;) {
    if (in_range > limit && lo < hi && ++rounds < kRounds) {
      const int shift = max(0, 32 - __clz(hi - lo) - kBinBits);   // (hi - lo) >> shift < 1024
      int* hist = sh.hist[buf];
#pragma unroll 4
      for (int j = tid; j < n; j += kSel) {
        const uint32_t x = key(j);
        if (x >= lo && x <= hi) atomicAdd(&hist[(x - lo) >> shift], 1);
      }
      find_bin(k);
      k -= sh.above;
      in_range = sh.in_bin;
      lo += (uint32_t)sh.bin << shift;
      hi = min(hi, lo + ((1u << shift) - 1u));
      continue;
    }
    // ---- the keys of the bin and of 2 eps around it, in every CTA ---------------
    const uint32_t list_lo = min(lo, order_key(order_value(lo) - eps2));
    list_hi = max(hi, order_key(order_value(hi) + eps2));
    if (tid == 0) sh.n[0] = 0;
    __syncthreads();
    int c = 0;
#pragma unroll 4
    for (int jw = warp * 32; jw < n; jw += kSel) {
      const int j = jw + lane;
      const uint32_t x = j < n ? key(j) : 0u;
      const unsigned word = __ballot_sync(0xffffffffu, j < n && x > list_hi);
      if (lane == 0) {
        bits[jw / 32] = word;
        c += __popc(word);
      }
      if (j < n && x >= list_lo && x <= list_hi) {
        const int at = atomicAdd(&sh.n[0], 1);
        if (at < kList) {
          sh.list_key[at] = x;
          sh.list_j[at] = j0 + j;
        }
      }
    }
    c = block_count(sh, c);
    if (tid == 0) sh.n[1] = c;
    cluster_sync<CS>();
    // every CTA's counts, and with them the first entries of its list: more than
    // kAhead of them are read in a second step
    int2 pn[CS];
    constexpr int kAhead = kSel / CS < kList ? kSel / CS : kList;
    const int ar = min(tid / kAhead, CS - 1), ai = tid - ar * kAhead;
    const uint32_t akey = ai < kAhead ? peer<CS>(sh.list_key, ar)[ai] : 0u;
    const int aj = ai < kAhead ? peer<CS>(sh.list_j, ar)[ai] : 0;
#pragma unroll
    for (int r = 0; r < CS; ++r) pn[r] = *reinterpret_cast<const int2*>(peer<CS>(sh.n, r));
    m = above = before_me = 0;
    int at = 0, from = -1, place = -1;                   // entry tid: of CTA `from`, its entry `at`
    bool more = false;
#pragma unroll
    for (int r = 0; r < CS; ++r) {
      if (tid >= m && tid < m + pn[r].x) {
        from = r;
        at = tid - m;
      }
      if (r == ar && ai < min(pn[r].x, kAhead)) place = m + ai;
      more |= pn[r].x > kAhead;
      m += pn[r].x;
      above += pn[r].y;
      if (r < rank) before_me += pn[r].y;
    }
    if (m <= kList) {
      if (tid < kList && tid >= m) sh.all_key[tid] = 0u;
      if (place >= 0) {
        sh.all_key[place] = akey;
        sh.all_j[place] = aj;
      }
      if (more && from >= 0 && at >= kAhead) {
        sh.all_key[tid] = peer<CS>(sh.list_key, max(from, 0))[at];
        sh.all_j[tid] = peer<CS>(sh.list_j, max(from, 0))[at];
      }
      __syncthreads();
      break;
    }
    if (lo >= hi || ++rounds >= kRounds) break;          // a row of ties
    // too many: narrow by keys, from the whole range, and at last to one key
    limit = by_value ? kNarrow : 0;
    if (by_value) {
      lo = lo0;
      hi = hi0;
    }
    by_value = false;
    cluster_sync<CS>();                                  // sh.n is read
  }

  if (m <= kList) {
    // ---- T by rank, then the close blocks ----------------------------------------
    const uint32_t x = sh.all_key[tid & (kList - 1)];
    const int j = sh.all_j[tid & (kList - 1)];             // of the threads below m
    int gt = 0, eq = 0, page = 0;
    if (tid < m) {
      page = __ldg(pages + page_index(a.cs, j));           // in flight during the ranking
      count_keys(sh, m, x, &gt, &eq);
      if (above + gt < K && above + gt + eq >= K) sh.tkey = x;
    }
    __syncthreads();
    const uint32_t tkey = sh.tkey;
    const float tval = order_value(tkey);
    const uint32_t clo = min(tkey, order_key(tval - eps2)), chi = max(tkey, order_key(tval + eps2));
    const bool sure = tid < m && x > chi, close = tid < m && x >= clo && x <= chi;
    if (close && (unsigned)page < (unsigned)a.cs.n_pages) {
      // the key's bytes, on their way while the close blocks are counted
      const int r = j - page_index(a.cs, j) * a.cs.page_size;
      const uint8_t* base = a.cache + page_base(a.cs, page);
      asm volatile("prefetch.global.L1 [%0];" ::"l"(base + row_code(a.cs, r)));
      asm volatile("prefetch.global.L1 [%0];" ::"l"(base + row_scale(a.cs, r)));
    }
    const unsigned sm = __ballot_sync(0xffffffffu, sure), cm = __ballot_sync(0xffffffffu, close);
    if (lane == 0) {
      sh.warp_n[warp] = __popc(sm);
      sh.warp_m[warp] = __popc(cm);
    }
    __syncthreads();
    const int need = K - above - __reduce_add_sync(0xffffffffu, sh.warp_n[lane]);
    const int mc = __reduce_add_sync(0xffffffffu, sh.warp_m[lane]);
    const int place = __reduce_add_sync(0xffffffffu, lane < warp ? sh.warp_m[lane] : 0) +
                      __popc(cm & ((1u << lane) - 1u));
    if (close) {
      sh.close_j[place] = j;
      sh.close_page[place] = page;
    }
    __syncthreads();
    bool in = sure;
    if (need < mc && eps2 > 0.f) {
      // Every CTA scores all close blocks itself where one round of its warps
      // does, otherwise over its share of the heads.
      const bool whole = CS == 1 || mc * ((a.H + 7) / 8) <= kSelWarps;
      const int share = whole ? a.H : (a.H + CS - 1) / CS, h0 = whole ? 0 : min(rank * share, a.H);
      score_exact<T, BITS>(sh, a, row, k_s, mc, h0, min(share, a.H - h0), ae, ke,
                           [&](int e) { return sh.close_j[e]; },
                           [&](int e) { return sh.close_page[e]; },
                           [&](int e, float2 v) { sh.exact[e] = v; });
      if (whole) {
        __syncthreads();
        if (tid < mc) sh.all_exact[tid] = pair_key(sh.exact[tid]);
      } else {
        cluster_sync<CS>();
        if (tid < mc) {
          float2 v[CS];
#pragma unroll
          for (int r = 0; r < CS; ++r) v[r] = peer<CS>(sh.exact, r)[tid];
#pragma unroll
          for (int r = 1; r < CS; ++r) v[0] = pair_add(v[0], v[r]);
          sh.all_exact[tid] = pair_key(v[0]);
        }
      }
    } else {
      // all of them, or blocks whose scores are exactly equal
      if (tid < mc) sh.all_exact[tid] = 0;
    }
    __syncthreads();
    if (close) {
      const unsigned long long v = sh.all_exact[place];
      int better = 0;
      for (int e = 0; e < mc; ++e) {
        const unsigned long long y = sh.all_exact[e];
        better += y > v || (y == v && sh.close_j[e] < j);
      }
      in = better < need;
    }
    // this CTA's place: behind the chosen blocks of the parts before it
    before_me += block_count(sh, in && j < j0 ? 1 : 0);
    if (in && j >= j0 && j < j0 + n) atomicOr(&bits[(j - j0) / 32], 1u << (j & 31));
    __syncthreads();
    // the chosen blocks in ascending order, a word of the bitmap a thread
    for (int w0 = 0; w0 * 32 < n; w0 += kSel) {
      const int wi = w0 + tid;
      uint32_t mask = wi * 32 < n ? bits[wi] : 0u;
      const int c = __popc(mask);
      int at = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, at, o);
        if (lane >= o) at += v;
      }
      if (lane == 31) sh.warp_n[warp] = at;
      __syncthreads();
      at += before_me - c + __reduce_add_sync(0xffffffffu, lane < warp ? sh.warp_n[lane] : 0);
      for (; mask != 0; mask &= mask - 1, ++at)
        if (at < K) out[at] = j0 + wi * 32 + __ffs(mask) - 1;
      before_me += __reduce_add_sync(0xffffffffu, sh.warp_n[lane]);
      __syncthreads();
    }
    cluster_sync<CS>();                                  // no CTA leaves while another reads it
    return;
  }
  cluster_sync<CS>();
  if (rank != 0) return;

  // ---- a row of ties (T = lo = hi): one CTA, lists in global memory --------------
  const int need = K - above;
  const uint32_t list_lo = min(lo, order_key(order_value(lo) - eps2));
  int32_t* list = a.list + row * a.slots;
  compact(sh, vis,
          [&](int j) {
            const uint32_t x = order_key(score[j]);
            return x >= list_lo && x <= list_hi;
          },
          [&](int j, int at) { list[at] = j; });
  if (need < m && eps2 > 0.f) {
    double* ex = a.exact + row * a.slots;
    score_exact<T, BITS>(sh, a, row, k_s, m, 0, a.H, ae, ke, [&](int e) { return list[e]; },
                         [&](int e) { return pages[page_index(a.cs, list[e])]; },
                         [&](int e, float2 v) { ex[e] = (double)v.x + (double)v.y; });
    int eq = 0;
    const unsigned long long bar =
        radix_select(sh, m, need, [&](int e) { return order_key(ex[e]); }, &eq);
    compact(sh, m, [&](int e) { return order_key(ex[e]) == bar; },
            [&](int e, int at) { score[list[e]] = at < eq ? INFINITY : -INFINITY; });
    for (int e = tid; e < m; e += kSel) {
      const unsigned long long x = order_key(ex[e]);
      if (x != bar) score[list[e]] = x > bar ? INFINITY : -INFINITY;
    }
  } else {
    for (int e = tid; e < m; e += kSel) score[list[e]] = e < need ? INFINITY : -INFINITY;
  }
  __syncthreads();
  const uint32_t top = min(list_hi, order_key(INFINITY) - 1);
  compact(sh, vis, [&](int j) { return order_key(score[j]) > top; },
          [&](int j, int at) { if (at < K) out[at] = j; });
}

template <typename T, int BITS, int CS>
cudaError_t launch_select_cs(const IndexDecodeArgs& a, cudaStream_t st) {
  int cap = ((a.slots + CS - 1) / CS + 127) / 128 * 128;
  cap = cap < kMaxStaged ? cap : kMaxStaged;
  const size_t smem = (size_t)cap * 4 + cap / 8 + (size_t)kSelWarps * (a.d + 16) * sizeof(float);
  auto k = index_select_kernel<T, BITS, CS>;
  static SmemOnce once;
  const cudaError_t e = once(k, (size_t)kMaxStaged * 4 + kMaxStaged / 8 + kSelWarps * (kMaxDecodeDI + 16) * sizeof(float));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.b * a.s_q * CS));
  cfg.blockDim = dim3(kSel);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)CS;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CS > 1 ? 2 : 1;
  count_launches(1);
  return cudaLaunchKernelEx(&cfg, k, a, cap);
}

// CTAs of a row, up to eight: one for every 32768 slots, and where SMs are left
// one for every 8192 (a cluster barrier costs about as much as passing over
// 8192 scores).
template <typename T, int BITS>
cudaError_t launch_select(const IndexDecodeArgs& a, cudaStream_t st) {
  int cs = 1;
  const long long rows = (long long)a.b * a.s_q;
  while (cs < kMaxCluster &&
         (a.slots > cs * kMaxStaged || (a.slots > cs * 8192 && rows * cs * 2 <= 152)))
    cs *= 2;
  switch (cs) {
    case 1: return launch_select_cs<T, BITS, 1>(a, st);
    case 2: return launch_select_cs<T, BITS, 2>(a, st);
    case 4: return launch_select_cs<T, BITS, 4>(a, st);
    default: return launch_select_cs<T, BITS, 8>(a, st);
  }
}

}  // namespace

// Launched as a programmatic dependent of the score kernel: its CTAs compute
// the rows' error scale, and write the rows that take every block, beside it.
cudaError_t launch_index_select(const IndexDecodeArgs& a, bool bf16, int bits, cudaStream_t st) {
  if (bf16)
    return bits == 4 ? launch_select<__nv_bfloat16, 4>(a, st) : launch_select<__nv_bfloat16, 8>(a, st);
  return bits == 4 ? launch_select<float, 4>(a, st) : launch_select<float, 8>(a, st);
}

}  // namespace csa
