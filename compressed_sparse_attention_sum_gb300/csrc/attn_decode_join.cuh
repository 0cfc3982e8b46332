// What the tensor-core kernels of csa_attn_decode share: the reduction of a
// column over a warp's lanes, and the end of a CTA: its part joined with those of
// the cluster, or written as the whole query.
#pragma once

#include <cooperative_groups.h>

#include "attn_decode.h"
#include "cache_expand.cuh"
#include "tcgen05.cuh"

namespace csa {
namespace adt {

using namespace csa::umma;
namespace cg = cooperative_groups;

constexpr int kSiteDecode = 0x73;
constexpr float kRescale = 8.f;               // a column's maximum may lag by 2^8

// Frees the TMEM of a CTA, by the warp that allocated it and issued the products.
// After a wait that gave up, products may still run: they are waited for first,
// again with a limit.
__device__ __forceinline__ void free_tmem(uint32_t tmem, uint32_t columns, bool dead, uint64_t* bar_end) {
  if (dead) {
    if (elect_one()) mma_commit(bar_end);
    __syncwarp();
    mbar_wait(bar_end, 0);
    __syncwarp();
  }
  fence_after();
  tmem_dealloc(tmem, columns);
}

// Transposing butterfly: v[c] holds this lane's value of column c; afterwards
// lanes l and l + 16 hold op over all 32 lanes of column l % 16.
template <bool kMax>
__device__ __forceinline__ float lane_reduce16(float (&v)[16]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int off = 8, n = 8; off >= 1; off >>= 1, n >>= 1) {
    const bool up = (lane & off) != 0;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float send = up ? v[i] : v[i + n];
      const float keep = up ? v[i + n] : v[i];
      const float recv = __shfl_xor_sync(0xffffffffu, send, off);
      v[i] = kMax ? fmaxf(keep, recv) : keep + recv;
    }
  }
  const float other = __shfl_xor_sync(0xffffffffu, v[0], 16);
  return kMax ? fmaxf(v[0], other) : v[0] + other;
}

// Joins the (m, l, O) of the CS CTAs of a cluster for this CTA's share of the
// columns, from their shared memory, four channels a thread: all of its reads
// are in flight at once.  final: also the sink, o and lse; otherwise the
// cluster's entry of the partial results.
template <typename C, int D, int NC, int CS>
__device__ __forceinline__ void join_cluster(const AttnDecodeArgs& a, unsigned char* sm, int rank,
                                             int part, int per_group, int nq, int heads, int h0,
                                             long long row0) {
  constexpr int kCols = NC / CS;                           // columns of this CTA
  const bool final = a.parts == 1;
  const float* sink = reinterpret_cast<const float*>(sm + C::SINK);
  const unsigned char* base[CS];
#pragma unroll
  for (int r = 0; r < CS; ++r) base[r] = cg::this_cluster().map_shared_rank(sm, r);
  for (int e = threadIdx.x; e < kCols * (D / 4); e += C::kThreads) {
    const int col = rank * kCols + e / (D / 4), c = e % (D / 4) * 4;
    float4 ml[CS];                                         // maximum, sum, O's factor
    float4 v[CS];
#pragma unroll
    for (int r = 0; r < CS; ++r) {
      ml[r] = *reinterpret_cast<const float4*>(base[r] + C::ML + col * 16);
      v[r] = *reinterpret_cast<const float4*>(base[r] + C::STAGE + (col * D + c) * 4);
    }
    const int qi = per_group > 1 ? col / a.H : 0, h = per_group > 1 ? col - qi * a.H : col;
    if (qi >= nq || h >= heads) continue;
    const float sink2 = final ? sink[h] : -INFINITY;
    float m = sink2, total = 0.f;
#pragma unroll
    for (int r = 0; r < CS; ++r) m = fmaxf(m, ml[r].x);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int r = 0; r < CS; ++r) {
      if (ml[r].y > 0.f) {                                 // a CTA without a tile has no O
        const float f = ex2(ml[r].x - m), fo = f * ml[r].z;
        total = fmaf(ml[r].y, f, total);
        acc.x = fmaf(v[r].x, fo, acc.x);
        acc.y = fmaf(v[r].y, fo, acc.y);
        acc.z = fmaf(v[r].z, fo, acc.z);
        acc.w = fmaf(v[r].w, fo, acc.w);
      }
    }
    const long long row = row0 + qi;
    if (!final) {
      const long long at = (row * a.parts + part) * a.H + h0 + h;
      *reinterpret_cast<float4*>(a.part_o + at * D + c) = acc;
      if (c == 0) a.part_ml[at] = make_float2(m, total);
      continue;
    }
    const bool rows = total > 0.f;
    if (sink2 > -INFINITY) total += ex2(sink2 - m);
    const float inv = total > 0.f ? __fdividef(1.f, total) : 0.f;
    *reinterpret_cast<uint2*>((__nv_bfloat16*)a.o + (row * a.H + h0 + h) * D + c) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (c == 0)
      a.lse[row * a.H + h0 + h] = rows ? (m + log2f(total)) * kLn2
                                       : sink2 > -INFINITY ? a.sink[h0 + h] : -INFINITY;
  }
}

// Sixteen columns (c0 ..) of O^T at channel position p = 32 x + lane, times the
// columns' factors, to o [columns][D].  Neighbouring channels lie two positions
// apart: such a pair of lanes exchanges halves, and each stores both channels of
// eight columns.
template <int D, int BITS>
__device__ __forceinline__ void store_o16(const uint32_t (&v)[16], const float* factor, int c0,
                                          int cols, __nv_bfloat16* o, int p) {
  const bool high = (p & 2) != 0;
  o += (long long)(c0 + (high ? 8 : 0)) * D + channel_of<BITS>(p & ~2);
  cols -= c0 + (high ? 8 : 0);
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const uint32_t own = pack_bf16x2(__uint_as_float(v[c]) * factor[c0 + c],
                                     __uint_as_float(v[c + 8]) * factor[c0 + c + 8]);
    const uint32_t other = __shfl_xor_sync(0xffffffffu, own, 2);
    const uint32_t out = high ? __byte_perm(other, own, 0x7632) : __byte_perm(own, other, 0x5410);
    if (c < cols) *reinterpret_cast<uint32_t*>(o + (long long)c * D) = out;
  }
}

// The end of a CTA with n tiles that shares its queries with others (cs > 1:
// C::STAGE holds its O as [column][channel], C::ML its columns' (maximum, sum, factor)) or
// had nothing to attend to.  Called by all threads.
template <typename C, int D, int NC>
__device__ __forceinline__ void finish_decode(const AttnDecodeArgs& a, unsigned char* sm, bool dead,
                                              int n, int cs, int rank, int split, int per_group,
                                              int nq, int heads, int h0, long long row0) {
  const int tid = threadIdx.x;
  if (dead) {
    if (tid == 0) set_status(a.status, kDevTimeout, kSiteDecode);
  } else if (cs == 1) {
    if (n > 0) return;                                     // o and lse are written
    uint4* dst = reinterpret_cast<uint4*>((__nv_bfloat16*)a.o + (row0 * a.H + h0) * D);
    const int chunks = nq * heads * (D / 8);
    for (int e = tid; e < chunks; e += C::kThreads) dst[e] = make_uint4(0u, 0u, 0u, 0u);
    if (tid < nq * heads) {
      const int qi = tid / heads, h = tid - qi * heads;
      a.lse[(row0 + qi) * a.H + h0 + h] = a.sink != nullptr ? a.sink[h0 + h] : -INFINITY;
    }
  } else {
    const int part = split / cs;
    switch (cs) {
      case 2: join_cluster<C, D, NC, 2>(a, sm, rank, part, per_group, nq, heads, h0, row0); break;
      case 4: join_cluster<C, D, NC, 4>(a, sm, rank, part, per_group, nq, heads, h0, row0); break;
      default: join_cluster<C, D, NC, 8>(a, sm, rank, part, per_group, nq, heads, h0, row0); break;
    }
  }
}

}  // namespace adt
}  // namespace csa
