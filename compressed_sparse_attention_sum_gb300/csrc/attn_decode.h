// Arguments and split of csa_attn_decode, shared by its kernels and the entry
// point (internal to the library).
#pragma once

#include <cfloat>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cache_format.cuh"

namespace csa {

constexpr int kDecodeTile = 64;      // slots of one tile of the split (CUDA cores)
constexpr int kDecodeSms = 152;      // SMs of a GB300

struct AttnDecodeArgs {
  const void* q;
  const uint8_t* cache;
  const int32_t* raw_table;
  const int32_t* cmp_table;
  const int32_t* idx;
  const float* sink;
  const int32_t* seq_lens;
  float scale;
  void* o;
  float* lse;
  float* part_o;       // [b * s_q][parts][H][d], not normalized (parts > 1)
  float2* part_ml;     // [b * s_q][parts][H]: running maximum (log2 units), sum
  int b, s_q, H, d, ratio, window, K, P_raw, P_cmp;
  int parts;           // partial results of a query
  CacheShape cs;
  int* status;
};

// A sink in log2 units, always finite (a sink of -inf has no weight all the same).
// Where the rows' part of the denominator is 0 next to it, LSE is the sink as given.
__device__ __forceinline__ float sink_log2(float sink) {
  return fminf(fmaxf(sink * kLog2e, -FLT_MAX), FLT_MAX);
}

// Slots of one query are numbered: the window's `window` positions, then the
// K index entries (or the visible blocks).  Every slot is looked up on its
// own, so a split is a range of slots and needs no compaction; masked slots
// (before position 0, -1 entries) have weight zero.
struct DecodeRow {
  int t;        // position of the query; < 0: nothing to attend to
  int vis;      // visible compressed rows
  int slots;    // slots of this query
  int w0;       // position of slot 0 (may be negative)
};

__device__ __forceinline__ DecodeRow decode_row(const AttnDecodeArgs& a, int bi, int i) {
  DecodeRow r;
  int n = a.seq_lens[bi];
  if (n < 0) {
    set_status(a.status, kDevCheck, kSiteCacheRange);
    n = 0;
  }
  r.t = n - a.s_q + i;
  r.vis = r.t >= 0 ? (int)((unsigned)(r.t + 1) / (unsigned)a.ratio) : 0;
  const long long cap = (long long)a.P_cmp * a.cs.page_size;
  if (r.vis > cap) {
    if (a.P_cmp > 0) set_status(a.status, kDevCheck, kSiteCacheRange);
    r.vis = (int)cap;
  }
  r.w0 = r.t - a.window + 1;
  r.slots = r.t < 0 ? 0 : a.window + (a.idx != nullptr ? a.K : r.vis);
  return r;
}

// Byte offsets of slot s of the query (0 <= s < r.slots); false when masked.
__device__ __forceinline__ bool decode_slot(const AttnDecodeArgs& a, const DecodeRow& r, int bi,
                                            long long row, int s, long long* code,
                                            long long* scale) {
  if (s < a.window) {
    const int pos = r.w0 + s;
    if (pos < 0) return false;
    const int slot = (int)((unsigned)pos % (unsigned)(a.P_raw * a.cs.page_size));
    return cache_row(a.cs, a.raw_table + (long long)bi * a.P_raw, slot, code, scale, a.status);
  }
  const int k = s - a.window;
  const int j = a.idx != nullptr ? a.idx[row * a.K + k] : k;
  if (j < 0 || j >= r.vis) return false;
  return cache_row(a.cs, a.cmp_table + (long long)bi * a.P_cmp, j, code, scale, a.status);
}

// How a call is cut into CTAs: queries of one sequence that share a CTA (and
// their groups), head groups, CTAs of a cluster that join a part of the slots
// among themselves, and parts, which a second kernel joins.
struct DecodePlan {
  int cols, per_group, groups, head_groups, cluster, parts;
};

inline DecodePlan decode_plan_simt(int b, int s_q, int H, int window, long long cmp_rows) {
  DecodePlan p{8, 1, s_q, (H + 7) / 8, 1, 1};
  // enough CTAs to fill the GPU twice over, at most one per tile
  const long long tiles = (window + cmp_rows + kDecodeTile - 1) / kDecodeTile;
  long long n = 2ll * kDecodeSms / ((long long)b * s_q * p.head_groups);
  n = n > tiles ? tiles : n;
  p.parts = n < 1 ? 1 : (int)n;
  return p;
}

inline bool decode_tc_width(int d) { return d == 64 || d == 128 || d == 256 || d == 512; }

// CTAs of the tensor-core kernel that the GPU holds at once, one on an SM, in
// clusters of a size (a cluster stays within a GPC: what
// cudaOccupancyMaxActiveClusters answers on a GB300).  Two on an SM, with 80
// registers a thread, were slower: 64 queries of 32 x 128 in 14.7 us, not 12.1.
inline long long decode_tc_capacity(int cluster) {
  return cluster <= 2 ? 152 : cluster == 4 ? 144 : 120;
}

// Without an index list the queries of a sequence see the same rows (all but
// the newest), so as many of them as fit 64 columns share a CTA.  The tiles of
// 128 slots go to a cluster of up to eight CTAs, as long as the GPU holds all
// of them at once (a second wave doubles the time), and where it holds twelve
// a query or more to several clusters of four, joined by a second kernel.
inline DecodePlan decode_plan_tc(int b, int s_q, int H, int window, int K, bool dense,
                                 long long cmp_cap) {
  DecodePlan p{};
  p.per_group = dense && H % 16 == 0 && H <= 32 ? 64 / H : 1;
  if (p.per_group > s_q) p.per_group = s_q;
  p.groups = (s_q + p.per_group - 1) / p.per_group;
  p.cols = p.per_group * H <= 32 ? 32 : 64;
  p.head_groups = p.per_group > 1 ? 1 : (H + p.cols - 1) / p.cols;
  const long long slots = window + p.per_group - 1 + (dense ? cmp_cap : K);
  const long long tiles = (slots + 127) / 128;
  const long long ctas = (long long)b * p.groups * p.head_groups;
  const long long most = decode_tc_capacity(4) / ctas;   // CTAs of a query in clusters of four
  p.cluster = 1;
  p.parts = 1;
  if (tiles > 8 && most >= 12) {
    const long long n = most < tiles ? most : tiles;
    p.cluster = 4;
    p.parts = (int)((n + (most < tiles ? 0 : 3)) / 4);
  } else {
    while (p.cluster < 8 && p.cluster < tiles &&
           ctas * p.cluster * 2 <= decode_tc_capacity(p.cluster * 2))
      p.cluster *= 2;
  }
  return p;
}

// Combines the parts of every (row, head): o and lse.
cudaError_t launch_attn_decode_combine(const AttnDecodeArgs& a, bool bf16, cudaStream_t st);
cudaError_t launch_attn_decode_simt(const AttnDecodeArgs& a, bool bf16, int bits,
                                    cudaStream_t st);
cudaError_t launch_attn_decode_512(const AttnDecodeArgs& a, const DecodePlan& p, int bits,
                                   cudaStream_t st);
cudaError_t launch_attn_decode_tc(const AttnDecodeArgs& a, const DecodePlan& p, int bits,
                                  cudaStream_t st);

}  // namespace csa
