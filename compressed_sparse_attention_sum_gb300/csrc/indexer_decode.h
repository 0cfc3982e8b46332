// Arguments and workspace layout of csa_indexer_topk_decode (internal).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "cache_format.cuh"

namespace csa {

constexpr int kIdxTile = 128;       // keys of one score tile
constexpr int kMaxDecodeHI = 128;   // indexer heads
constexpr int kMaxDecodeDI = 256;   // indexer head dim

struct IndexDecodeArgs {
  const void* q;
  const uint8_t* cache;
  const int32_t* table;
  const float* w;
  const int32_t* seq_lens;
  int32_t* out;
  // workspace, one row of `slots` entries per query
  float* scores;       // [b * s_q][slots]
  double* exact;       // [b * s_q][slots]: exact scores of the row's close candidates
  int32_t* list;       // [b * s_q][slots]: their blocks, ascending
  float4* tile_info;   // [b * s_q][tiles]: bound on |k_j| of a tile's keys, its smallest and largest score
  float err;           // bound of a score's error over sum_h |w_h| |q_h| times |k_j|
  int b, s_q, H, d, ratio, topk, P, slots, tiles;
  CacheShape cs;
  int* status;
};

// Visible blocks of query i of sequence bi.
__device__ __forceinline__ int index_vis(const IndexDecodeArgs& a, int bi, int i) {
  const int n = a.seq_lens[bi];
  if (n < 0) set_status(a.status, kDevCheck, kSiteCacheRange);
  const int t = n - a.s_q + i;
  if (n < 0 || t < 0) return 0;
  int vis = (int)((unsigned)(t + 1) / (unsigned)a.ratio);
  if (vis > a.slots) {
    set_status(a.status, kDevCheck, kSiteCacheRange);
    vis = a.slots;
  }
  return vis;
}

// Workspace bytes and the pointers into it (ws may be null to size it).
inline size_t index_decode_layout(IndexDecodeArgs* a, unsigned char* ws) {
  const size_t rows = (size_t)a->b * a->s_q, n = rows * (size_t)a->slots;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    unsigned char* p = ws + at;
    at += (bytes + 15) / 16 * 16;
    return p;
  };
  a->exact = (double*)take(n * sizeof(double));
  a->scores = (float*)take(n * sizeof(float));
  a->list = (int32_t*)take(n * sizeof(int32_t));
  a->tile_info = (float4*)take(rows * (size_t)a->tiles * sizeof(float4));
  return at;
}

cudaError_t launch_index_scores_simt(const IndexDecodeArgs& a, bool bf16, int bits,
                                     cudaStream_t st);
bool index_decode_tc_supported(int H, int d);
cudaError_t launch_index_scores_tc(const IndexDecodeArgs& a, int bits, cudaStream_t st);
cudaError_t launch_index_select(const IndexDecodeArgs& a, bool bf16, int bits, cudaStream_t st);

}  // namespace csa
