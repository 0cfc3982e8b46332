// csa_cache_write and csa_cache_read: rows into and out of the paged cache.
//
// Both move each row once: d elements of bf16 / fp32 on one side, d * bits / 8
// code bytes and d / 32 scale bytes on the other, so HBM bounds them (launch
// latency when a decode step appends a few rows).  A thread owns eight
// channels (16 or 32 bytes of the row, 4 or 8 bytes of codes), so four lanes
// share a group's maximum through two shuffles and a warp's accesses are
// contiguous.
#include "cache_format.cuh"

namespace csa {
namespace {

constexpr int kThreads = 256;

// Row `i` of sequence `bi`: its slot in the ring, or -1 when it is not moved
// (past the count; a later row of the same call takes the slot).
__device__ __forceinline__ int ring_slot(const int32_t* pos0, const int32_t* counts, int bi, int i,
                                         int s, int ring, bool write, int* status) {
  int n = s;
  if (counts != nullptr) {
    n = counts[bi];
    if (n < 0 || n > s) {
      if (i == 0) set_status(status, kDevCheck, kSiteCacheRange);
      n = max(0, min(n, s));
    }
  }
  if (i >= n) return -1;
  const int p0 = pos0[bi];
  if (p0 < 0 || (long long)p0 + n > 0x7fffffffll) {
    if (i == 0) set_status(status, kDevCheck, kSiteCacheRange);
    return -1;
  }
  if (write && i < n - ring) return -1;
  return (int)(((unsigned)p0 + (unsigned)i) % (unsigned)ring);
}

template <typename T, int BITS>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(
    const T* __restrict__ x, long long x_bs, long long x_rs, const int32_t* __restrict__ table,
    const int32_t* __restrict__ pos0, const int32_t* __restrict__ counts,
    uint8_t* __restrict__ cache, int s, int d, int P, CacheShape cs, long long items,
    int* status) {
  const int per_row = d / 8;
  const long long item = (long long)blockIdx.x * kThreads + threadIdx.x;
  // items is a multiple of 4 (d % 32 == 0): the four lanes of a group are all in or all out
  if (item >= items) return;
  const long long rowi = item / per_row;
  const int c0 = (int)(item - rowi * per_row) * 8;
  const int bi = (int)(rowi / s), i = (int)(rowi - (long long)bi * s);
  const int slot = ring_slot(pos0, counts, bi, i, s, P * cs.page_size, true, status);
  long long code = 0, scale = 0;
  const bool live = slot >= 0 &&
                    cache_row(cs, table + (long long)bi * P, slot, &code, &scale, status);
  float v[8];
  if (live) {
    load8(x + bi * x_bs + i * x_rs + c0, v);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = 0.f;
  }
  float m = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) m = fmaxf(m, fabsf(v[k]));
  const unsigned mask = __activemask();
  m = fmaxf(m, __shfl_xor_sync(mask, m, 1));
  m = fmaxf(m, __shfl_xor_sync(mask, m, 2));
  if (!live) return;
  const int e = scale_exponent<BITS>(m);
  const float inv = pow2f(-e);
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] *= inv;
  if constexpr (BITS == 4) {
    *reinterpret_cast<uint32_t*>(cache + code + c0 / 2) = encode8_e2m1(v);
  } else {
    *reinterpret_cast<uint2*>(cache + code + c0) =
        make_uint2(encode4_e4m3(v[0], v[1], v[2], v[3]), encode4_e4m3(v[4], v[5], v[6], v[7]));
  }
  if ((c0 & 31) == 0) cache[scale + c0 / kCacheGroup] = (uint8_t)(e + 127);
}

template <typename T, int BITS>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(
    const uint8_t* __restrict__ cache, const int32_t* __restrict__ table,
    const int32_t* __restrict__ pos0, const int32_t* __restrict__ counts, T* __restrict__ out,
    long long o_bs, long long o_rs, int s, int d, int P, CacheShape cs, long long items,
    int* status) {
  const int per_row = d / 8;
  const long long item = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (item >= items) return;
  const long long rowi = item / per_row;
  const int c0 = (int)(item - rowi * per_row) * 8;
  const int bi = (int)(rowi / s), i = (int)(rowi - (long long)bi * s);
  const int slot = ring_slot(pos0, counts, bi, i, s, P * cs.page_size, false, status);
  if (slot < 0) return;
  long long code, scale;
  float v[8];
  if (cache_row(cs, table + (long long)bi * P, slot, &code, &scale, status)) {
    cache_load8<BITS>(cache + code, scale_value(cache[scale + c0 / kCacheGroup]), c0, v);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = 0.f;
  }
  store8(out + bi * o_bs + i * o_rs + c0, v);
}

}  // namespace

cudaError_t launch_cache_write(const void* x, long long x_bs, long long x_rs, bool bf16,
                               const int32_t* table, const int32_t* pos0, const int32_t* counts,
                               void* cache, int b, int s, int d, int P, int n_pages,
                               int page_size, int bits, int* status, cudaStream_t st) {
  const CacheShape cs = cache_shape(page_size, n_pages, d, bits);
  const long long items = (long long)b * s * (d / 8);
  const unsigned grid = (unsigned)((items + kThreads - 1) / kThreads);
  uint8_t* c = (uint8_t*)cache;
#define CSA_WRITE(T, B)                                                                          \
  cache_write_kernel<T, B><<<grid, kThreads, 0, st>>>((const T*)x, x_bs, x_rs, table, pos0,      \
                                                      counts, c, s, d, P, cs, items, status)
  if (bf16) {
    if (bits == 4) CSA_WRITE(__nv_bfloat16, 4); else CSA_WRITE(__nv_bfloat16, 8);
  } else {
    if (bits == 4) CSA_WRITE(float, 4); else CSA_WRITE(float, 8);
  }
#undef CSA_WRITE
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_cache_read(const void* cache, const int32_t* table, const int32_t* pos0,
                              const int32_t* counts, void* out, long long o_bs, long long o_rs,
                              bool bf16, int b, int s, int d, int P, int n_pages, int page_size,
                              int bits, int* status, cudaStream_t st) {
  const CacheShape cs = cache_shape(page_size, n_pages, d, bits);
  const long long items = (long long)b * s * (d / 8);
  const unsigned grid = (unsigned)((items + kThreads - 1) / kThreads);
  const uint8_t* c = (const uint8_t*)cache;
#define CSA_READ(T, B)                                                                           \
  cache_read_kernel<T, B><<<grid, kThreads, 0, st>>>(c, table, pos0, counts, (T*)out, o_bs,      \
                                                     o_rs, s, d, P, cs, items, status)
  if (bf16) {
    if (bits == 4) CSA_READ(__nv_bfloat16, 4); else CSA_READ(__nv_bfloat16, 8);
  } else {
    if (bits == 4) CSA_READ(float, 4); else CSA_READ(float, 8);
  }
#undef CSA_READ
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace csa
