// csa_cache_write and csa_cache_read: rows into and out of the paged cache.
//
// Both move each row once: d elements of bf16 / fp32 on one side, d * bits / 8
// code bytes and d / 32 scale bytes on the other, so HBM bounds them (launch
// latency when a decode step appends a few rows).  A thread owns eight
// channels (16 or 32 bytes of a row, 4 or 8 bytes of codes), so four lanes
// share a group's maximum through two shuffles and a warp's accesses are
// contiguous; of long ranges it takes several rows, whose page ids and then
// whose bytes are read all at once.
#include "cache_expand.cuh"
#include "cache_format.cuh"

namespace csa {
namespace {

constexpr int kThreads = 256;

// The rows [0, n) of a sequence that a call moves and its first position; n = 0
// where the position is outside its range.
__device__ __forceinline__ int range_of(const int32_t* pos0, const int32_t* counts, int bi, int s,
                                        int* p0, int* status) {
  int n = s;
  if (counts != nullptr) {
    n = counts[bi];
    if (n < 0 || n > s) {
      set_status(status, kDevCheck, kSiteCacheRange);
      n = max(0, min(n, s));
    }
  }
  *p0 = pos0[bi];
  if (n > 0 && (*p0 < 0 || (long long)*p0 + n > 0x7fffffffll)) {
    set_status(status, kDevCheck, kSiteCacheRange);
    n = 0;
  }
  return n;
}

// The slots of U rows i, i + step, ... : pages read together; -1 for a row that
// is not moved.
template <int U>
__device__ __forceinline__ void slots_of(const CacheShape& cs, const int32_t* pages, int i, int step,
                                         int first, int n, int p0, int ring, int* status,
                                         int (&slot)[U], int (&page)[U]) {
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int r = i + u * step;
    slot[u] = r >= first && r < n ? (int)(((unsigned)p0 + (unsigned)r) % (unsigned)ring) : -1;
    page[u] = __ldg(pages + (slot[u] < 0 ? 0 : page_index(cs, slot[u])));
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (slot[u] >= 0 && (unsigned)page[u] >= (unsigned)cs.n_pages) {
      set_status(status, kDevCheck, kSiteCachePage);
      page[u] = -1;
    }
  }
}

// blockIdx.y: sequence; a block takes kThreads / (d / 8) rows at a time, U
// times.  Threads past the last whole row idle (d / 8 is a multiple of 4, so
// the lanes of a group stay together).
template <typename T, int BITS, int U>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(
    const T* __restrict__ x, long long x_bs, long long x_rs, const int32_t* __restrict__ table,
    const int32_t* __restrict__ pos0, const int32_t* __restrict__ counts,
    uint8_t* __restrict__ cache, int s, int d, int P, CacheShape cs, int* status) {
  const int tpr = d / 8, rpb = kThreads / tpr;
  const int rr = (int)threadIdx.x / tpr, c0 = ((int)threadIdx.x - rr * tpr) * 8;
  const int bi = blockIdx.y, ring = P * cs.page_size;
  const int i = (int)blockIdx.x * rpb * U + rr;
  int p0;
  const int n = range_of(pos0, counts, bi, s, &p0, status);
  int slot[U], page[U];
  // of more rows than the ring holds the last are kept
  slots_of<U>(cs, table + (long long)bi * P, i, rpb, rr < rpb ? max(0, n - ring) : n, n, p0, ring,
              status, slot, page);
  float v[U][8];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (slot[u] >= 0) {
      load8(x + bi * x_bs + (long long)(i + u * rpb) * x_rs + c0, v[u]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[u][k] = 0.f;
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float m = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = fmaxf(m, fabsf(v[u][k]));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    if (slot[u] < 0 || page[u] < 0) continue;
    const int e = scale_exponent<BITS>(m);
    const float inv = pow2f(-e);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[u][k] *= inv;
    const int row = slot[u] - page_index(cs, slot[u]) * cs.page_size;
    uint8_t* base = cache + page_base(cs, page[u]);
    uint8_t* code = base + row_code(cs, row);
    if constexpr (BITS == 4) {
      *reinterpret_cast<uint32_t*>(code + c0 / 2) = encode8_e2m1(v[u]);
    } else {
      *reinterpret_cast<uint2*>(code + c0) =
          make_uint2(encode4_e4m3(v[u][0], v[u][1], v[u][2], v[u][3]),
                     encode4_e4m3(v[u][4], v[u][5], v[u][6], v[u][7]));
    }
    if ((c0 & 31) == 0) base[row_scale(cs, row) + c0 / kCacheGroup] = (uint8_t)(e + 127);
  }
}

// The same for long ranges of bf16 rows on 32-byte boundaries: 16 channels a
// thread, read at once (ld.global.v8), so that two lanes share a group.
template <int BITS, int U>
__global__ void __launch_bounds__(kThreads) cache_write16_kernel(
    const __nv_bfloat16* __restrict__ x, long long x_bs, long long x_rs,
    const int32_t* __restrict__ table, const int32_t* __restrict__ pos0,
    const int32_t* __restrict__ counts, uint8_t* __restrict__ cache, int s, int d, int P,
    CacheShape cs, int* status) {
  const int tpr = d / 16, rpb = kThreads / tpr;
  const int rr = (int)threadIdx.x / tpr, c0 = ((int)threadIdx.x - rr * tpr) * 16;
  const int bi = blockIdx.y, ring = P * cs.page_size;
  const int i = (int)blockIdx.x * rpb * U + rr;
  int p0;
  const int n = range_of(pos0, counts, bi, s, &p0, status);
  int slot[U], page[U];
  slots_of<U>(cs, table + (long long)bi * P, i, rpb, rr < rpb ? max(0, n - ring) : n, n, p0, ring,
              status, slot, page);
  uint32_t w[U][8];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const __nv_bfloat16* src = slot[u] >= 0 ? x + bi * x_bs + (long long)(i + u * rpb) * x_rs + c0
                                            : reinterpret_cast<const __nv_bfloat16*>(g_zero_row);
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(w[u][0]), "=r"(w[u][1]), "=r"(w[u][2]), "=r"(w[u][3]), "=r"(w[u][4]),
                   "=r"(w[u][5]), "=r"(w[u][6]), "=r"(w[u][7])
                 : "l"(src));
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float v[2][8], m = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      v[k / 4][k % 4 * 2] = __uint_as_float(w[u][k] << 16);
      v[k / 4][k % 4 * 2 + 1] = __uint_as_float(w[u][k] & 0xffff0000u);
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) m = fmaxf(m, fabsf(v[k / 8][k % 8]));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    if (slot[u] < 0 || page[u] < 0) continue;
    const int e = scale_exponent<BITS>(m);
    const float inv = pow2f(-e);
#pragma unroll
    for (int k = 0; k < 16; ++k) v[k / 8][k % 8] *= inv;
    const int row = slot[u] - page_index(cs, slot[u]) * cs.page_size;
    uint8_t* base = cache + page_base(cs, page[u]);
    uint8_t* code = base + row_code(cs, row) + c0 * BITS / 8;
    if constexpr (BITS == 4) {
      *reinterpret_cast<uint2*>(code) = make_uint2(encode8_e2m1(v[0]), encode8_e2m1(v[1]));
    } else {
      *reinterpret_cast<uint4*>(code) =
          make_uint4(encode4_e4m3(v[0][0], v[0][1], v[0][2], v[0][3]),
                     encode4_e4m3(v[0][4], v[0][5], v[0][6], v[0][7]),
                     encode4_e4m3(v[1][0], v[1][1], v[1][2], v[1][3]),
                     encode4_e4m3(v[1][4], v[1][5], v[1][6], v[1][7]));
    }
    if ((c0 & 31) == 0) base[row_scale(cs, row) + c0 / kCacheGroup] = (uint8_t)(e + 127);
  }
}

template <typename T, int BITS, int U>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(
    const uint8_t* __restrict__ cache, const int32_t* __restrict__ table,
    const int32_t* __restrict__ pos0, const int32_t* __restrict__ counts, T* __restrict__ out,
    long long o_bs, long long o_rs, int s, int d, int P, CacheShape cs, int* status) {
  const int tpr = d / 8, rpb = kThreads / tpr;
  const int rr = (int)threadIdx.x / tpr, c0 = ((int)threadIdx.x - rr * tpr) * 8;
  const int bi = blockIdx.y;
  const int i = (int)blockIdx.x * rpb * U + rr;
  int p0;
  const int n = range_of(pos0, counts, bi, s, &p0, status);
  int slot[U], page[U];
  slots_of<U>(cs, table + (long long)bi * P, i, rpb, rr < rpb ? 0 : n, n, p0, P * cs.page_size,
              status, slot, page);
  uint2 w[U];
  uint32_t sc[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const bool live = slot[u] >= 0 && page[u] >= 0;
    const int row = slot[u] - page_index(cs, slot[u]) * cs.page_size;
    const uint8_t* base = cache + page_base(cs, page[u]);
    const uint8_t* zero = reinterpret_cast<const uint8_t*>(g_zero_row);
    const uint8_t* code = live ? base + row_code(cs, row) + c0 * BITS / 8 : zero;
    w[u].y = 0;
    if constexpr (BITS == 4) w[u].x = __ldg(reinterpret_cast<const uint32_t*>(code));
    else w[u] = __ldg(reinterpret_cast<const uint2*>(code));
    sc[u] = __ldg(live ? base + row_scale(cs, row) + c0 / kCacheGroup : zero);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (slot[u] < 0) continue;
    T* dst = out + bi * o_bs + (long long)(i + u * rpb) * o_rs + c0;
    if constexpr (sizeof(T) == 2) {
      uint32_t o[4];
      expand8<BITS>(w[u].x, w[u].y, o);
      scale8<BITS>(sc[u], o);
      *reinterpret_cast<uint4*>(dst) = natural8<BITS>(o);
    } else {
      float v[8];
      const float f = scale_value(sc[u]);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if constexpr (BITS == 4) v[k] = code_e2m1(w[u].x >> (4 * k)) * f;
        else v[k] = code_e4m3((k < 4 ? w[u].x : w[u].y) >> (8 * (k & 3))) * f;
      }
      store8(dst, v);
    }
  }
}

// The same for long ranges of bf16 rows on 32-byte boundaries: 16 channels a
// thread, stored at once (st.global.v8: a warp writes 1 KB an instruction).
template <int BITS, int U>
__global__ void __launch_bounds__(kThreads) cache_read16_kernel(
    const uint8_t* __restrict__ cache, const int32_t* __restrict__ table,
    const int32_t* __restrict__ pos0, const int32_t* __restrict__ counts,
    __nv_bfloat16* __restrict__ out, long long o_bs, long long o_rs, int s, int d, int P,
    CacheShape cs, int* status) {
  const int tpr = d / 16, rpb = kThreads / tpr;
  const int rr = (int)threadIdx.x / tpr, c0 = ((int)threadIdx.x - rr * tpr) * 16;
  const int bi = blockIdx.y;
  const int i = (int)blockIdx.x * rpb * U + rr;
  int p0;
  const int n = range_of(pos0, counts, bi, s, &p0, status);
  int slot[U], page[U];
  slots_of<U>(cs, table + (long long)bi * P, i, rpb, rr < rpb ? 0 : n, n, p0, P * cs.page_size,
              status, slot, page);
  uint32_t w[U][BITS / 2];
  uint32_t sc[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const bool live = slot[u] >= 0 && page[u] >= 0;
    const int row = slot[u] - page_index(cs, slot[u]) * cs.page_size;
    const uint8_t* base = cache + page_base(cs, page[u]);
    const uint8_t* zero = reinterpret_cast<const uint8_t*>(g_zero_row);
    const uint8_t* code = live ? base + row_code(cs, row) + c0 * BITS / 8 : zero;
    if constexpr (BITS == 4) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(code));
      w[u][0] = v.x;
      w[u][1] = v.y;
    } else {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(code));
      w[u][0] = v.x;
      w[u][1] = v.y;
      w[u][2] = v.z;
      w[u][3] = v.w;
    }
    sc[u] = __ldg(live ? base + row_scale(cs, row) + c0 / kCacheGroup : zero);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (slot[u] < 0) continue;
    uint4 r[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t o[4];
      if constexpr (BITS == 4) expand8<4>(w[u][h], 0u, o);
      else expand8<8>(w[u][2 * h], w[u][2 * h + 1], o);
      scale8<BITS>(sc[u], o);
      r[h] = natural8<BITS>(o);
    }
    __nv_bfloat16* dst = out + bi * o_bs + (long long)(i + u * rpb) * o_rs + c0;
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(r[0].x),
                 "r"(r[0].y), "r"(r[0].z), "r"(r[0].w), "r"(r[1].x), "r"(r[1].y), "r"(r[1].z),
                 "r"(r[1].w)
                 : "memory");
  }
}

// Rows of a thread: several once the call fills the GPU with one each.
inline int rows_per_thread(int b, int s, int d) {
  const long long rpb = kThreads / (d / 8);
  return (long long)b * ((s + rpb - 1) / rpb) > 152ll * 16 ? 8 : 1;
}
inline dim3 rows_grid(int b, int s, int d, int U, int channels = 8) {
  const int rows = kThreads / (d / channels) * U;
  return dim3((unsigned)(((long long)s + rows - 1) / rows), (unsigned)b);
}
// Rows [b, s, d] of bf16 on 32-byte boundaries.
inline bool wide_rows(const void* p, long long bs, long long rs) {
  return ((uintptr_t)p & 31) == 0 && bs % 16 == 0 && rs % 16 == 0;
}
constexpr int kWide = 4;             // rows of a thread of the 16-channel kernels

}  // namespace

cudaError_t launch_cache_write(const void* x, long long x_bs, long long x_rs, bool bf16,
                               const int32_t* table, const int32_t* pos0, const int32_t* counts,
                               void* cache, int b, int s, int d, int P, int n_pages,
                               int page_size, int bits, int* status, cudaStream_t st) {
  const CacheShape cs = cache_shape(page_size, n_pages, d, bits);
  const int u = rows_per_thread(b, s, d) > 1 ? 4 : 1;    // eight rows of fp32 values would spill
  const dim3 grid = rows_grid(b, s, d, u);
  uint8_t* c = (uint8_t*)cache;
  if (bf16 && u > 1 && wide_rows(x, x_bs, x_rs)) {
    const dim3 g = rows_grid(b, s, d, kWide, 16);
    const __nv_bfloat16* xb = (const __nv_bfloat16*)x;
    if (bits == 4)
      cache_write16_kernel<4, kWide><<<g, kThreads, 0, st>>>(xb, x_bs, x_rs, table, pos0, counts, c,
                                                             s, d, P, cs, status);
    else
      cache_write16_kernel<8, kWide><<<g, kThreads, 0, st>>>(xb, x_bs, x_rs, table, pos0, counts, c,
                                                             s, d, P, cs, status);
    count_launches(1);
    return cudaGetLastError();
  }
#define CSA_WRITE(T, B)                                                                          \
  (u > 1 ? cache_write_kernel<T, B, 4><<<grid, kThreads, 0, st>>>(                               \
               (const T*)x, x_bs, x_rs, table, pos0, counts, c, s, d, P, cs, status)             \
         : cache_write_kernel<T, B, 1><<<grid, kThreads, 0, st>>>(                               \
               (const T*)x, x_bs, x_rs, table, pos0, counts, c, s, d, P, cs, status))
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
  const int u = rows_per_thread(b, s, d);
  const dim3 grid = rows_grid(b, s, d, u);
  const uint8_t* c = (const uint8_t*)cache;
  if (bf16 && u > 1 && wide_rows(out, o_bs, o_rs)) {
    const dim3 g = rows_grid(b, s, d, kWide, 16);
    __nv_bfloat16* o = (__nv_bfloat16*)out;
    if (bits == 4)
      cache_read16_kernel<4, kWide><<<g, kThreads, 0, st>>>(c, table, pos0, counts, o, o_bs, o_rs,
                                                            s, d, P, cs, status);
    else
      cache_read16_kernel<8, kWide><<<g, kThreads, 0, st>>>(c, table, pos0, counts, o, o_bs, o_rs,
                                                            s, d, P, cs, status);
    count_launches(1);
    return cudaGetLastError();
  }
#define CSA_READ(T, B)                                                                           \
  (u > 1 ? cache_read_kernel<T, B, 8><<<grid, kThreads, 0, st>>>(                                \
               c, table, pos0, counts, (T*)out, o_bs, o_rs, s, d, P, cs, status)                 \
         : cache_read_kernel<T, B, 1><<<grid, kThreads, 0, st>>>(                                \
               c, table, pos0, counts, (T*)out, o_bs, o_rs, s, d, P, cs, status))
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
