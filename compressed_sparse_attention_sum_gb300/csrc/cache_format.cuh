// The paged cache of the serving calls: where a row's bytes are, and the
// conversion between its codes and values.
//
// A group of 32 channels shares one power of two, kept as its exponent plus
// 127 in a byte.  A code has at most four significant bits, so code * 2^e is
// a bf16 value as long as it is a normal number; the exponents start at -110
// so that the smallest non-zero code, 2^-9, stays one.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "csa_common.cuh"

namespace csa {

constexpr int kCacheGroup = 32;
constexpr int kCacheMinExp = -110;

// Sites recorded with CSA_ERR_DEVICE_CHECK: a page id outside the cache; a
// sequence length, position or count outside its range.
constexpr int kSiteCachePage = 0x71, kSiteCacheRange = 0x72;

struct CacheShape {
  long long page_bytes;
  long long scale_off;     // of a page's scale bytes
  int page_size, n_pages;
  int code_row, scale_row; // bytes of a row
};

inline CacheShape cache_shape(int page_size, int n_pages, int d, int bits) {
  CacheShape c;
  c.page_size = page_size;
  c.n_pages = n_pages;
  c.code_row = d * bits / 8;
  c.scale_row = d / kCacheGroup;
  c.scale_off = (long long)page_size * c.code_row;
  c.page_bytes = c.scale_off + (long long)page_size * c.scale_row;
  return c;
}

// Byte offsets of the row in `slot` of a sequence whose page ids are `pages`;
// false (and the status word set) when the page id is outside the cache.
__device__ __forceinline__ bool cache_row(const CacheShape& c, const int32_t* pages, int slot,
                                          long long* code, long long* scale, int* status) {
  const int pi = slot / c.page_size, row = slot - pi * c.page_size;
  const int page = pages[pi];
  if ((unsigned)page >= (unsigned)c.n_pages) {
    set_status(status, kDevCheck, kSiteCachePage);
    return false;
  }
  const long long base = (long long)page * c.page_bytes;
  *code = base + (long long)row * c.code_row;
  *scale = base + c.scale_off + (long long)row * c.scale_row;
  return true;
}

// 2^e for e in [-126, 127].
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// The value 2^(s - 127) of a scale byte that csa_cache_write wrote.
__device__ __forceinline__ float scale_value(uint32_t s) { return __uint_as_float(s << 23); }

// Exponent e of the smallest 2^e that holds amax: amax <= 1.5 * 2^2 * 2^e for
// e2m1 (largest code 6), 1.75 * 2^8 * 2^e for e4m3 (448).
template <int BITS>
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax) & 0x7fffffffu;
  const int ex = (int)(u >> 23) - 127;
  const uint32_t man = u & 0x7fffffu;
  const int e = BITS == 4 ? ex - 2 + (man > 0x400000u ? 1 : 0) : ex - 8 + (man > 0x600000u ? 1 : 0);
  return min(max(e, kCacheMinExp), 125);   // 125: an infinite amax
}

// Eight values, already divided by the scale -> codes (4 bits: one word; 8
// bits: two words), rounded to nearest even.
__device__ __forceinline__ uint32_t encode8_e2m1(const float (&y)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return r;
}
__device__ __forceinline__ uint32_t encode4_e4m3(float y0, float y1, float y2, float y3) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(y1), "f"(y0));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(y3), "f"(y2));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

// One code -> fp32, not yet scaled by the group's power of two.  The code's
// exponent and mantissa bits, moved to the top of fp32's mantissa, are the
// value times 2^-126 (e2m1) or 2^-120 (e4m3), subnormal codes included.
__device__ __forceinline__ float code_e2m1(uint32_t c) {
  return __uint_as_float(((c & 8u) << 28) | ((c & 7u) << 22)) * pow2f(126);
}
__device__ __forceinline__ float code_e4m3(uint32_t c) {
  return __uint_as_float(((c & 0x80u) << 24) | ((c & 0x7fu) << 20)) * pow2f(120);
}

// Eight consecutive channels (c0 a multiple of 8) of a row as fp32.
template <int BITS>
__device__ __forceinline__ void cache_load8(const uint8_t* code, float scale, int c0,
                                            float (&v)[8]) {
  if constexpr (BITS == 4) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(code + c0 / 2);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = code_e2m1(w >> (4 * i)) * scale;
  } else {
    const uint2 w = *reinterpret_cast<const uint2*>(code + c0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = code_e4m3(w.x >> (8 * i)) * scale;
      v[i + 4] = code_e4m3(w.y >> (8 * i)) * scale;
    }
  }
}

}  // namespace csa
