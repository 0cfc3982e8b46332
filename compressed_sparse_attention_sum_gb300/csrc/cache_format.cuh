// The paged cache of the serving calls: where a row's bytes are, and the
// conversion between its codes and values.
//
// A group of 32 channels shares one power of two, kept as its exponent plus
// 127 in a byte.  A code has at most four significant bits, so code * 2^e is
// a bf16 value as long as it is a normal number; the exponents start at -110
// so that the smallest non-zero code, 2^-9, stays one, and end where the largest
// does: a masked row's weight of 0 times what it holds is 0.
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

// Slots of a sequence (P * page_size) and rows of a page: below these, a
// division by page_size is one multiplication, and all offsets within a page
// fit 32 bits.
constexpr long long kMaxSlots = 1ll << 24;
constexpr int kMaxPageSize = 32768;

struct CacheShape {
  uint32_t page_bytes;
  uint32_t scale_off;      // of a page's scale bytes
  uint32_t code_row, scale_row;   // bytes of a row
  int page_size, n_pages;
  uint32_t recip;          // ceil(2^31 / (page_size / 16))
};

inline CacheShape cache_shape(int page_size, int n_pages, int d, int bits) {
  CacheShape c;
  c.page_size = page_size;
  c.n_pages = n_pages;
  c.code_row = (uint32_t)(d * bits / 8);
  c.scale_row = (uint32_t)(d / kCacheGroup);
  c.scale_off = (uint32_t)page_size * c.code_row;
  c.page_bytes = c.scale_off + (uint32_t)page_size * c.scale_row;
  const uint32_t g = (uint32_t)page_size / 16;
  c.recip = (uint32_t)(((1ull << 31) + g - 1) / g);
  return c;
}

// slot / page_size for 0 <= slot < 2^24: with g = page_size / 16 < 2^11 + 1 and
// n = slot / 16 < 2^20, recip exceeds 2^31 / g by less than 1, so n * recip /
// 2^31 exceeds n / g by less than 2^20 / 2^31 <= 1 / g: the floor is the same.
__device__ __forceinline__ int page_index(const CacheShape& c, int slot) {
  return (int)__umulhi(((uint32_t)slot >> 4) << 1, c.recip);
}

// Byte offset of a page, and of a row's codes and scales in it.
__device__ __forceinline__ long long page_base(const CacheShape& c, int page) {
  return (long long)((unsigned long long)(uint32_t)page * c.page_bytes);
}
__device__ __forceinline__ uint32_t row_code(const CacheShape& c, int row) {
  return (uint32_t)row * c.code_row;
}
__device__ __forceinline__ uint32_t row_scale(const CacheShape& c, int row) {
  return c.scale_off + (uint32_t)row * c.scale_row;
}

// Byte offsets of the row in `slot` of a sequence whose page ids are `pages`;
// false (and the status word set) when the page id is outside the cache.
__device__ __forceinline__ bool cache_row(const CacheShape& c, const int32_t* pages, int slot,
                                          long long* code, long long* scale, int* status) {
  const int pi = page_index(c, slot), row = slot - pi * c.page_size;
  const int page = pages[pi];
  if ((unsigned)page >= (unsigned)c.n_pages) {
    set_status(status, kDevCheck, kSiteCachePage);
    return false;
  }
  const long long base = page_base(c, page);
  *code = base + row_code(c, row);
  *scale = base + row_scale(c, row);
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
  // at most what leaves the largest code (e4m3: its NaN code too, 480) a bf16 value
  return min(max(e, kCacheMinExp), BITS == 4 ? 125 : 119);
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
