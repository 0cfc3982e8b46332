// Codes of the cache to bf16 tiles in shared memory, the operands of the
// tensor-core kernels of the serving calls.
//
// A code's exponent and mantissa bits, moved under bf16's, are its value times
// 2^-126 (e2m1) or 2^-120 (e4m3), subnormal codes included; one product with
// the group's scale times that power makes it right, exactly (a code has at
// most four significant bits).  A shift of a 32-bit word moves two codes at
// once, four (e2m1) or two (e4m3) codes apart, so a row's channels come out
// permuted within each eight: position p holds channel channel_of(p).  The
// other operand of a product over channels is permuted alike (permute8).
#pragma once

#include "cache_format.cuh"

namespace csa {

// A row of zeros, read in the place of a masked one: with an address chosen
// instead of a branch, a load stays in flight until its value is used.
static __device__ __align__(32) uint4 g_zero_row[32];

template <int BITS>
__device__ __forceinline__ int channel_of(int p) {
  return BITS == 4 ? (p & ~7) | ((p >> 1) & 3) | ((p & 1) << 2)
                   : (p & ~3) | ((p >> 1) & 1) | ((p & 1) << 1);
}

// Eight bf16 channels into the expanded codes' order.
template <int BITS>
__device__ __forceinline__ uint4 permute8(uint4 v) {
  if constexpr (BITS == 4)
    return make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                      __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
  else
    return make_uint4(__byte_perm(v.x, v.y, 0x5410), __byte_perm(v.x, v.y, 0x7632),
                      __byte_perm(v.z, v.w, 0x5410), __byte_perm(v.z, v.w, 0x7632));
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// One scale group (32 channels) of a row as fetched.
template <int BITS>
struct Codes {
  uint4 w[BITS / 4];
  uint32_t scale;
};

// Eight codes -> four words of two bf16, not yet scaled, in permuted order.
template <int BITS>
__device__ __forceinline__ void expand8(uint32_t w0, uint32_t w1, uint32_t (&o)[4]) {
  constexpr uint32_t S = 0x80008000u;
  if constexpr (BITS == 4) {
    constexpr uint32_t M = 0x01C001C0u;
    o[0] = ((w0 << 12) & S) | ((w0 << 6) & M);
    o[1] = ((w0 << 8) & S) | ((w0 << 2) & M);
    o[2] = ((w0 << 4) & S) | ((w0 >> 2) & M);
    o[3] = (w0 & S) | ((w0 >> 6) & M);
  } else {
    constexpr uint32_t M = 0x07F007F0u;
    o[0] = ((w0 << 8) & S) | ((w0 << 4) & M);
    o[1] = (w0 & S) | ((w0 >> 4) & M);
    o[2] = ((w1 << 8) & S) | ((w1 << 4) & M);
    o[3] = (w1 & S) | ((w1 >> 4) & M);
  }
}

// Words of expand8 times the group's scale byte's 2^(s - 127).
template <int BITS>
__device__ __forceinline__ void scale8(uint32_t s, uint32_t (&o)[4]) {
  // scale * 2^126 (2^120) as bf16 bits; where that is beyond bf16 (a scale
  // above 2^1, 2^7) a second factor carries the rest
  const int e = (int)s + (BITS == 4 ? 126 : 120);
  const uint32_t f1 = (uint32_t)min(e, 254) * 0x00800080u;
#pragma unroll
  for (int x = 0; x < 4; ++x) o[x] = mul_bf16x2(o[x], f1);
  if (e > 254) {
    const uint32_t f2 = (uint32_t)(e - 254 + 127) * 0x00800080u;
#pragma unroll
    for (int x = 0; x < 4; ++x) o[x] = mul_bf16x2(o[x], f2);
  }
}

// Permuted words of eight channels back into channel order.
template <int BITS>
__device__ __forceinline__ uint4 natural8(const uint32_t (&o)[4]) {
  if constexpr (BITS == 4)
    return make_uint4(__byte_perm(o[0], o[1], 0x5410), __byte_perm(o[2], o[3], 0x5410),
                      __byte_perm(o[0], o[1], 0x7632), __byte_perm(o[2], o[3], 0x7632));
  else
    return make_uint4(__byte_perm(o[0], o[1], 0x5410), __byte_perm(o[0], o[1], 0x7632),
                      __byte_perm(o[2], o[3], 0x5410), __byte_perm(o[2], o[3], 0x7632));
}

// A scale group (32 channels) -> 16 words of two bf16, in permuted order.
template <int BITS>
__device__ __forceinline__ void expand_words(const Codes<BITS>& c, uint32_t (&o)[16]) {
  const uint32_t words[8] = {c.w[0].x, c.w[0].y, c.w[0].z, c.w[0].w,
                             c.w[BITS / 4 - 1].x, c.w[BITS / 4 - 1].y, c.w[BITS / 4 - 1].z,
                             c.w[BITS / 4 - 1].w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t v[4];
    if constexpr (BITS == 4) expand8<4>(words[j], 0u, v);
    else expand8<8>(words[2 * j], words[2 * j + 1], v);
    scale8<BITS>(c.scale, v);
#pragma unroll
    for (int x = 0; x < 4; ++x) o[4 * j + x] = v[x];
  }
}

// Those words as four 16-byte chunks (ch0 .. ch0 + 3) of a row of 128 bytes in
// the 128-byte swizzle (row & 7 = sw).
__device__ __forceinline__ void store_words(const uint32_t (&o)[16], unsigned char* row, int ch0,
                                            int sw) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *reinterpret_cast<uint4*>(row + (((ch0 + j) ^ sw) << 4)) =
        make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
}

// The sum of their squares, added in bf16 (16 to an accumulator: within 4%
// below and above).
__device__ __forceinline__ float words_norm2(const uint32_t (&o)[16]) {
  __nv_bfloat162 sq = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
  for (int x = 0; x < 16; ++x) {
    const __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162*>(&o[x]);
    sq = __hfma2(v, v, sq);
  }
  const float2 f = __bfloat1622float2(sq);
  return f.x + f.y;
}

}  // namespace csa
