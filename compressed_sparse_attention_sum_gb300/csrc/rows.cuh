// Device helpers of the row calls (include/csa_rows.h): rotary positions, and
// how a row's channels lie on lanes so that both members of a pair do on one.
#pragma once

#include "csa_common.cuh"
#include "rows.h"

namespace csa {

// cos and sin of the angle that `turn` (2^-64 turns a position) makes at position
// pos.  The product modulo 2^64 is exact: whole turns drop out, for any int32
// position.  Its top 32 bits are the angle to 2^-32 turns; the nearest quarter turn
// is split off in integers, so the rest is within pi / 4 and rounds to fp32 with an
// error below 2^-25 of it, where the Taylor series of sine and cosine up to x^9 and
// x^10 end at 1.8e-9 and 2e-10.
__device__ __forceinline__ void turn_cos_sin(long long turn, int pos, float* c, float* s) {
  const uint32_t u = (uint32_t)((unsigned long long)(turn * (long long)pos) >> 32);
  const uint32_t q = (u + 0x20000000u) >> 30;           // quarter turns, mod 4
  const float x = (float)(int32_t)(u - (q << 30)) * 0x1.921fb6p-30f;   // 2 pi / 2^32
  const float z = x * x;
  float sn = fmaf(z, 1.f / 362880.f, -1.f / 5040.f);
  sn = fmaf(z, sn, 1.f / 120.f);
  sn = fmaf(z, sn, -1.f / 6.f);
  sn = fmaf(z * x, sn, x);
  float cn = fmaf(z, -1.f / 3628800.f, 1.f / 40320.f);
  cn = fmaf(z, cn, -1.f / 720.f);
  cn = fmaf(z, cn, 1.f / 24.f);
  cn = fmaf(z, cn, -0.5f);
  cn = fmaf(z, cn, 1.f);
  const float a = (q & 1) ? sn : cn, b = (q & 1) ? cn : sn;
  *c = ((q + 1) & 2) ? -a : a;
  *s = (q & 2) ? -b : b;
}

// V consecutive elements as floats (V = 8: 16-byte accesses, or two for fp32).
template <int V, typename T>
__device__ __forceinline__ void load_v(const T* p, float* f) {
  if constexpr (V == 8) {
    load8(p, f);
  } else {
    static_assert(V == 2, "");
    if constexpr (sizeof(T) == 2) {
      const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p));
      f[0] = v.x;
      f[1] = v.y;
    } else {
      const float2 v = *reinterpret_cast<const float2*>(p);
      f[0] = v.x;
      f[1] = v.y;
    }
  }
}
template <int V, typename T>
__device__ __forceinline__ void store_v(T* p, const float* f) {
  if constexpr (V == 8) {
    store8(p, f);
  } else {
    if constexpr (sizeof(T) == 2)
      *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(f[0], f[1]);
    else
      *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]);
  }
}

// A row's channels as d / V vectors, two of them (a unit) at a time on one lane.
//   no rotation, interleaved pairs: unit u has the vectors u and u + ceil(n / 2);
//     a pair lies within a vector, as V and `first` are even
//   half: the units of the turned channels have the vectors that are dim / 2
//     apart, first the pairs' first members; the other vectors follow in order
enum { kRopeNone = 0, kRopeInter = 1, kRopeHalf = 2 };

template <int ROPE, int V>
struct Unit {
  int c[2];          // first channels of the two vectors, -1: none
  int pair;          // half: index of the first of its V pairs, -1: not turned

  __device__ __forceinline__ Unit(int u, int d, int first, int dim) {
    const int n = d / V;
    pair = -1;
    if (ROPE == kRopeHalf) {
      const int hr = dim / (2 * V), r0 = first / V, others = n - 2 * hr;
      if (u < hr) {
        c[0] = (r0 + u) * V;
        c[1] = c[0] + hr * V;
        pair = u * V;
      } else {
        const int e0 = u - hr, e1 = e0 + (others + 1) / 2;
        c[0] = e0 < (others + 1) / 2 ? (e0 < r0 ? e0 : e0 + 2 * hr) * V : -1;
        c[1] = c[0] >= 0 && e1 < others ? (e1 < r0 ? e1 : e1 + 2 * hr) * V : -1;
      }
    } else {
      const int m = (n + 1) / 2;
      c[0] = u < m ? u * V : -1;
      c[1] = u < m && u + m < n ? (u + m) * V : -1;
    }
  }
  // index of pair e (0 .. V-1) of the unit, -1: not turned
  __device__ __forceinline__ int index(int e, int first, int dim) const {
    if (ROPE == kRopeNone) return -1;
    if (ROPE == kRopeHalf) return pair < 0 ? -1 : pair + e;
    const int v = e / (V / 2), at = c[v] + 2 * (e % (V / 2)) - first;
    return c[v] >= 0 && at >= 0 && at < dim ? at / 2 : -1;
  }
};

// The members of pair e in a unit's values v[2][V].
template <int ROPE, int V>
__device__ __forceinline__ void turn_pair(float (&v)[2][V], int e, float c, float s) {
  float &a = ROPE == kRopeHalf ? v[0][e] : v[e / (V / 2)][2 * (e % (V / 2))];
  float &b = ROPE == kRopeHalf ? v[1][e] : v[e / (V / 2)][2 * (e % (V / 2)) + 1];
  const float x = a, y = b;
  a = x * c - y * s;
  b = x * s + y * c;
}

// Sum over the `lanes` (a power of two) neighbouring lanes that share a row.
__device__ __forceinline__ float group_sum(float v, int lanes) {
  for (int o = lanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

}  // namespace csa
