// Device helpers of the row calls (include/csa_rows.h): rotary positions, and
// how a row's channels lie on lanes so that both members of a pair do on one.
#pragma once

#include <algorithm>

#include "csa_common.cuh"
#include "rows.h"

namespace csa {

// Two fp32 operations in one instruction (sm_100 and later), rounded as two.
__device__ __forceinline__ float2 as_f2(unsigned long long v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r) : "l"(pack_f32x2(a.x, a.y)), "l"(pack_f32x2(b.x, b.y)), "l"(pack_f32x2(c.x, c.y)));
  return as_f2(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pack_f32x2(a.x, a.y)), "l"(pack_f32x2(b.x, b.y)));
  return as_f2(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pack_f32x2(a.x, a.y)), "l"(pack_f32x2(b.x, b.y)));
  return as_f2(r);
}

// cos and sin of the angles that `turn` (2^-64 turns a position) makes at position pos,
// of two pairs.  angle_of gives the angle to 2^-32 turns; the nearest quarter turn is split
// off in integers, so the rest x is within pi / 4 and rounds to fp32 with an error below
// 2^-25 of it.  Minimax polynomials (Remez exchange over that range) of
// (sin x / x - 1) / x^2 and (cos x - 1 + x^2 / 2) / x^4: 1.8e-9 and 1e-10; with all
// roundings sine and cosine are within 1.7 x 2^-24.
__device__ __forceinline__ void turn_cos_sin(const long long (&turn)[2], int pos, float2* c,
                                             float2* s) {
  uint32_t q[2];
  float2 x;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t u = angle_of(turn[i], pos);
    q[i] = (u + 0x20000000u) >> 30;                     // quarter turns, mod 4
    (i ? x.y : x.x) = (float)(int32_t)(u - (q[i] << 30));
  }
  const auto all = [](float v) { return make_float2(v, v); };
  x = mul2(x, all(0x1.921fb6p-30f));                    // 2 pi / 2^32
  const float2 z = mul2(x, x);
  float2 sn = fma2(z, all(-0x1.98da70p-13f), all(0x1.1105b4p-7f));
  sn = fma2(z, sn, all(-0x1.555540p-3f));
  sn = fma2(mul2(z, x), sn, x);
  float2 cn = fma2(z, all(0x1.9a025ep-16f), all(-0x1.6c0c8cp-10f));
  cn = fma2(z, cn, all(0x1.55554ap-5f));
  cn = fma2(z, cn, all(-0.5f));
  cn = fma2(z, cn, all(1.f));
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float sv = i ? sn.y : sn.x, cv = i ? cn.y : cn.x;
    const float a = (q[i] & 1) ? sv : cv, b = (q[i] & 1) ? cv : sv;
    // the sign bits of quarters 1, 2 and of 2, 3
    (i ? c->y : c->x) = __uint_as_float(__float_as_uint(a) ^ (((q[i] + 1) & 2) << 30));
    (i ? s->y : s->x) = __uint_as_float(__float_as_uint(b) ^ ((q[i] & 2) << 30));
  }
}

// V consecutive elements in memory's form, so that rows in flight take no more
// registers than their bytes.
template <typename T, int V>
struct Pack {
  static constexpr int kWords = V * (int)sizeof(T) / 4;
  uint32_t w[kWords];

  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kWords == 1) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (kWords == 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x; w[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 v = reinterpret_cast<const uint4*>(p)[i / 4];
        w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
      }
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  __device__ __forceinline__ float2 two(int i) const {   // elements 2i and 2i + 1
    if constexpr (sizeof(T) == 4)
      return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    else
      return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  __device__ __forceinline__ void set(int i, float2 v) {
    if constexpr (sizeof(T) == 4) {
      w[2 * i] = __float_as_uint(v.x);
      w[2 * i + 1] = __float_as_uint(v.y);
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
      w[i] = reinterpret_cast<const uint32_t&>(h);
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (kWords == 1) {
      *reinterpret_cast<uint32_t*>(p) = w[0];
    } else if constexpr (kWords == 2) {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 4)
        reinterpret_cast<uint4*>(p)[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    }
  }
};

// A vector's copy into the thread's own place in shared memory: rows in flight take
// no registers, and nobody else has to be waited for.  Its pieces of up to 16 bytes
// are a CTA's threads apart, so that neighbouring threads have neighbouring pieces.
// THREADS: of the CTA, 0: blockDim.x.
template <typename VEC, int THREADS>
struct VecSlot {
  static constexpr int kPiece = sizeof(VEC) < 16 ? (int)sizeof(VEC) : 16;
  static constexpr int kPieces = sizeof(VEC) / kPiece;

  static __device__ __forceinline__ uint32_t threads() {
    return THREADS > 0 ? THREADS : blockDim.x;
  }
  // piece k of slot i of this thread
  static __device__ __forceinline__ unsigned char* place(unsigned char* base, int i, int k) {
    return base + ((uint32_t)(i * kPieces + k) * threads() + threadIdx.x) * kPiece;
  }
  static __device__ __forceinline__ void ask(unsigned char* base, int i, const void* from) {
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      const uint32_t to = (uint32_t)__cvta_generic_to_shared(place(base, i, k));
      const char* p = (const char*)from + k * kPiece;
      if constexpr (kPiece == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(p) : "memory");
      else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(p), "n"(kPiece) : "memory");
    }
  }
  // places that nothing is ever asked for, so that they count as zeros
  static __device__ __forceinline__ void zero(unsigned char* base, int i) {
#pragma unroll
    for (int k = 0; k < kPieces; ++k)
#pragma unroll
      for (int q = 0; q < kPiece / 4; ++q) reinterpret_cast<uint32_t*>(place(base, i, k))[q] = 0;
  }
  static __device__ __forceinline__ void take(unsigned char* base, int i, VEC& v) {
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      const unsigned char* p = place(base, i, k);
      if constexpr (kPiece == 16) {
        const uint4 x = *reinterpret_cast<const uint4*>(p);
        v.w[4 * k] = x.x; v.w[4 * k + 1] = x.y; v.w[4 * k + 2] = x.z; v.w[4 * k + 3] = x.w;
      } else {
#pragma unroll
        for (int q = 0; q < kPiece / 4; ++q) v.w[q] = reinterpret_cast<const uint32_t*>(p)[q];
      }
    }
  }
};
struct Word { uint32_t w[1]; };
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {   // all but the newest N groups
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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
  // whether a rotation changes channels of vector i
  __device__ __forceinline__ bool turned(int i, int first, int dim) const {
    if (ROPE == kRopeNone || c[i] < 0) return false;
    if (ROPE == kRopeHalf) return pair >= 0;
    return c[i] + V > first && c[i] < first + dim;
  }
  // index of pair e (0 .. V-1) of the unit, -1: not turned
  __device__ __forceinline__ int index(int e, int first, int dim) const {
    if (ROPE == kRopeNone) return -1;
    if (ROPE == kRopeHalf) return pair < 0 ? -1 : pair + e;
    const int v = e / (V / 2), at = c[v] + 2 * (e % (V / 2)) - first;
    return c[v] >= 0 && at >= 0 && at < dim ? at / 2 : -1;
  }
};

// Sines and cosines of a unit's pairs at position pos, times scale (the sines' sign says
// which way): `turns` has a bit for each pair that turns.
template <int ROPE, int V>
__device__ __forceinline__ void unit_cos_sin(const Unit<ROPE, V>& un, uint32_t turns,
                                             const int64_t* table, const RopeArgs& r, int pos,
                                             float (&cs)[V], float (&sn)[V]) {
  const float2 k = make_float2(r.scale, r.scale);
  const float2 back = r.back ? make_float2(-r.scale, -r.scale) : k;
#pragma unroll
  for (int e = 0; e < V; e += 2) {
    if ((turns >> e & 3u) == 0) continue;
    const long long t[2] = {table[max(0, un.index(e, r.first, r.dim))],
                            table[max(0, un.index(e + 1, r.first, r.dim))]};
    float2 c, s;
    turn_cos_sin(t, pos, &c, &s);
    c = mul2(c, k);
    s = mul2(s, back);
    cs[e] = c.x, cs[e + 1] = c.y;
    sn[e] = s.x, sn[e + 1] = s.y;
  }
}

// The turned pairs of a unit's values v[2][V / 2] (two neighbouring channels each),
// with cs and sn of its V pairs; `turns` has a bit for each pair that turns.
template <int ROPE, int V>
__device__ __forceinline__ void turn_unit(float2 (&v)[2][V / 2], const float (&cs)[V],
                                          const float (&sn)[V], uint32_t turns) {
  if (ROPE == kRopeHalf) {
    if (turns == 0) return;                       // all pairs of a unit turn, or none
#pragma unroll
    for (int e = 0; e < V / 2; ++e) {
      const float2 c = make_float2(cs[2 * e], cs[2 * e + 1]);
      const float2 s = make_float2(sn[2 * e], sn[2 * e + 1]);
      const float2 a = v[0][e], b = v[1][e];
      v[0][e] = fma2(a, c, mul2(b, make_float2(-s.x, -s.y)));
      v[1][e] = fma2(a, s, mul2(b, c));
    }
  } else if (ROPE == kRopeInter) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t all = ((1u << V / 2) - 1) << i * V / 2;
      if ((turns & all) == 0) continue;
      if ((turns & all) == all) {
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
          const int p = i * V / 2 + e;
          const float2 x = v[i][e];
          v[i][e] = make_float2(x.x * cs[p] - x.y * sn[p], x.x * sn[p] + x.y * cs[p]);
        }
      } else {                                    // first and dim are any even numbers
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
          const int p = i * V / 2 + e;
          const float2 x = v[i][e];
          if (turns >> p & 1u)
            v[i][e] = make_float2(x.x * cs[p] - x.y * sn[p], x.x * sn[p] + x.y * cs[p]);
        }
      }
    }
  }
}

// The rows as runs of up to `run` of the inner dimension, dealt out in turn: the heads of
// a token, which share its position, or (few heads) the tokens of a head.
struct Walk {
  int run, per_outer, runs, rounds;   // runs of an outer index, of all, of the lanes of a row
  bool tokens;                        // the inner dimension is the tokens

  struct At {
    int run, slot, len;               // run, row in it, its rows
    int t, bi;                        // of the run's first row
    char* p;                          // the present row
  };
  __device__ __forceinline__ void open(At& x, int s, int H, const RowStrides& st, const void* base,
                                       int esz) const {
    x.slot = x.len = 0;
    if (x.run >= runs) return;
    const int o = x.run / per_outer, i0 = (x.run - o * per_outer) * run;
    const int n = tokens ? H : s, q = o / n, r = o - q * n;
    x.bi = q;
    x.t = tokens ? i0 : r;
    x.len = min(run, (tokens ? s : H) - i0);
    x.p = (char*)base + (q * st.b + x.t * st.t + (tokens ? r : i0) * st.h) * esz;
  }
};

// The walk of `ctas` CTAs (on return no more than have a run), each with `groups` rows at a
// time and `batch` of a run together.  Runs of up to 16 rows: all read and write near one
// another, and a run's rows have one stride and, of heads, one position; shorter ones where
// they can be dealt out more evenly (opening one costs as much as a part of a row: with nothing
// for it rotations of 2 x 4096 x 32 x 128 take 54 us instead of 26, with 1.5 rows' work 25, but one
// head's 44 instead of 43).
inline Walk make_walk(int b, int s, int H, bool turned, int groups, int batch, int* ctas) {
  Walk best{};
  best.tokens = turned && H < 4;
  const long long rows = (long long)b * s * H, inner = best.tokens ? s : H;
  const long long most = (long long)*ctas * groups;
  const double open = turned && !best.tokens ? 0.6 : 0.2;
  // one round: the shortest runs; very many: the longest
  const int longest = rows <= most ? batch : 16, shortest = rows > 64 * most ? 16 : batch;
  double least = 0;
  for (int run = longest; run >= shortest; run -= batch) {
    Walk w = best;
    const long long pieces = (inner + run - 1) / run;
    w.run = (int)(((inner + pieces - 1) / pieces + batch - 1) / batch * batch);
    w.per_outer = (int)((inner + w.run - 1) / w.run);
    w.runs = (int)(rows / inner * w.per_outer);
    w.rounds = (int)((w.runs + most - 1) / most);
    const double cost = w.rounds * (w.run + open);
    if (least > 0 && cost >= least) continue;
    least = cost;
    best = w;
  }
  *ctas = (int)std::min<long long>((best.runs + groups - 1) / groups, *ctas);
  best.rounds = (best.runs + *ctas * groups - 1) / (*ctas * groups);
  return best;
}

// Lanes of a row of d channels: a power of two, with 16 channels on each.
template <int V>
int row_lanes(int d) {
  const int units = (d / V + 1) / 2;
  int l = 1;
  while (l * (8 / V) < units) l *= 2;
  return l;
}

// Whether dim and first allow vectors of v channels for the half layout's pairs.
inline bool half_by(int v, const RopeArgs& r) { return r.dim % (2 * v) == 0 && r.first % v == 0; }

// Sums over the `lanes` (a power of two) neighbouring lanes that share a row.
template <int N>
__device__ __forceinline__ void group_sums(float (&v)[N], int lanes) {
  for (int o = lanes / 2; o > 0; o >>= 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  }
}

}  // namespace csa
