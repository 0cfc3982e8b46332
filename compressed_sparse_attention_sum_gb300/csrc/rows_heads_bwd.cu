// The gradient of the norms of rows of up to 512 channels, and of a norm followed by
// rotary positions (csa_norm_rope_bwd, csa_norm_bwd of narrow rows).
//
// With dy the gradient turned back by the row's angle, g = dy weight and xh = (x - m) r:
// dx = r (g - mean(g) - xh mean(g xh)), dweight = sum dy xh, dbias = sum dy (RMS: m = 0
// and no mean(g)).  Rows lie on lanes as in rows_heads.cu.
#include "csa_kernels.h"
#include "rows.cuh"

namespace csa {
namespace {

constexpr int kThreads = 256;

template <int V>
__device__ __forceinline__ void load_v(const float* p, float* f) {
  Pack<float, V> k;
  k.load(p);
#pragma unroll
  for (int e = 0; e < V; ++e) f[e] = __uint_as_float(k.w[e]);
}
template <int V, typename T>
__device__ __forceinline__ void get(const Pack<T, V>& p, float (&f)[V]) {
#pragma unroll
  for (int e = 0; e < V / 2; ++e) f[2 * e] = p.two(e).x, f[2 * e + 1] = p.two(e).y;
}
template <int V, typename T>
__device__ __forceinline__ void store_v(T* p, const float* f) {
  Pack<T, V> k;
#pragma unroll
  for (int e = 0; e < V / 2; ++e) k.set(e, make_float2(f[2 * e], f[2 * e + 1]));
  k.store(p);
}
template <int ROPE, int V>
__device__ __forceinline__ void turn_pair(float (&v)[2][V], int e, float c, float s) {
  float &a = ROPE == kRopeHalf ? v[0][e] : v[e / (V / 2)][2 * (e % (V / 2))];
  float &b = ROPE == kRopeHalf ? v[1][e] : v[e / (V / 2)][2 * (e % (V / 2)) + 1];
  const float x = a, y = b;
  a = x * c - y * s;
  b = x * s + y * c;
}

__device__ __forceinline__ float group_sum(float v, int lanes) {
  float x[1] = {v};
  group_sums(x, lanes);
  return x[0];
}

// Sums that a norm needs of a row's values v (zero where there are none); n channels.
template <int V, int NU>
__device__ __forceinline__ void row_stats(float (&v)[NU][2][V], const bool (&has)[NU][2], int kind,
                                          float eps, int lanes, float inv_n, float* mean,
                                          float* rstd) {
  float m = 0.f;
  if (kind == kNormLayer) {
#pragma unroll
    for (int k = 0; k < NU; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) m += v[k][0][e] + v[k][1][e];
    m = group_sum(m, lanes) * inv_n;
  }
  float q = 0.f;
#pragma unroll
  for (int k = 0; k < NU; ++k)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float c = has[k][i] ? v[k][i][e] - m : 0.f;
        q = fmaf(c, c, q);
      }
  q = group_sum(q, lanes) * inv_n;
  *mean = m;
  *rstd = 1.f / sqrtf(q + eps);
}

template <typename TX, typename TG, typename TD, int ROPE, int V>
__global__ void __launch_bounds__(kThreads) rows_bwd_kernel(RowsBwd a, int lanes) {
  constexpr int NU = 8 / V;
  extern __shared__ float s_sum[];                // [warps][wanted][d]
  const int lane = threadIdx.x & (lanes - 1);
  const int rows = a.b * a.s * a.H, step = (int)((long long)gridDim.x * kThreads / lanes);
  float dw[NU][2][V], db[NU][2][V];
  bool has[NU][2];
  int at[NU][2];
#pragma unroll
  for (int k = 0; k < NU; ++k) {
    const Unit<ROPE, V> u(lane + k * lanes, a.d, a.rope.first, a.rope.dim);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      at[k][i] = u.c[i];
      has[k][i] = u.c[i] >= 0;
#pragma unroll
      for (int e = 0; e < V; ++e) dw[k][i][e] = db[k][i][e] = 0.f;
    }
  }
  const float inv_n = 1.f / a.d;
  const long long row0 = ((long long)blockIdx.x * kThreads + threadIdx.x) / lanes;
  // every lane of a warp takes part in every round of its first row (shuffles)
  const long long warp0 = ((long long)blockIdx.x * kThreads + (threadIdx.x & ~31)) / lanes;
  for (long long off = 0; warp0 + off < rows; off += step) {
    const bool live = row0 + off < rows;
    const int r = live ? (int)(row0 + off) : rows - 1;
    const int tok = r / a.H, h = r - tok * a.H, bi = tok / a.s, t = tok - bi * a.s;
    const TX* x = (const TX*)a.x + bi * a.xs.b + t * a.xs.t + h * a.xs.h;
    const TG* g = (const TG*)a.dout + bi * a.gs.b + t * a.gs.t + h * a.gs.h;
    TD* dx = (TD*)a.dx + bi * a.ds.b + t * a.ds.t + h * a.ds.h;
    float v[NU][2][V], dy[NU][2][V];
#pragma unroll
    for (int k = 0; k < NU; ++k)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (has[k][i]) {
          Pack<TX, V> px;
          Pack<TG, V> pg;
          px.load(x + at[k][i]);
          pg.load(g + at[k][i]);
          get<V>(px, v[k][i]);
          get<V>(pg, dy[k][i]);
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e) v[k][i][e] = dy[k][i][e] = 0.f;
        }
      }
    if constexpr (ROPE != kRopeNone) {
      const int pos = a.pos != nullptr ? a.pos[bi * a.pos_stride + t] : t;
#pragma unroll
      for (int k = 0; k < NU; ++k) {
        const Unit<ROPE, V> u(lane + k * lanes, a.d, a.rope.first, a.rope.dim);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const int p = u.index(e, a.rope.first, a.rope.dim);
          if (p < 0) continue;
          const long long turn[2] = {a.rope.turns[p], 0};
          float2 c, s;
          turn_cos_sin(turn, pos, &c, &s);
          turn_pair<ROPE, V>(dy[k], e, c.x * a.rope.scale, -s.x * a.rope.scale);
        }
      }
    }
    float mean, rstd;
    row_stats<V, NU>(v, has, a.kind, a.eps, lanes, inv_n, &mean, &rstd);
    float sg = 0.f, sgx = 0.f;
#pragma unroll
    for (int k = 0; k < NU; ++k)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (!has[k][i]) continue;
        float w[V];
        if (a.weight != nullptr) load_v<V>(a.weight + at[k][i], w);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float xh = (v[k][i][e] - mean) * rstd;
          if (live) {
            dw[k][i][e] = fmaf(dy[k][i][e], xh, dw[k][i][e]);
            db[k][i][e] += dy[k][i][e];
          }
          v[k][i][e] = xh;
          if (a.weight != nullptr) dy[k][i][e] *= w[e];
          sg += dy[k][i][e];
          sgx = fmaf(dy[k][i][e], xh, sgx);
        }
      }
    sgx = group_sum(sgx, lanes) * inv_n;
    sg = a.kind == kNormLayer ? group_sum(sg, lanes) * inv_n : 0.f;
    if (!live) continue;
#pragma unroll
    for (int k = 0; k < NU; ++k)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (!has[k][i]) continue;
        float o[V];
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = rstd * (dy[k][i][e] - sg - v[k][i][e] * sgx);
        store_v<V>(dx + at[k][i], o);
      }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int wanted = (a.dweight != nullptr) + (a.dbias != nullptr);
  if (wanted == 0) return;
  const int warp = threadIdx.x >> 5;
#pragma unroll
  for (int k = 0; k < NU; ++k)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float x = dw[k][i][e], y = db[k][i][e];
        for (int o = lanes; o < 32; o <<= 1) {
          x += __shfl_xor_sync(0xffffffffu, x, o);
          y += __shfl_xor_sync(0xffffffffu, y, o);
        }
        if ((threadIdx.x & 31) < lanes && has[k][i]) {
          float* to = s_sum + (size_t)warp * wanted * a.d + at[k][i] + e;
          if (a.dweight != nullptr) *to = x;
          if (a.dbias != nullptr) to[(wanted - 1) * a.d] = y;
        }
      }
  __syncthreads();
  for (int c = threadIdx.x; c < wanted * a.d; c += kThreads) {
    float x = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) x += s_sum[(size_t)w * wanted * a.d + c];
    a.parts[(size_t)blockIdx.x * wanted * a.d + c] = x;
  }
}

template <typename TX, typename TG, typename TD, int ROPE, int V>
cudaError_t bwd(const RowsBwd& a, int ctas, cudaStream_t st) {
  const int wanted = (a.dweight != nullptr) + (a.dbias != nullptr);
  const size_t smem = (size_t)(kThreads / 32) * wanted * a.d * sizeof(float);
  rows_bwd_kernel<TX, TG, TD, ROPE, V>
      <<<(unsigned)ctas, kThreads, smem, st>>>(a, row_lanes<V>(a.d));
  count_launches(1);
  return cudaGetLastError();
}

template <typename TX, typename TG, typename TD>
cudaError_t bwd_rope(const RowsBwd& a, int ctas, cudaStream_t st) {
  if (a.rope.turns == nullptr) return bwd<TX, TG, TD, kRopeNone, 8>(a, ctas, st);
  if (!a.rope.half) return bwd<TX, TG, TD, kRopeInter, 8>(a, ctas, st);
  if (half_by(8, a.rope)) return bwd<TX, TG, TD, kRopeHalf, 8>(a, ctas, st);
  return bwd<TX, TG, TD, kRopeHalf, 2>(a, ctas, st);
}

template <typename TX>
cudaError_t bwd_types(const RowsBwd& a, int ctas, cudaStream_t st) {
  using bf = __nv_bfloat16;
  if (a.g_bf16) return a.dx_bf16 ? bwd_rope<TX, bf, bf>(a, ctas, st) : bwd_rope<TX, bf, float>(a, ctas, st);
  return a.dx_bf16 ? bwd_rope<TX, float, bf>(a, ctas, st) : bwd_rope<TX, float, float>(a, ctas, st);
}

}  // namespace

cudaError_t launch_rows_bwd(const RowsBwd& a, int ctas, cudaStream_t st) {
  return a.x_bf16 ? bwd_types<__nv_bfloat16>(a, ctas, st) : bwd_types<float>(a, ctas, st);
}

}  // namespace csa
