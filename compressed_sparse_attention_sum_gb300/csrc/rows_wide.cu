// Layer and RMS norm of rows of up to 32768 channels, one CTA a row, and their
// gradient (the formulas stand in rows_heads.cu); the sums of the CTAs' shares of
// the weight's and the bias's gradient.
#include "csa_kernels.h"
#include "rows.cuh"

namespace csa {
namespace {

// Sum over the CTA; every thread gets it.  `s` has room for 32 floats, and a
// barrier lies between two uses.
__device__ __forceinline__ float block_sum(float v, float* s) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  return warp_sum(lane < (int)(blockDim.x >> 5) ? s[lane] : 0.f);
}

template <typename T, int NV>
__global__ void __launch_bounds__(1024) norm_wide_kernel(RowsFwd a) {
  __shared__ float s_a[32], s_b[32];
  const int n = a.d, nv = n / 8;
  const T* x = (const T*)a.x + (long long)blockIdx.x * a.xs.h;
  T* out = (T*)a.out + (long long)blockIdx.x * a.os.h;
  float v[NV][8];
  float m = 0.f, q = 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = threadIdx.x + k * blockDim.x;
    if (i >= nv) continue;
    load8(x + i * 8, v[k]);
#pragma unroll
    for (int e = 0; e < 8; ++e) m += v[k][e];
  }
  m = a.kind == kNormLayer ? block_sum(m, s_a) / n : 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = threadIdx.x + k * blockDim.x;
    if (i >= nv) continue;
#pragma unroll
    for (int e = 0; e < 8; ++e) q = fmaf(v[k][e] - m, v[k][e] - m, q);
  }
  const float rstd = 1.f / sqrtf(block_sum(q, s_b) / n + a.eps);
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = threadIdx.x + k * blockDim.x;
    if (i >= nv) continue;
    float w[8], b[8];
    if (a.weight != nullptr) load8(a.weight + i * 8, w);
    if (a.bias != nullptr) load8(a.bias + i * 8, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float y = (v[k][e] - m) * rstd;
      if (a.weight != nullptr) y *= w[e];
      if (a.bias != nullptr) y += b[e];
      v[k][e] = y;
    }
    store8(out + i * 8, v[k]);
  }
}

template <typename TX, typename TG, typename TD, int NV>
__global__ void __launch_bounds__(1024) norm_wide_bwd_kernel(RowsBwd a) {
  __shared__ float s_a[32], s_b[32], s_c[32], s_d[32];
  const int n = a.d, nv = n / 8;
  float dw[NV][8], db[NV][8];
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[k][e] = db[k][e] = 0.f;
  for (int row = blockIdx.x; row < a.H; row += gridDim.x) {
    const TX* x = (const TX*)a.x + row * a.xs.h;
    const TG* g = (const TG*)a.dout + row * a.gs.h;
    TD* dx = (TD*)a.dx + row * a.ds.h;
    float v[NV][8], gy[NV][8];
    float m = 0.f, q = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = threadIdx.x + k * blockDim.x;
      if (i >= nv) continue;
      load8(x + i * 8, v[k]);
      load8(g + i * 8, gy[k]);
#pragma unroll
      for (int e = 0; e < 8; ++e) m += v[k][e];
    }
    m = a.kind == kNormLayer ? block_sum(m, s_a) / n : 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = threadIdx.x + k * blockDim.x;
      if (i >= nv) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) q = fmaf(v[k][e] - m, v[k][e] - m, q);
    }
    const float rstd = 1.f / sqrtf(block_sum(q, s_b) / n + a.eps);
    float sg = 0.f, sgx = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = threadIdx.x + k * blockDim.x;
      if (i >= nv) continue;
      float w[8];
      if (a.weight != nullptr) load8(a.weight + i * 8, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float xh = (v[k][e] - m) * rstd;
        dw[k][e] = fmaf(gy[k][e], xh, dw[k][e]);
        db[k][e] += gy[k][e];
        v[k][e] = xh;
        if (a.weight != nullptr) gy[k][e] *= w[e];
        sg += gy[k][e];
        sgx = fmaf(gy[k][e], xh, sgx);
      }
    }
    sgx = block_sum(sgx, s_c) / n;
    sg = block_sum(sg, s_d) / n;
    if (a.kind != kNormLayer) sg = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = threadIdx.x + k * blockDim.x;
      if (i >= nv) continue;
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = rstd * (gy[k][e] - sg - v[k][e] * sgx);
      store8(dx + i * 8, o);
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int wanted = (a.dweight != nullptr) + (a.dbias != nullptr);
  float* to = a.parts + (size_t)blockIdx.x * wanted * n;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = threadIdx.x + k * blockDim.x;
    if (i >= nv) continue;
    if (a.dweight != nullptr) store8(to + i * 8, dw[k]);
    if (a.dbias != nullptr) store8(to + (size_t)(wanted - 1) * n + i * 8, db[k]);
  }
}

// A programmatic dependent of the kernel that wrote the parts: 32 columns a CTA,
// the parts dealt to its warps and joined in a fixed order.
constexpr int kSumWarps = 8;
__global__ void __launch_bounds__(32 * kSumWarps) sum_parts_kernel(
    const float* __restrict__ parts, int ctas, float* __restrict__ dweight,
    float* __restrict__ dbias, int n) {
  __shared__ float s[kSumWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cols = n * ((dweight != nullptr) + (dbias != nullptr)), c = blockIdx.x * 32 + lane;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float x = 0.f;
  if (c < cols)
    for (int p = warp; p < ctas; p += kSumWarps) x += parts[(size_t)p * cols + c];
  s[warp][lane] = x;
  __syncthreads();
  if (warp != 0 || c >= cols) return;
  x = 0.f;
#pragma unroll
  for (int w = 0; w < kSumWarps; ++w) x += s[w][lane];
  if (dweight == nullptr)
    dbias[c] = x;
  else if (c < n)
    dweight[c] = x;
  else
    dbias[c - n] = x;
}

// Threads of a row of n channels (a multiple of 32, at most 1024) and its vectors of
// 8 on each.
int wide_threads(int n, int nv) { return ((n / 8 + nv - 1) / nv + 31) / 32 * 32; }
int wide_vectors(int n) { return n <= 8192 ? 1 : n <= 16384 ? 2 : 4; }

template <typename TX, typename TG, typename TD>
cudaError_t wide_bwd(const RowsBwd& a, int ctas, cudaStream_t st) {
  const int nv = wide_vectors(a.d);
  const int threads = wide_threads(a.d, nv);
  if (nv == 1)
    norm_wide_bwd_kernel<TX, TG, TD, 1><<<ctas, threads, 0, st>>>(a);
  else if (nv == 2)
    norm_wide_bwd_kernel<TX, TG, TD, 2><<<ctas, threads, 0, st>>>(a);
  else
    norm_wide_bwd_kernel<TX, TG, TD, 4><<<ctas, threads, 0, st>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

template <typename TX>
cudaError_t wide_bwd_types(const RowsBwd& a, int ctas, cudaStream_t st) {
  using bf = __nv_bfloat16;
  if (a.g_bf16) return a.dx_bf16 ? wide_bwd<TX, bf, bf>(a, ctas, st) : wide_bwd<TX, bf, float>(a, ctas, st);
  return a.dx_bf16 ? wide_bwd<TX, float, bf>(a, ctas, st) : wide_bwd<TX, float, float>(a, ctas, st);
}

template <typename T>
cudaError_t wide_fwd(const RowsFwd& a, cudaStream_t st) {
  const int nv = wide_vectors(a.d);
  const int threads = wide_threads(a.d, nv);
  if (nv == 1)
    norm_wide_kernel<T, 1><<<(unsigned)a.H, threads, 0, st>>>(a);
  else if (nv == 2)
    norm_wide_kernel<T, 2><<<(unsigned)a.H, threads, 0, st>>>(a);
  else
    norm_wide_kernel<T, 4><<<(unsigned)a.H, threads, 0, st>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace

int rows_bwd_ctas(long long rows, int n) {
  const long long most = n <= kMaxHeadWidth ? 152 * 4 : 152 * 2;
  // rows of a CTA of the narrow kernel at once: at least 8 (32 lanes a row)
  const long long need = n <= kMaxHeadWidth ? (rows + 7) / 8 : rows;
  return (int)(need < most ? (need > 0 ? need : 1) : most);
}

cudaError_t launch_norm_wide(const RowsFwd& a, cudaStream_t st) {
  return a.x_bf16 ? wide_fwd<__nv_bfloat16>(a, st) : wide_fwd<float>(a, st);
}

cudaError_t launch_norm_wide_bwd(const RowsBwd& a, int ctas, cudaStream_t st) {
  return a.x_bf16 ? wide_bwd_types<__nv_bfloat16>(a, ctas, st) : wide_bwd_types<float>(a, ctas, st);
}

cudaError_t launch_sum_parts(const float* parts, int ctas, float* dweight, float* dbias, int n,
                             cudaStream_t st) {
  const int cols = n * ((dweight != nullptr) + (dbias != nullptr));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((cols + 31) / 32));
  cfg.blockDim = dim3(32 * kSumWarps);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  count_launches(1);
  return cudaLaunchKernelEx(&cfg, sum_parts_kernel, parts, ctas, dweight, dbias, n);
}

}  // namespace csa
