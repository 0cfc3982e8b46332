// C ABI entry points of the row calls (include/csa_rows.h): argument validation
// and dispatch.  Every check runs before the first CUDA call.
#include <cmath>
#include <cstdint>

#include "../../include/csa_rows.h"
#include "cache_format.cuh"
#include "compress_decode.h"
#include "csa_kernels.h"
#include "indexer_host.h"
#include "rows.h"

namespace csa {
int* device_status_word();
}  // namespace csa

namespace {

using csa::aligned16;
using csa::RopeArgs;

csa_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? CSA_OK : CSA_ERR_CUDA; }

bool valid_dtype(csa_dtype_t dt) { return dt == CSA_FP32 || dt == CSA_BF16; }

bool valid_norm(int kind, const float* weight, const float* bias, float eps) {
  return (kind == CSA_NORM_RMS || kind == CSA_NORM_LAYER) && aligned16(weight) && aligned16(bias) &&
         eps >= 0.f && std::isfinite(eps);
}

bool valid_rope(const csa_rope_t* r, int d) {
  if (r == nullptr || r->turns == nullptr || !aligned16(r->turns)) return false;
  if (r->layout != CSA_ROPE_INTERLEAVED && r->layout != CSA_ROPE_HALF) return false;
  if (r->dim < 2 || r->dim % 2 != 0 || (r->layout == CSA_ROPE_HALF && r->dim % 4 != 0)) return false;
  if (r->first < 0 || r->first % 2 != 0 || r->dim > d || r->first > d - r->dim) return false;
  return std::isfinite(r->scale);
}

// null: no rotation
RopeArgs rope_args(const csa_rope_t* r, bool back) {
  RopeArgs a{};
  if (r == nullptr) return a;
  a.turns = r->turns;
  a.dim = r->dim;
  a.first = r->first;
  a.scale = r->scale;
  a.half = r->layout == CSA_ROPE_HALF;
  a.back = back;
  return a;
}

constexpr long long kMaxRowCount = 1ll << 30;   // row and run indexes, with a step more, fit 32 bits

// Rows [b, s, H] at these strides start on 16-byte boundaries.
bool valid_in(const void* p, csa_row_strides_t st, csa_dtype_t dt, int b, int s, int H) {
  const long long unit = dt == CSA_BF16 ? 8 : 4;
  if (p == nullptr || !aligned16(p)) return false;
  const long long strides[3] = {st.batch, st.token, st.head};
  const int sizes[3] = {b, s, H};
  for (int i = 0; i < 3; ++i)
    if (sizes[i] > 1 && (strides[i] < 0 || strides[i] % unit != 0)) return false;
  return true;
}

// ... and share no element: in the order of their strides, each spans the smaller ones.
bool valid_out(const void* p, csa_row_strides_t st, csa_dtype_t dt, int b, int s, int H, int d) {
  if (!valid_in(p, st, dt, b, s, H)) return false;
  long long strides[3] = {st.batch, st.token, st.head};
  int sizes[3] = {b, s, H};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (strides[j] > strides[j + 1]) {
        const long long x = strides[j];
        strides[j] = strides[j + 1];
        strides[j + 1] = x;
        const int n = sizes[j];
        sizes[j] = sizes[j + 1];
        sizes[j + 1] = n;
      }
  using Wide = __int128;
  Wide reach = d;
  for (int i = 0; i < 3; ++i) {
    if (sizes[i] < 2) continue;
    if (strides[i] < reach) return false;
    reach += (Wide)(sizes[i] - 1) * strides[i];
  }
  return true;
}

csa::RowStrides to_rows(csa_row_strides_t s) { return {s.batch, s.token, s.head}; }

bool same(csa_row_strides_t x, csa_row_strides_t y, int b, int s, int H) {
  return (b < 2 || x.batch == y.batch) && (s < 2 || x.token == y.token) &&
         (H < 2 || x.head == y.head);
}

// Sizes of a call on heads: INVALID_ARG, or UNSUPPORTED for sizes beyond the limits.
csa_status_t head_sizes(int b, int s, int H, int d) {
  if (b < 0 || s < 0 || H < 0 || d < 8 || d % 8 != 0) return CSA_ERR_INVALID_ARG;
  using Wide = __int128;
  if (d > csa::kMaxHeadWidth || (Wide)b * s * H > kMaxRowCount) return CSA_ERR_UNSUPPORTED;
  return CSA_OK;
}

bool valid_pos(const int32_t* pos, long long stride) {
  return pos == nullptr || (((uintptr_t)pos & 3u) == 0 && stride >= 0);
}

// csa_rope (norm kind 0) and csa_norm_rope.
csa_status_t rows_forward(const void* x, const csa_row_strides_t* xs, csa_dtype_t dt, int kind,
                          const float* weight, const float* bias, float eps, const int32_t* pos,
                          long long pos_stride, const csa_rope_t* rope, bool back, void* out,
                          const csa_row_strides_t* os, csa_dtype_t out_dt, int b, int s, int H,
                          int d, csa_stream_t stream) {
  if (!valid_dtype(dt) || !valid_dtype(out_dt)) return CSA_ERR_INVALID_ARG;
  const csa_status_t sizes = head_sizes(b, s, H, d);
  if (sizes == CSA_ERR_INVALID_ARG) return sizes;
  if (kind != csa::kNormNone && !valid_norm(kind, weight, bias, eps)) return CSA_ERR_INVALID_ARG;
  if (b == 0 || s == 0 || H == 0) return CSA_OK;
  if (!valid_rope(rope, d) || !valid_pos(pos, pos_stride) || xs == nullptr || os == nullptr)
    return CSA_ERR_INVALID_ARG;
  if (!valid_in(x, *xs, dt, b, s, H) || !valid_out(out, *os, out_dt, b, s, H, d))
    return CSA_ERR_INVALID_ARG;
  if (sizes != CSA_OK) return sizes;
  csa::RowsFwd a{};
  a.x = x;
  a.out = out;
  a.xs = to_rows(*xs);
  a.os = to_rows(*os);
  a.x_bf16 = dt == CSA_BF16;
  a.out_bf16 = out_dt == CSA_BF16;
  a.kind = kind;
  a.weight = weight;
  a.bias = bias;
  a.eps = eps;
  a.pos = pos;
  a.pos_stride = pos_stride;
  a.rope = rope_args(rope, back);
  a.b = b;
  a.s = s;
  a.H = H;
  a.d = d;
  a.in_place = x == out && dt == out_dt && same(*xs, *os, b, s, H);
  return from_cuda(csa::launch_rows_fwd(a, (cudaStream_t)stream));
}

csa_status_t rows_backward(csa::RowsBwd& a, void* workspace, size_t workspace_bytes,
                           long long rows, cudaStream_t st) {
  const size_t need = csa_norm_bwd_workspace_size(rows, a.d, a.dweight != nullptr, a.dbias != nullptr);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return CSA_ERR_WORKSPACE;
  a.parts = (float*)workspace;
  const int ctas = csa::rows_bwd_ctas(rows, a.d);
  const cudaError_t e = a.d > csa::kMaxHeadWidth ? csa::launch_norm_wide_bwd(a, ctas, st)
                                                 : csa::launch_rows_bwd(a, ctas, st);
  if (e != cudaSuccess || need == 0) return from_cuda(e);
  return from_cuda(csa::launch_sum_parts(a.parts, ctas, a.dweight, a.dbias, a.d, st));
}

// Without rows the sums are zero.
csa_status_t no_rows(float* dweight, float* dbias, int n, cudaStream_t st) {
  if (!aligned16(dweight) || !aligned16(dbias)) return CSA_ERR_INVALID_ARG;
  if (dweight == nullptr && dbias == nullptr) return CSA_OK;
  if (dweight == nullptr) return from_cuda(csa::launch_zero_f32(dbias, (size_t)n, st));
  return from_cuda(csa::launch_zero_f32_pair(dweight, (size_t)n, dbias, dbias ? (size_t)n : 0, st));
}

}  // namespace

extern "C" {

csa_status_t csa_norm(const void* x, long long x_stride, csa_dtype_t dt, int kind,
                      const float* weight, const float* bias, float eps, void* out,
                      long long out_stride, long long rows, int n, csa_stream_t stream) {
  if (!valid_dtype(dt) || !valid_norm(kind, weight, bias, eps)) return CSA_ERR_INVALID_ARG;
  if (rows < 0 || n < 8 || n % 8 != 0) return CSA_ERR_INVALID_ARG;
  if (rows == 0) return CSA_OK;
  const int few = rows > 1 ? 2 : 1;      // whether the stride counts
  const csa_row_strides_t xs = {0, 0, x_stride}, os = {0, 0, out_stride};
  if (!valid_in(x, xs, dt, 1, 1, few) || !valid_out(out, os, dt, 1, 1, few, n))
    return CSA_ERR_INVALID_ARG;
  if (n > csa::kMaxNormWidth || rows > kMaxRowCount) return CSA_ERR_UNSUPPORTED;
  csa::RowsFwd a{};
  a.x = x;
  a.out = out;
  a.xs = to_rows(xs);
  a.os = to_rows(os);
  a.x_bf16 = a.out_bf16 = dt == CSA_BF16;
  a.kind = kind;
  a.weight = weight;
  a.bias = bias;
  a.eps = eps;
  a.b = a.s = 1;
  a.H = (int)rows;
  a.d = n;
  const cudaStream_t st = (cudaStream_t)stream;
  return from_cuda(n > csa::kMaxHeadWidth ? csa::launch_norm_wide(a, st) : csa::launch_rows_fwd(a, st));
}

size_t csa_norm_bwd_workspace_size(long long rows, int n, int want_dweight, int want_dbias) {
  const int wanted = (want_dweight != 0) + (want_dbias != 0);
  if (rows < 1 || n < 8 || n > csa::kMaxNormWidth || wanted == 0) return 0;
  return (size_t)csa::rows_bwd_ctas(rows, n) * wanted * n * sizeof(float);
}

csa_status_t csa_norm_bwd(const void* x, long long x_stride, csa_dtype_t dt, int kind,
                          const float* weight, float eps, const void* dout,
                          long long dout_stride, csa_dtype_t dout_dt, void* dx,
                          long long dx_stride, csa_dtype_t dx_dt, float* dweight, float* dbias,
                          long long rows, int n, void* workspace, size_t workspace_bytes,
                          csa_stream_t stream) {
  if (!valid_dtype(dt) || !valid_dtype(dout_dt) || !valid_dtype(dx_dt) ||
      !valid_norm(kind, weight, nullptr, eps))
    return CSA_ERR_INVALID_ARG;
  if (rows < 0 || n < 8 || n % 8 != 0) return CSA_ERR_INVALID_ARG;
  const cudaStream_t st = (cudaStream_t)stream;
  if (rows == 0) return no_rows(dweight, dbias, n, st);
  const int few = rows > 1 ? 2 : 1;
  const csa_row_strides_t xs = {0, 0, x_stride}, gs = {0, 0, dout_stride}, ds = {0, 0, dx_stride};
  if (!valid_in(x, xs, dt, 1, 1, few) || !valid_in(dout, gs, dout_dt, 1, 1, few) ||
      !valid_out(dx, ds, dx_dt, 1, 1, few, n) || !aligned16(dweight) || !aligned16(dbias) ||
      !aligned16(workspace))
    return CSA_ERR_INVALID_ARG;
  if (n > csa::kMaxNormWidth || rows > kMaxRowCount) return CSA_ERR_UNSUPPORTED;
  csa::RowsBwd a{};
  a.x = x;
  a.dout = dout;
  a.dx = dx;
  a.xs = to_rows(xs);
  a.gs = to_rows(gs);
  a.ds = to_rows(ds);
  a.x_bf16 = dt == CSA_BF16;
  a.g_bf16 = dout_dt == CSA_BF16;
  a.dx_bf16 = dx_dt == CSA_BF16;
  a.kind = kind;
  a.weight = weight;
  a.eps = eps;
  a.dweight = dweight;
  a.dbias = dbias;
  a.b = a.s = 1;
  a.H = (int)rows;
  a.d = n;
  return rows_backward(a, workspace, workspace_bytes, rows, st);
}

csa_status_t csa_rope_freqs(int dim, double base, int scaling, double factor, double original_len,
                            double beta_fast, double beta_slow, double* freqs) {
  const auto positive = [](double v) { return std::isfinite(v) && v > 0; };
  if (freqs == nullptr || dim < 2 || dim % 2 != 0 || !positive(base)) return CSA_ERR_INVALID_ARG;
  if (scaling != CSA_ROPE_PLAIN && scaling != CSA_ROPE_LINEAR && scaling != CSA_ROPE_BY_PARTS)
    return CSA_ERR_INVALID_ARG;
  if (scaling != CSA_ROPE_PLAIN && !positive(factor)) return CSA_ERR_INVALID_ARG;
  double lo = 0, hi = 0;
  if (scaling == CSA_ROPE_BY_PARTS) {
    if (base == 1 || !positive(original_len) || !positive(beta_slow) || !positive(beta_fast) ||
        beta_fast < beta_slow)
      return CSA_ERR_INVALID_ARG;
    const double pi = 3.14159265358979323846;
    const auto pair = [&](double turns) {
      return dim * std::log(original_len / (2 * pi * turns)) / (2 * std::log(base));
    };
    const auto clamp = [&](double v) { return std::fmin(std::fmax(v, 0.0), dim - 1.0); };
    lo = clamp(std::floor(pair(beta_fast)));
    hi = clamp(std::ceil(pair(beta_slow)));
  }
  for (int i = 0; i < dim / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / dim);
    if (scaling == CSA_ROPE_PLAIN) {
      freqs[i] = f;
    } else if (scaling == CSA_ROPE_LINEAR) {
      freqs[i] = f / factor;
    } else {
      const double g = std::fmin(std::fmax((i - lo) / std::fmax(hi - lo, 0.001), 0.0), 1.0);
      freqs[i] = f * (1 - g) + f / factor * g;
    }
  }
  return CSA_OK;
}

csa_status_t csa_rope_turns(const double* freqs, int n, int64_t* turns) {
  if (freqs == nullptr || turns == nullptr || n < 1) return CSA_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i)
    if (!std::isfinite(freqs[i])) return CSA_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i) {
    const double t = freqs[i] / 6.28318530717958647692;
    const double part = std::ldexp(t - std::floor(t), 64);     // [0, 2^64], 2^64 when rounded up
    turns[i] = (int64_t)(part < 0x1p64 ? (uint64_t)part : 0u);
  }
  return CSA_OK;
}

csa_status_t csa_rope(const void* x, const csa_row_strides_t* x_strides, csa_dtype_t dt,
                      const int32_t* pos, long long pos_stride, const csa_rope_t* rope,
                      int inverse, void* out, const csa_row_strides_t* out_strides, int b, int s,
                      int H, int d, csa_stream_t stream) {
  return rows_forward(x, x_strides, dt, csa::kNormNone, nullptr, nullptr, 0.f, pos, pos_stride, rope,
                      inverse != 0, out, out_strides, dt, b, s, H, d, stream);
}

csa_status_t csa_rope_bwd(const void* dout, const csa_row_strides_t* dout_strides,
                          csa_dtype_t dout_dt, const int32_t* pos, long long pos_stride,
                          const csa_rope_t* rope, int inverse, void* dx,
                          const csa_row_strides_t* dx_strides, csa_dtype_t dx_dt, int b, int s,
                          int H, int d, csa_stream_t stream) {
  return rows_forward(dout, dout_strides, dout_dt, csa::kNormNone, nullptr, nullptr, 0.f, pos,
                      pos_stride, rope, inverse == 0, dx, dx_strides, dx_dt, b, s, H, d, stream);
}

csa_status_t csa_norm_rope(const void* x, const csa_row_strides_t* x_strides, csa_dtype_t dt,
                           int kind, const float* weight, const float* bias, float eps,
                           const int32_t* pos, long long pos_stride, const csa_rope_t* rope,
                           void* out, const csa_row_strides_t* out_strides, int b, int s, int H,
                           int d, csa_stream_t stream) {
  if (kind == csa::kNormNone) return CSA_ERR_INVALID_ARG;
  return rows_forward(x, x_strides, dt, kind, weight, bias, eps, pos, pos_stride, rope, false, out,
                      out_strides, dt, b, s, H, d, stream);
}

csa_status_t csa_norm_rope_bwd(const void* x, const csa_row_strides_t* x_strides, csa_dtype_t dt,
                               int kind, const float* weight, float eps, const int32_t* pos,
                               long long pos_stride, const csa_rope_t* rope, const void* dout,
                               const csa_row_strides_t* dout_strides, csa_dtype_t dout_dt,
                               void* dx, const csa_row_strides_t* dx_strides, csa_dtype_t dx_dt,
                               float* dweight, float* dbias, int b, int s, int H, int d,
                               void* workspace, size_t workspace_bytes, csa_stream_t stream) {
  if (!valid_dtype(dt) || !valid_dtype(dout_dt) || !valid_dtype(dx_dt) ||
      !valid_norm(kind, weight, nullptr, eps))
    return CSA_ERR_INVALID_ARG;
  const csa_status_t sizes = head_sizes(b, s, H, d);
  if (sizes == CSA_ERR_INVALID_ARG) return sizes;
  const cudaStream_t st = (cudaStream_t)stream;
  if (b == 0 || s == 0 || H == 0) return no_rows(dweight, dbias, d, st);
  if (!valid_rope(rope, d) || !valid_pos(pos, pos_stride) || x_strides == nullptr ||
      dout_strides == nullptr || dx_strides == nullptr)
    return CSA_ERR_INVALID_ARG;
  if (!valid_in(x, *x_strides, dt, b, s, H) || !valid_in(dout, *dout_strides, dout_dt, b, s, H) ||
      !valid_out(dx, *dx_strides, dx_dt, b, s, H, d) || !aligned16(dweight) || !aligned16(dbias) ||
      !aligned16(workspace))
    return CSA_ERR_INVALID_ARG;
  if (sizes != CSA_OK) return sizes;
  csa::RowsBwd a{};
  a.x = x;
  a.dout = dout;
  a.dx = dx;
  a.xs = to_rows(*x_strides);
  a.gs = to_rows(*dout_strides);
  a.ds = to_rows(*dx_strides);
  a.x_bf16 = dt == CSA_BF16;
  a.g_bf16 = dout_dt == CSA_BF16;
  a.dx_bf16 = dx_dt == CSA_BF16;
  a.kind = kind;
  a.weight = weight;
  a.eps = eps;
  a.pos = pos;
  a.pos_stride = pos_stride;
  a.rope = rope_args(rope, true);
  a.dweight = dweight;
  a.dbias = dbias;
  a.b = b;
  a.s = s;
  a.H = H;
  a.d = d;
  return rows_backward(a, workspace, workspace_bytes, (long long)b * s * H, st);
}

csa_status_t csa_compress_decode(const void* kv, long long kv_batch_stride,
                                 long long kv_row_stride, const void* score,
                                 long long score_batch_stride, long long score_row_stride,
                                 int score_width, void* kv_ring, void* score_ring, int ring_rows,
                                 const int32_t* seq_lens, int kind, const float* weight,
                                 const float* bias, float eps, const csa_rope_t* rope, void* out,
                                 long long out_stride, int32_t* first, int32_t* counts, int b,
                                 int s_q, int d, int ratio, int coff, csa_dtype_t dt,
                                 csa_stream_t stream) {
  if (!valid_dtype(dt) || b < 0 || s_q < 0 || d < 8 || d % 8 != 0 || ratio < 1 || coff < 1)
    return CSA_ERR_INVALID_ARG;
  if (score_width != 1 && score_width != d) return CSA_ERR_INVALID_ARG;
  if (ring_rows < (long long)coff * ratio) return CSA_ERR_INVALID_ARG;
  if (kind != csa::kNormNone && !valid_norm(kind, weight, bias, eps)) return CSA_ERR_INVALID_ARG;
  if (rope != nullptr && !valid_rope(rope, d)) return CSA_ERR_INVALID_ARG;
  if (b == 0 || s_q == 0) return CSA_OK;
  if (kv == nullptr || score == nullptr || kv_ring == nullptr || score_ring == nullptr ||
      seq_lens == nullptr || out == nullptr || first == nullptr || counts == nullptr)
    return CSA_ERR_INVALID_ARG;
  const int blocks = (s_q - 1) / ratio + 1;
  const csa_row_strides_t ks = {kv_batch_stride, kv_row_stride, 0};
  const csa_row_strides_t ss = {score_batch_stride, score_row_stride, 0};
  const csa_row_strides_t os = {out_stride, d, 0};
  if (!aligned16(kv_ring) || !valid_in(kv, ks, dt, b, s_q, 1) ||
      !valid_out(out, os, dt, b, blocks, 1, d))
    return CSA_ERR_INVALID_ARG;
  if (score_width != 1) {
    if (!aligned16(score_ring) || !valid_in(score, ss, dt, b, s_q, 1)) return CSA_ERR_INVALID_ARG;
  } else if (((uintptr_t)score | (uintptr_t)score_ring) % (dt == CSA_BF16 ? 2 : 4) != 0 ||
             (s_q > 1 && score_row_stride < 0) || (b > 1 && score_batch_stride < 0)) {
    return CSA_ERR_INVALID_ARG;
  }
  if (d > csa::kMaxHeadWidth || coff > 2 || b > 65535 || (long long)coff * ratio > csa::kMaxSlots ||
      ring_rows > csa::kMaxSlots)
    return CSA_ERR_UNSUPPORTED;
  csa::CompressDecodeArgs a{};
  a.kv = kv;
  a.score = score;
  a.kv_bs = kv_batch_stride;
  a.kv_rs = kv_row_stride;
  a.sc_bs = score_batch_stride;
  a.sc_rs = score_row_stride;
  a.sw = score_width;
  a.kv_ring = kv_ring;
  a.score_ring = score_ring;
  a.R = ring_rows;
  a.seq_lens = seq_lens;
  a.kind = kind;
  a.weight = weight;
  a.bias = bias;
  a.eps = eps;
  a.rope = rope_args(rope, false);
  a.out = out;
  a.out_bs = out_stride;
  a.first = first;
  a.counts = counts;
  a.b = b;
  a.s_q = s_q;
  a.d = d;
  a.ratio = ratio;
  a.coff = coff;
  a.status = csa::device_status_word();
  return from_cuda(csa::launch_compress_decode(a, dt == CSA_BF16, (cudaStream_t)stream));
}

}  // extern "C"
