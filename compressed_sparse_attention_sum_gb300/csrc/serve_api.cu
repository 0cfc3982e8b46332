// C ABI entry points of the serving calls (include/csa_serve.h): argument
// validation and dispatch.  Every check runs before the first CUDA call, so a
// rejected call leaves the device untouched.
#include <cmath>
#include <cstdint>

#include "../../include/csa_serve.h"
#include "attn_decode.h"
#include "cache_format.cuh"
#include "indexer_decode.h"
#include "indexer_host.h"

namespace csa {
int* device_status_word();
cudaError_t launch_cache_write(const void* x, long long x_bs, long long x_rs, bool bf16,
                               const int32_t* table, const int32_t* pos0, const int32_t* counts,
                               void* cache, int b, int s, int d, int P, int n_pages,
                               int page_size, int bits, int* status, cudaStream_t st);
cudaError_t launch_cache_read(const void* cache, const int32_t* table, const int32_t* pos0,
                              const int32_t* counts, void* out, long long o_bs, long long o_rs,
                              bool bf16, int b, int s, int d, int P, int n_pages, int page_size,
                              int bits, int* status, cudaStream_t st);
}  // namespace csa

namespace {

using csa::aligned16;
using csa::kMaxSlots;

constexpr int kMaxDecodeH = 128;
constexpr int kMaxRows = 65535;           // queries of one call

csa_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? CSA_OK : CSA_ERR_CUDA; }

bool valid_dtype(csa_dtype_t dt) { return dt == CSA_FP32 || dt == CSA_BF16; }

bool valid_format(int page_size, int d, int bits) {
  return (bits == 4 || bits == 8) && page_size >= 16 && page_size % 16 == 0 &&
         page_size <= csa::kMaxPageSize && d >= 32 && d <= 512 && d % 32 == 0;
}

// P pages of page_size rows: slots are counted in 31 bits.
bool valid_table(int P, int page_size) {
  return P >= 1 && (long long)P * page_size <= 0x7fffffffll;
}

// Rows [b, s, d] with contiguous channels: every row on a 16-byte boundary.
bool valid_rows(const void* p, long long batch_stride, long long row_stride, csa_dtype_t dt,
                int d, int s, int b) {
  const long long esz = dt == CSA_BF16 ? 2 : 4;
  if (!aligned16(p) || (batch_stride * esz) % 16 != 0 || (row_stride * esz) % 16 != 0) return false;
  if (s > 1 && row_stride < d) return false;
  return b == 1 || batch_stride >= 0;
}

// Whether rows [b, s] of d elements at these strides share elements (a row stride
// below d is refused already where s > 1).  Only two batches can, in rows i and
// i + m whose distance is within d of a multiple of the row stride.
bool rows_overlap(long long bs, long long rs, int d, int s, int b) {
  if (b < 2) return false;
  if (bs < d) return true;
  if (s < 2) return false;
  using Wide = __int128;
  const Wide last = (Wide)(s - 1) * rs;
  if (bs >= last + d || rs >= (Wide)(b - 1) * bs + d) return false;
  for (int m = 1; m < b && m * (Wide)bs < last + d; ++m) {
    const Wide at = m * (Wide)bs, below = at / rs * rs, above = below + rs;
    if (at - below < d && below <= last && below > 0) return true;
    if (above - at < d && above <= last) return true;
  }
  return false;
}

csa_status_t check_cache_rows(const void* x, long long bs, long long rs, csa_dtype_t dt,
                              const int32_t* table, const int32_t* pos0, const void* cache, int b,
                              int s, int d, int P, int n_pages, int page_size, int bits) {
  if (!valid_dtype(dt) || !valid_format(page_size, d, bits)) return CSA_ERR_INVALID_ARG;
  if (b < 0 || s < 0) return CSA_ERR_INVALID_ARG;
  if (b == 0 || s == 0) return CSA_OK;
  if (x == nullptr || table == nullptr || pos0 == nullptr || cache == nullptr)
    return CSA_ERR_INVALID_ARG;
  if (!aligned16(cache) || !valid_rows(x, bs, rs, dt, d, s, b)) return CSA_ERR_INVALID_ARG;
  if (n_pages < 1 || !valid_table(P, page_size)) return CSA_ERR_INVALID_ARG;
  if (b > kMaxRows || (long long)P * page_size > kMaxSlots) return CSA_ERR_UNSUPPORTED;
  return CSA_OK;
}

bool decode_sizes(int b, int s_q, int H, int d, int window, long long cmp_rows) {
  return b >= 1 && s_q >= 1 && H >= 1 && d >= 32 && d % 32 == 0 && window >= 1 && cmp_rows >= 0;
}

// Partial results of a call whose queries are cut into parts: rows * parts * H of
// them.  On CUDA cores rows * parts * ceil(H / 8) <= 304, so at most 2432; on the
// tensor cores rows * H <= 64 c for c CTAs a split and parts <= (144 / c + 3) / 4
// with c <= 12, so at most 2880: the bound that csa_serve.h gives.
size_t attn_decode_layout(csa::AttnDecodeArgs* a, int parts, unsigned char* ws) {
  a->parts = parts;
  if (parts == 1) return 0;
  const size_t n = (size_t)a->b * a->s_q * parts * a->H;
  a->part_ml = reinterpret_cast<float2*>(ws);
  const size_t at = (n * sizeof(float2) + 15) / 16 * 16;
  a->part_o = reinterpret_cast<float*>(ws + at);
  return at + n * a->d * sizeof(float);
}

}  // namespace

extern "C" {

size_t csa_cache_page_bytes(int page_size, int d, int bits) {
  if (!valid_format(page_size, d, bits)) return 0;
  return (size_t)csa::cache_shape(page_size, 1, d, bits).page_bytes;
}

csa_status_t csa_cache_write(const void* x, long long x_batch_stride, long long x_row_stride,
                             csa_dtype_t dt, const int32_t* table, const int32_t* pos0,
                             const int32_t* counts, void* cache, int b, int s, int d, int P,
                             int n_pages, int page_size, int bits, csa_stream_t stream) {
  const csa_status_t st = check_cache_rows(x, x_batch_stride, x_row_stride, dt, table, pos0, cache,
                                           b, s, d, P, n_pages, page_size, bits);
  if (st != CSA_OK || b == 0 || s == 0) return st;
  return from_cuda(csa::launch_cache_write(
      x, x_batch_stride, x_row_stride, dt == CSA_BF16, table, pos0, counts, cache, b, s, d, P,
      n_pages, page_size, bits, csa::device_status_word(), (cudaStream_t)stream));
}

csa_status_t csa_cache_read(const void* cache, const int32_t* table, const int32_t* pos0,
                            const int32_t* counts, void* out, long long out_batch_stride,
                            long long out_row_stride, csa_dtype_t dt, int b, int s, int d, int P,
                            int n_pages, int page_size, int bits, csa_stream_t stream) {
  const csa_status_t st = check_cache_rows(out, out_batch_stride, out_row_stride, dt, table, pos0,
                                           cache, b, s, d, P, n_pages, page_size, bits);
  if (st == CSA_ERR_INVALID_ARG || b == 0 || s == 0) return st;
  if (b <= kMaxRows && rows_overlap(out_batch_stride, out_row_stride, d, s, b))
    return CSA_ERR_INVALID_ARG;
  if (st != CSA_OK) return st;
  if (s > (long long)P * page_size) return CSA_ERR_INVALID_ARG;
  return from_cuda(csa::launch_cache_read(
      cache, table, pos0, counts, out, out_batch_stride, out_row_stride, dt == CSA_BF16, b, s, d,
      P, n_pages, page_size, bits, csa::device_status_word(), (cudaStream_t)stream));
}

size_t csa_indexer_topk_decode_workspace_size(int b, int s_q, int H_I, int d_I, int slots) {
  if (b < 1 || s_q < 1 || H_I < 1 || d_I < 32 || slots < 1) return 0;
  csa::IndexDecodeArgs a{};
  a.b = b;
  a.s_q = s_q;
  a.slots = slots;
  a.tiles = (slots + csa::kIdxTile - 1) / csa::kIdxTile;
  return csa::index_decode_layout(&a, nullptr);
}

csa_status_t csa_indexer_topk_decode(const void* q_I, const void* cache, const int32_t* table,
                                     const float* w, const int32_t* seq_lens, int32_t* topk_idx,
                                     int b, int s_q, int H_I, int d_I, int ratio, int topk, int P,
                                     int n_pages, int page_size, int bits, csa_dtype_t dt,
                                     void* workspace, size_t workspace_bytes,
                                     csa_stream_t stream) {
  if (!valid_dtype(dt) || !valid_format(page_size, d_I, bits)) return CSA_ERR_INVALID_ARG;
  if (q_I == nullptr || cache == nullptr || table == nullptr || w == nullptr ||
      seq_lens == nullptr || topk_idx == nullptr || workspace == nullptr)
    return CSA_ERR_INVALID_ARG;
  if (!aligned16(q_I) || !aligned16(cache) || !aligned16(w) || !aligned16(workspace))
    return CSA_ERR_INVALID_ARG;
  if (b < 1 || s_q < 1 || H_I < 1 || ratio < 1 || topk < 1 || n_pages < 1 ||
      !valid_table(P, page_size))
    return CSA_ERR_INVALID_ARG;
  const long long slots = (long long)P * page_size;
  if (d_I > csa::kMaxDecodeDI || H_I > csa::kMaxDecodeHI || (long long)b * s_q > kMaxRows ||
      slots > kMaxSlots || topk > kMaxSlots)
    return CSA_ERR_UNSUPPORTED;
  csa::IndexDecodeArgs a{};
  a.q = q_I;
  a.cache = (const uint8_t*)cache;
  a.table = table;
  a.w = w;
  a.seq_lens = seq_lens;
  a.out = topk_idx;
  a.b = b;
  a.s_q = s_q;
  a.H = H_I;
  a.d = d_I;
  a.ratio = ratio;
  a.topk = topk;
  a.P = P;
  a.slots = (int)slots;
  a.tiles = (a.slots + csa::kIdxTile - 1) / csa::kIdxTile;
  a.cs = csa::cache_shape(page_size, n_pages, d_I, bits);
  if (workspace_bytes < csa::index_decode_layout(&a, (unsigned char*)workspace))
    return CSA_ERR_WORKSPACE;
  a.status = csa::device_status_word();
  const cudaStream_t s = (cudaStream_t)stream;
  const bool tc = dt == CSA_BF16 && csa::index_decode_tc_supported(H_I, d_I);
  // see indexer_select.cu: fp32 sums on the tensor cores and on CUDA cores
  a.err = (tc ? (float)(11 * d_I / 16 + H_I / 4 + 8) : (float)(d_I + H_I + 16)) * 0x1p-24f;
  const cudaError_t e = tc ? csa::launch_index_scores_tc(a, bits, s)
                           : csa::launch_index_scores_simt(a, dt == CSA_BF16, bits, s);
  if (e != cudaSuccess) return CSA_ERR_CUDA;
  return from_cuda(csa::launch_index_select(a, dt == CSA_BF16, bits, s));
}

size_t csa_attn_decode_workspace_size(int b, int s_q, int H, int d, int window, int cmp_rows) {
  if (!decode_sizes(b, s_q, H, d, window, cmp_rows)) return 0;
  csa::AttnDecodeArgs a{};
  a.b = b;
  a.s_q = s_q;
  a.H = H;
  a.d = d;
  // the largest over the kernels and over calls with and without an index list
  int parts = csa::decode_plan_simt(b, s_q, H, window, cmp_rows).parts;
  if (csa::decode_tc_width(d)) {
    for (const bool dense : {false, true}) {
      const int t = csa::decode_plan_tc(b, s_q, H, window, dense ? 0 : cmp_rows, dense, cmp_rows).parts;
      parts = t > parts ? t : parts;
    }
  }
  return attn_decode_layout(&a, parts, nullptr);
}

csa_status_t csa_attn_decode(const void* q, const void* cache, const int32_t* raw_table,
                             const int32_t* cmp_table, const int32_t* idx, const float* sink,
                             const int32_t* seq_lens, float scale, void* o, float* lse, int b,
                             int s_q, int H, int d, int ratio, int window, int K, int P_raw,
                             int P_cmp, int n_pages, int page_size, int bits, csa_dtype_t dt,
                             void* workspace, size_t workspace_bytes, csa_stream_t stream) {
  if (!valid_dtype(dt) || !valid_format(page_size, d, bits)) return CSA_ERR_INVALID_ARG;
  if (q == nullptr || cache == nullptr || raw_table == nullptr || seq_lens == nullptr ||
      o == nullptr || lse == nullptr)
    return CSA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(cache) || !aligned16(o) || !aligned16(workspace))
    return CSA_ERR_INVALID_ARG;
  if (b < 1 || s_q < 1 || H < 1 || ratio < 1 || window < 1 || n_pages < 1 || K < 0 || P_cmp < 0 ||
      !valid_table(P_raw, page_size) || (P_cmp > 0 && !valid_table(P_cmp, page_size)))
    return CSA_ERR_INVALID_ARG;
  if ((idx == nullptr) != (K == 0) || (P_cmp > 0 && cmp_table == nullptr) ||
      (K > 0 && P_cmp == 0))
    return CSA_ERR_INVALID_ARG;
  if ((long long)P_raw * page_size < (long long)window + s_q - 1) return CSA_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return CSA_ERR_INVALID_ARG;
  const long long cmp_rows = K > 0 ? K : (long long)P_cmp * page_size;
  if (H > kMaxDecodeH || (long long)b * s_q > kMaxRows || K > kMaxSlots ||
      (long long)P_raw * page_size > kMaxSlots || (long long)P_cmp * page_size > kMaxSlots)
    return CSA_ERR_UNSUPPORTED;
  csa::AttnDecodeArgs a{};
  a.q = q;
  a.cache = (const uint8_t*)cache;
  a.raw_table = raw_table;
  a.cmp_table = cmp_table;
  a.idx = idx;
  a.sink = sink;
  a.seq_lens = seq_lens;
  a.scale = scale;
  a.o = o;
  a.lse = lse;
  a.b = b;
  a.s_q = s_q;
  a.H = H;
  a.d = d;
  a.ratio = ratio;
  a.window = window;
  a.K = K;
  a.P_raw = P_raw;
  a.P_cmp = P_cmp;
  a.cs = csa::cache_shape(page_size, n_pages, d, bits);
  const bool tc = dt == CSA_BF16 && csa::decode_tc_width(d);
  const csa::DecodePlan plan =
      tc ? csa::decode_plan_tc(b, s_q, H, window, K, idx == nullptr,
                               (long long)P_cmp * page_size)
         : csa::decode_plan_simt(b, s_q, H, window, cmp_rows);
  const size_t need = csa_attn_decode_workspace_size(b, s_q, H, d, window, (int)cmp_rows);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return CSA_ERR_WORKSPACE;
  attn_decode_layout(&a, plan.parts, (unsigned char*)workspace);
  a.status = csa::device_status_word();
  const cudaStream_t s = (cudaStream_t)stream;
  return from_cuda(tc ? csa::launch_attn_decode_tc(a, plan, bits, s)
                      : csa::launch_attn_decode_simt(a, dt == CSA_BF16, bits, s));
}

}  // extern "C"
