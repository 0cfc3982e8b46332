/*
 * csa_serve.h - C ABI of the serving calls of a Compressed Sparse Attention
 * layer: single-token (decode) steps over a paged cache held in 4 or 8 bits.
 *
 *   csa_cache_write          quantise rows into the cache as they are appended
 *   csa_cache_read           the rows of a range of positions, as bf16 or fp32
 *   csa_indexer_topk_decode  lightning-indexer scores of the newest tokens
 *                            against the cached index keys, exact top-k
 *   csa_attn_decode          sparse MQA of the newest tokens over the cached
 *                            window rows, the selected compressed rows and the
 *                            sink; returns O and LSE
 *
 * A decode step of one layer: csa_cache_write of the new tokens' raw rows;
 * where a token completes a block of `ratio` tokens, csa_compress of the block
 * and csa_cache_write of its pooled row and of its index key;
 * csa_indexer_topk_decode; csa_attn_decode.  A layer of csa_compress_overlap
 * with coff 2 gives it the last two blocks and keeps the second entry.  A layer
 * of csa_compress_norm_rope cannot pool its blocks as they complete: that call
 * turns entry j of the rows it is given to position (j + 1) * ratio - 1 of those
 * rows, so a block pooled alone is turned as block 0; its rows go into the cache
 * from calls on the whole sequence.  Conventions (ownership, streams,
 * errors, status codes, dtypes) are those of csa.h: the caller owns every
 * buffer, no call synchronizes or allocates, argument errors are found before
 * any CUDA call, and conditions met on the device are recorded in the status
 * word that csa_get_device_status() reads.
 *
 * Cache.  `cache` is n_pages pages of csa_cache_page_bytes(page_size, d, bits)
 * bytes each, packed.  A page holds page_size rows of d channels: first
 * page_size x (d * bits / 8) bytes of codes, then page_size x (d / 32) scale
 * bytes.  A group of 32 consecutive channels has one scale byte s and stands
 * for code * 2^(s - 127):
 *   bits 4: e2m1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), two
 *           to a byte, channel 2i in the low half of byte i
 *   bits 8: e4m3 codes (largest 448)
 * Every value the cache can hold is a bf16 value.
 *
 * Positions.  Each of the b sequences has a row of P page ids in a page table
 * [b, P] (int32); its position p (p >= 0) lies in slot r = p mod (P *
 * page_size), that is in row r mod page_size of page table[r / page_size].
 * With P * page_size at least the sequence's length the cache keeps every
 * row; with fewer pages it is a ring that keeps the newest rows, which is all
 * that the raw rows of a window need.  Page ids that a call does not need are
 * not looked at.  An id outside [0, n_pages) that it does need is never
 * followed: the row is skipped (write), returned as zeros (read), scored as a
 * zero key (indexer) or masked (attention), and CSA_ERR_DEVICE_CHECK is
 * recorded (site 0x71).  A sequence length or count outside its range is
 * clamped and recorded (site 0x72).  A bounded wait that gives up records
 * CSA_ERR_TIMEOUT (site 0x73 attention, 0x74 indexer); the call's outputs are
 * then unspecified.
 *
 * Limits: 32 <= d <= 512 and d % 32 == 0; page_size a multiple of 16, at most
 * 32768; bits 4 or 8; b at most 65535 and P * page_size at most 2^24
 * (UNSUPPORTED above); positions below 2^31.  NaN and infinite inputs give
 * unspecified values in their own rows, and in the results of the queries that
 * see those; no other result changes, and chosen blocks are always visible ones.
 */
#ifndef CSA_SERVE_H_
#define CSA_SERVE_H_

#include "csa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of one page; 0 for sizes outside the limits. */
size_t csa_cache_page_bytes(int page_size, int d, int bits);

/*
 * csa_cache_write - quantise rows into the cache.
 *
 * Row i < counts[s] of sequence s goes to position pos0[s] + i.  Per group of
 * 32 channels the scale is the smallest power of two 2^e with
 * max|x| <= 2^e * 6 (bits 4) or 2^e * 448 (bits 8), within -110 <= e <= 125
 * (bits 4) or 119 (bits 8), and the codes are x * 2^-e rounded to the nearest
 * code, ties to even, the largest beyond it.  When more
 * rows than the table has slots are given, the last P * page_size are kept.
 * Rows i >= counts[s] are not read, and no other slot is touched.  A page may
 * be written for one sequence only in a call, and appear once in its row of
 * the table; otherwise the shared slots' bytes are unspecified.
 *
 *   x       in   [b, s, d] of dt; strides in elements, rows contiguous
 *   table   in   [b, P] int32
 *   pos0    in   [b] int32, first position (>= 0)
 *   counts  in   [b] int32 in [0, s]; NULL = s rows of every sequence
 *   cache   out  written slots only
 * Errors: INVALID_ARG for null pointers, x or cache not 16-byte aligned, x
 * strides that are not multiples of 16 bytes, sizes outside the limits.
 * s == 0 or b == 0 is a no-op.
 */
csa_status_t csa_cache_write(const void* x, long long x_batch_stride, long long x_row_stride,
                             csa_dtype_t dt, const int32_t* table, const int32_t* pos0,
                             const int32_t* counts, void* cache, int b, int s, int d, int P,
                             int n_pages, int page_size, int bits, csa_stream_t stream);

/*
 * csa_cache_read - the rows at positions pos0[s] .. pos0[s] + counts[s] - 1,
 * as the values their codes stand for (exact in bf16 and in fp32).
 * Rows i >= counts[s] of out are left as they were.  s must not exceed
 * P * page_size.  A position that the ring no longer keeps reads as the newer
 * one that took its slot.
 *   out  out  [b, s, d] of dt; strides in elements, rows contiguous; rows may
 *             not overlap
 * Other arguments and errors as csa_cache_write; also INVALID_ARG for strides
 * at which two rows of out share an element.
 */
csa_status_t csa_cache_read(const void* cache, const int32_t* table, const int32_t* pos0,
                            const int32_t* counts, void* out, long long out_batch_stride,
                            long long out_row_stride, csa_dtype_t dt, int b, int s, int d, int P,
                            int n_pages, int page_size, int bits, csa_stream_t stream);

/*
 * csa_indexer_topk_decode - indexer scores and exact top-k of the newest s_q
 * tokens of each sequence.
 *
 * Sequence s has seq_lens[s] tokens, the newest s_q of which are queries:
 * query i is at t = seq_lens[s] - s_q + i and sees the blocks
 * j < vis(t) = (t + 1) / ratio (none when t < 0).  With k_j the cached index
 * key at position j,
 *   I[j] = sum_h w[h] * ReLU(q_I[h] . k_j),
 * and topk_idx receives the min(topk, vis) blocks with the largest I, ties to
 * the lower block, in ascending order, then -1.  The set is that of the exact
 * scores: blocks whose fp32 score lies within the fp32 error of the topk-th
 * are scored again at twice fp32's precision.  The choice therefore depends
 * on the row's own inputs alone, not on the batch.  This holds while no
 * |q_I[h]| |k_j| and no sum of |w[h]| |q_I[h]| |k_j| reaches 2^126 and no key
 * has a value above 2^60; a row beyond that is left to the fp32 scores, in
 * which sums that overflow rank as infinite or, where they are NaN, last.
 *
 *   q_I        in   [b, s_q, H_I, d_I] of dt      w  in  [b, s_q, H_I] fp32
 *   table      in   [b, P] page table of the index keys (no ring: P *
 *                   page_size slots, block j in slot j)
 *   seq_lens   in   [b] int32
 *   topk_idx   out  [b, s_q, topk] int32
 *   workspace       csa_indexer_topk_decode_workspace_size bytes, 16-byte
 *                   aligned, used by one call at a time
 * Errors: INVALID_ARG for null or misaligned (16 bytes: q_I, cache, w,
 * workspace) pointers and sizes outside the limits; UNSUPPORTED for
 * d_I > 256, H_I > 128, b * s_q > 65535; WORKSPACE when too small.
 *
 * bf16 queries of d_I 64 or 128 take the tensor cores; fp32 queries and other
 * widths are scored on CUDA cores (16 sequences of up to 131072 tokens: 197 us
 * instead of 41).
 */
size_t csa_indexer_topk_decode_workspace_size(int b, int s_q, int H_I, int d_I, int slots);
csa_status_t csa_indexer_topk_decode(const void* q_I, const void* cache, const int32_t* table,
                                     const float* w, const int32_t* seq_lens, int32_t* topk_idx,
                                     int b, int s_q, int H_I, int d_I, int ratio, int topk, int P,
                                     int n_pages, int page_size, int bits, csa_dtype_t dt,
                                     void* workspace, size_t workspace_bytes,
                                     csa_stream_t stream);

/*
 * csa_attn_decode - sparse MQA of the newest s_q tokens of each sequence.
 *
 * Query i of sequence s (t as above) attends, in one softmax, to the raw rows
 * t - window + 1 .. t (those >= 0), to the compressed rows j of its idx row
 * with 0 <= j < vis(t) (a repeated entry is a repeated term; idx NULL: every
 * j < vis(t)) and to the sink, which enters only the denominator.  Keys and
 * values are the same cached rows.  lse is the natural log of the denominator,
 * sink included.  A query with no row to attend to (t < 0) gets o = 0 and
 * lse = sink (-inf without one).
 *
 * Arithmetic: fp32 queries, and widths other than those below, are computed in
 * fp32 throughout, on CUDA cores (128 queries of 64 heads x 512 over 1152 rows:
 * 1.9 ms instead of 46 us).  bf16 queries of d 64, 128, 256 or 512 take the tensor cores:
 * logits, maxima, sums and o are accumulated in fp32, and each probability is
 * rounded to bf16 (2^-8 of itself) for its product with the row.  o is divided
 * by the sum of the rounded probabilities, so its weights add up to the rows'
 * share of the denominator; lse has the sum of the unrounded ones.
 *
 *   q          in   [b, s_q, H, d] of dt           sink  in  [H] fp32 or NULL
 *   raw_table  in   [b, P_raw] page table of the raw rows (a ring:
 *                   P_raw * page_size >= window + s_q - 1)
 *   cmp_table  in   [b, P_cmp] page table of the compressed rows (row j in
 *                   slot j); both tables index the same cache
 *   idx        in   [b, s_q, K] int32 or NULL
 *   o          out  [b, s_q, H, d] of dt           lse   out [b, s_q, H] fp32
 *   workspace       csa_attn_decode_workspace_size bytes (K, or
 *                   P_cmp * page_size when idx is NULL, as its last argument),
 *                   16-byte aligned, used by one call at a time.  The size is
 *                   that of the kernels of either dt, and a call needs it
 *                   whichever of them it takes; NULL where it is 0.  It does
 *                   not grow with b, s_q or the rows: fewer queries are cut
 *                   into more parts.  A workspace for calls of several sizes
 *                   has the largest of theirs, or 2880 * (4 d + 8) + 16 bytes,
 *                   which no size exceeds.
 * Errors: INVALID_ARG for null pointers (P_cmp == 0 allows a null cmp_table,
 * K must then be 0), misaligned q, cache, o, workspace, sizes outside the
 * limits, a ring smaller than the windows, a scale that is not finite; UNSUPPORTED
 * for H > 128 or b * s_q > 65535; WORKSPACE when too small.
 */
size_t csa_attn_decode_workspace_size(int b, int s_q, int H, int d, int window, int cmp_rows);
csa_status_t csa_attn_decode(const void* q, const void* cache, const int32_t* raw_table,
                             const int32_t* cmp_table, const int32_t* idx, const float* sink,
                             const int32_t* seq_lens, float scale, void* o, float* lse, int b,
                             int s_q, int H, int d, int ratio, int window, int K, int P_raw,
                             int P_cmp, int n_pages, int page_size, int bits, csa_dtype_t dt,
                             void* workspace, size_t workspace_bytes, csa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* CSA_SERVE_H_ */
