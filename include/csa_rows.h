/*
 * csa_rows.h - C ABI of the calls that make the rows a Compressed Sparse
 * Attention layer works on: norms and rotary positions of queries, raw KV
 * rows and index keys, in training, prompts and single-token steps.
 *
 *   csa_norm, csa_norm_bwd            layer or RMS norm of rows; gradient with
 *                                     the sums for the weight and the bias
 *   csa_rope, csa_rope_bwd            rotary positions of rows [b, s, H, d]
 *   csa_norm_rope, csa_norm_rope_bwd  the norm of each head's row followed by
 *                                     the rotation, in one pass
 *   csa_compress_decode               the compressed rows of the blocks that the
 *                                     newest tokens of a sequence complete:
 *                                     pooled, normalised and turned
 *
 * csa_compress_norm_rope (csa.h) pools, normalises and turns whole sequences.
 *
 * Conventions (ownership, streams, errors, status codes, dtypes) are those of
 * csa.h: the caller owns every buffer, no call synchronizes or allocates, and
 * argument errors are found before any CUDA call.  A call without rows is a
 * no-op that looks at no pointer.  All arithmetic is fp32; an output is
 * rounded once to its dtype.
 *
 * Rows.  Channels are contiguous; strides are in elements, not negative, and
 * multiples of 16 bytes, as are pointers; widths are multiples of 8.  Inputs
 * may share elements (a stride of 0 broadcasts).  Outputs may not: in the
 * order of their strides, each stride has to span what the smaller ones reach
 * (INVALID_ARG otherwise).  An output may be its input (same pointer, strides
 * and dtype; of the two inputs of a backward call, either); other overlaps of
 * inputs and outputs give unspecified values.  Gradients come for every row: those
 * of rows that share an input's elements are the caller's to add.
 *
 * NaN and infinite inputs give unspecified values in their own row, and in the
 * weight and bias gradients of the channels that they reach; channels that a
 * rotation leaves out keep their values (infinities and signed zeros among them; a NaN
 * stays a NaN, in bf16 perhaps another one).  Sums of squares are fp32: rows whose
 * magnitudes pass 2^63 / sqrt(width) overflow, and with eps 0 rows whose spread
 * is below 2^-62 underflow.
 */
#ifndef CSA_ROWS_H_
#define CSA_ROWS_H_

#include "csa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* CSA_NORM_RMS: m = 0.  CSA_NORM_LAYER: m = mean(x).  In both
 * y = (x - m) / sqrt(mean((x - m)^2) + eps) * weight + bias. */
typedef enum { CSA_NORM_RMS = 1, CSA_NORM_LAYER = 2 } csa_norm_kind_t;

/*
 * csa_norm - norm of rows of n channels.
 *
 *   x       in   [rows, n] of dt, row stride x_stride
 *   weight  in   [n] fp32, 16-byte aligned; NULL = ones
 *   bias    in   [n] fp32, 16-byte aligned; NULL = zeros
 *   eps          >= 0, finite (0: a row without spread has no norm: NaN)
 *   out     out  [rows, n] of dt, row stride out_stride
 * Errors: INVALID_ARG for null or misaligned pointers, n % 8 != 0, n < 8,
 * strides (above), an unknown kind or dtype, a bad eps; UNSUPPORTED for n >
 * 32768 or rows > 2^30.
 */
csa_status_t csa_norm(const void* x, long long x_stride, csa_dtype_t dt, int kind,
                      const float* weight, const float* bias, float eps, void* out,
                      long long out_stride, long long rows, int n, csa_stream_t stream);

/*
 * csa_norm_bwd - gradient of csa_norm.
 *
 * With xh = (x - m) / sqrt(...) recomputed from x and g = dout * weight:
 *   dx      = (g - mean(g) - xh * mean(g * xh)) / sqrt(...)   (RMS: no mean(g))
 *   dweight = sum over rows of dout * xh
 *   dbias   = sum over rows of dout
 * The sums over rows are taken in a fixed order: equal calls give equal bits.
 *
 *   x, weight, eps   in   as csa_norm
 *   dout     in   [rows, n] of dout_dt
 *   dx       out  [rows, n] of dx_dt; may be dout's or x's buffer
 *   dweight  out  [n] fp32 or NULL (not wanted); written, not added to
 *   dbias    out  [n] fp32 or NULL
 *   workspace     csa_norm_bwd_workspace_size bytes, 16-byte aligned, used by
 *                 one call at a time; NULL where it is 0
 * Without rows dweight and dbias become zeros (their pointers are looked at).
 * Errors: as csa_norm; WORKSPACE when too small.
 */
size_t csa_norm_bwd_workspace_size(long long rows, int n, int want_dweight, int want_dbias);
csa_status_t csa_norm_bwd(const void* x, long long x_stride, csa_dtype_t dt, int kind,
                          const float* weight, float eps, const void* dout,
                          long long dout_stride, csa_dtype_t dout_dt, void* dx,
                          long long dx_stride, csa_dtype_t dx_dt, float* dweight, float* dbias,
                          long long rows, int n, void* workspace, size_t workspace_bytes,
                          csa_stream_t stream);

/* Pairs of a rotation of the `dim` channels from `first` on.  Interleaved:
 * pair i is (first + 2i, first + 2i + 1).  Half: (first + i, first + dim/2 + i). */
typedef enum { CSA_ROPE_INTERLEAVED = 0, CSA_ROPE_HALF = 1 } csa_rope_layout_t;

/* Frequencies.  CSA_ROPE_PLAIN: f_i = base^(-2i / dim).  CSA_ROPE_LINEAR:
 * f_i / factor.  CSA_ROPE_BY_PARTS: f_i * (1 - g_i) + f_i / factor * g_i with
 * g_i = clamp((i - lo) / max(hi - lo, 0.001), 0, 1), lo = floor(c(beta_fast)),
 * hi = ceil(c(beta_slow)), both clamped to [0, dim - 1], where c(n) = dim *
 * ln(original_len / (2 pi n)) / (2 ln(base)) is the pair that makes n turns in
 * original_len positions ("YaRN: Efficient Context Window Extension of Large
 * Language Models", interpolation by parts, with the ramp over pair indices).  That paper's
 * factor on queries and keys, 0.1 ln(factor) + 1, is csa_rope_t.scale. */
typedef enum { CSA_ROPE_PLAIN = 0, CSA_ROPE_LINEAR = 1, CSA_ROPE_BY_PARTS = 2 } csa_rope_scaling_t;

/*
 * csa_rope_freqs - the dim / 2 frequencies (radians a position) in double, on
 * the host.  original_len, beta_fast and beta_slow are read for BY_PARTS only,
 * factor not for PLAIN.
 * Errors: INVALID_ARG for a null pointer, dim odd or < 2, base, factor or
 * original_len not positive and finite, BY_PARTS with base == 1 or betas that
 * are not positive, beta_fast < beta_slow.
 */
csa_status_t csa_rope_freqs(int dim, double base, int scaling, double factor, double original_len,
                            double beta_fast, double beta_slow, double* freqs);

/*
 * csa_rope_turns - n frequencies as the part of a turn that one position makes,
 * in units of 2^-64 turns, on the host: frac(freq / 2 pi) * 2^64.  A caller
 * copies them to the device once (csa_rope_t.turns).  pos * turns mod 2^64 is
 * then the angle at pos without any loss but the frequency's own rounding.
 * Errors: INVALID_ARG for null pointers, n < 1, frequencies that are not finite.
 */
csa_status_t csa_rope_turns(const double* freqs, int n, int64_t* turns);

/* A rotation; lives on the host and is read during the call only. */
typedef struct {
  const int64_t* turns; /* device, [dim / 2], 16-byte aligned */
  int dim;              /* turned channels: even, >= 2 */
  int first;            /* first of them: even, first + dim <= d */
  int layout;           /* csa_rope_layout_t; half: dim % 4 == 0 */
  float scale;          /* factor on the turned channels, finite */
} csa_rope_t;

/* Rows [b, s, H, d]: strides of a sequence, a token and a head. */
typedef struct {
  long long batch, token, head;
} csa_row_strides_t;

/*
 * csa_rope - rotary positions.
 *
 * Row (i, t, h) is turned by its token's position p (pos[i, t], any int32; t
 * where pos is NULL): with the angle a = p * freq of pair (u, v), negated when
 * inverse != 0,
 *   u' = scale * (u cos a - v sin a),   v' = scale * (u sin a + v cos a).
 * Channels outside [first, first + dim) are copied; in place they are not
 * touched.  Angles are formed modulo a turn in 64-bit integers and their sine
 * and cosine are fp32.
 *
 *   x    in   [b, s, H, d] of dt       out  out  the same, own strides
 *   pos  in   [b, s] int32, batch stride pos_stride (0: shared by all
 *             sequences), or NULL
 * Errors: INVALID_ARG for null or misaligned pointers, d % 8 != 0, d < 8,
 * strides (above), a rotation outside its limits or the row, an unknown dtype;
 * UNSUPPORTED for d > 512 or b * s * H > 2^30.
 */
csa_status_t csa_rope(const void* x, const csa_row_strides_t* x_strides, csa_dtype_t dt,
                      const int32_t* pos, long long pos_stride, const csa_rope_t* rope,
                      int inverse, void* out, const csa_row_strides_t* out_strides, int b, int s,
                      int H, int d, csa_stream_t stream);

/*
 * csa_rope_bwd - gradient of csa_rope: dout turned back and scaled.
 *   dout  in  [b, s, H, d] of dout_dt     dx  out  [b, s, H, d] of dx_dt
 * Other arguments (inverse: the forward call's) and errors as csa_rope.
 */
csa_status_t csa_rope_bwd(const void* dout, const csa_row_strides_t* dout_strides,
                          csa_dtype_t dout_dt, const int32_t* pos, long long pos_stride,
                          const csa_rope_t* rope, int inverse, void* dx,
                          const csa_row_strides_t* dx_strides, csa_dtype_t dx_dt, int b, int s,
                          int H, int d, csa_stream_t stream);

/*
 * csa_norm_rope - csa_norm of every row's d channels (weight and bias [d], of
 * all heads), then csa_rope; nothing is rounded in between.  Arguments and
 * errors as theirs.
 */
csa_status_t csa_norm_rope(const void* x, const csa_row_strides_t* x_strides, csa_dtype_t dt,
                           int kind, const float* weight, const float* bias, float eps,
                           const int32_t* pos, long long pos_stride, const csa_rope_t* rope,
                           void* out, const csa_row_strides_t* out_strides, int b, int s, int H,
                           int d, csa_stream_t stream);

/*
 * csa_norm_rope_bwd - gradient of csa_norm_rope: dout turned back and scaled,
 * then csa_norm_bwd.  workspace: csa_norm_bwd_workspace_size of b * s * H rows
 * of d channels.  Arguments and errors as theirs.
 */
csa_status_t csa_norm_rope_bwd(const void* x, const csa_row_strides_t* x_strides, csa_dtype_t dt,
                               int kind, const float* weight, float eps, const int32_t* pos,
                               long long pos_stride, const csa_rope_t* rope, const void* dout,
                               const csa_row_strides_t* dout_strides, csa_dtype_t dout_dt,
                               void* dx, const csa_row_strides_t* dx_strides, csa_dtype_t dx_dt,
                               float* dweight, float* dbias, int b, int s, int H, int d,
                               void* workspace, size_t workspace_bytes, csa_stream_t stream);

/*
 * csa_compress_decode - the compressor for the newest s_q tokens of each
 * sequence.
 *
 * Sequence i has n = seq_lens[i] tokens, row k of whose new ones is at position
 * t = n - s_q + k (no token where t < 0: rows of padding).  Block j is complete
 * when n >= (j + 1) * ratio; the call handles the blocks that its tokens
 * complete, first[i] = max(0, n - s_q) / ratio of them being complete before and
 * counts[i] new:
 *   pooled row: csa_compress_overlap's entry j, over the positions
 *     max(0, (j + 1 - coff) * ratio) .. (j + 1) * ratio - 1, cast once to dt
 *     (only the scores' distances to the largest of the window count: any finite
 *     ones, the type's lowest among them, may mask; scores of -inf have no weight, a
 *     channel of nothing else is NaN)
 *   norm kind csa_norm_kind_t (0: none; weight, bias and eps are then not read)
 *   rotation of position (j + 1) * ratio - 1 (rope NULL: none), as csa_rope
 *   out[i, j - first[i]] = the result, cast once to dt
 * With CSA_NORM_RMS, interleaved pairs of the last channels and scale 1 the rows
 * are those of csa_compress_norm_rope, up to fp32 rounding before the casts.
 * out, first and counts are csa_cache_write's x, pos0 and counts.
 *
 * The rings keep the newest ring_rows rows of each sequence, position p in row
 * p mod ring_rows, and the call writes its tokens into them (of more than
 * ring_rows tokens the last).  Positions before the new tokens are read from the
 * rings: those of the unfinished block and, for coff 2, of the block before it,
 * as calls on the tokens before have left them.  A prompt is one call, or several;
 * s_q can be any length.  ring_rows >= coff * ratio - 1 + s_q of the longest call
 * whose tokens may be taken back (drafts): the rings then still hold what a call
 * with fewer tokens at the same place reads.
 *
 *   kv          in      [b, s_q, d] of dt, strides in elements, rows contiguous
 *   score       in      [b, s_q, score_width] of dt, likewise (width 1 or d)
 *   kv_ring     in/out  [b, ring_rows, d] of dt, packed
 *   score_ring  in/out  [b, ring_rows, score_width] of dt, packed
 *   seq_lens    in      [b] int32, new tokens included (below 0: 0, site 0x72)
 *   rope        in      csa_rope_t or NULL
 *   out         out     [b, ceil(s_q / ratio), d] of dt, batch stride out_stride
 *                       elements, rows packed; rows from counts[i] on are left as
 *                       they were
 *   first, counts  out  [b] int32
 * Two buffers of a call may not overlap.  s_q == 0 or b == 0 is a no-op (first and
 * counts are not written).
 * Errors: INVALID_ARG for null pointers, pointers (int32 arrays and scores of width 1
 * excepted) not 16-byte aligned, d % 8 != 0, a score_width that is neither 1 nor d,
 * ratio < 1, coff < 1, ring_rows < coff * ratio, strides (above; scores of width 1 may
 * have any that are not negative), a bad norm or rope; UNSUPPORTED for d > 512,
 * coff > 2, b > 65535, coff * ratio or ring_rows > 2^24.
 */
csa_status_t csa_compress_decode(const void* kv, long long kv_batch_stride,
                                 long long kv_row_stride, const void* score,
                                 long long score_batch_stride, long long score_row_stride,
                                 int score_width, void* kv_ring, void* score_ring, int ring_rows,
                                 const int32_t* seq_lens, int kind, const float* weight,
                                 const float* bias, float eps, const csa_rope_t* rope, void* out,
                                 long long out_stride, int32_t* first, int32_t* counts, int b,
                                 int s_q, int d, int ratio, int coff, csa_dtype_t dt,
                                 csa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* CSA_ROWS_H_ */
