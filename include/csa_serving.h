/*
 * csa_serving.h -- the operators of libcsa around serving the Compressor's rows: the norms, one of which writes rows (in
 * 8 bits with scales) to the slots of a paged cache, the append of rows to such a cache with the position rotation on the
 * way, the tables that say where a request's rows lie, and the attention whose keys and values are those rows, for
 * requests by themselves and for a batch that shares a prefix.
 *
 * The conventions are csa.h's: device pointers on the current device, caller-owned; every call is asynchronous on
 * `stream`, never synchronises, and returns a csa_status (csa_last_error_message() has the text); a failed validation
 * launches nothing.  Kernels are programmatic dependents of their stream predecessor.  Workspace comes from the
 * library's stream-ordered pool, allocated and released in stream order inside the call, so calls can be captured
 * into CUDA graphs (make the first call on a device before the capture).  Results do not depend on what ran before
 * and are bitwise reproducible; no floating-point atomics.  Kernels bound their waits on shared-memory barriers as the
 * Compressor's do: one that expires is recorded in the device's status word (csa_device_status), and that call's results
 * are not valid.
 */
#ifndef CSA_SERVING_H_
#define CSA_SERVING_H_

#include "csa.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum csa_dtype {
    CSA_DTYPE_BF16 = 0,
    CSA_DTYPE_F16 = 1,
    CSA_DTYPE_F32 = 2,
    CSA_DTYPE_E4M3 = 3   /* 8-bit float, 4 exponent bits, largest value 448 */
} csa_dtype;

/*
 * Root-mean-square norm with the residual's addition:
 *   h = round(x + residual)    rounded to dtype (h = x when residual is NULL)
 *   rstd = 1 / sqrt(mean(h^2) + eps),  y = h * rstd * weight      in fp32
 *   out = round(y) in dtype, or with out_dtype E4M3: scale = max|y| / 448 over scale_group columns (0: the whole row;
 *   128), out = e4m3(y / scale); a group of zeros has scale 0, one with a NaN among its y scale NaN.
 *   y / scale is y times the rounded reciprocal: a quotient within two fp32 roundings of the middle between two 8-bit values
 *   may go to the other one.
 *
 * x, residual: [n_rows, dim] of dtype (BF16, F16 or F32), row strides in elements, at least dim.  weight: fp32 [dim]
 * or NULL (ones).  out_dtype: dtype or E4M3.  slots: int64 [n_rows] or NULL; row i goes to row slots[i] of out and
 * scales, and nowhere when slots[i] is outside [0, n_slots) (distinct rows need distinct slots); without slots row i
 * goes to row i and n_slots is ignored.  scales: fp32 [rows of out, groups], E4M3 only.  residual_out (h, contiguous) and rstd (fp32
 * [n_rows]) may be NULL.  Without slots an out of dtype and residual_out may be x or residual themselves (same stride);
 * otherwise outputs overlap no input.
 * dim in [1, 16384]; scale_group 128 needs dim a multiple of 128 and 16-byte aligned bases and strides
 * (CSA_ERR_MISALIGNED); everything else takes any alignment of its elements, faster where rows are 16-byte aligned.
 */
CSA_API int csa_rms_norm_fwd(const void *x, int64_t x_stride, const void *residual, int64_t residual_stride,
                     const float *weight, int64_t n_rows, int32_t dim, float eps, int32_t dtype,
                     const int64_t *slots, int64_t n_slots, void *out, int64_t out_stride, int32_t out_dtype,
                     float *scales, int32_t scale_group, void *residual_out, float *rstd, void *stream);

/*
 * Gradient of csa_rms_norm_fwd (outputs in dtype), from h (residual_out, or x without a residual) and rstd:
 *   c = mean(weight * grad_out * h * rstd)
 *   grad_x = rstd * (weight * grad_out - h * rstd * c) + grad_residual     (the residual's gradient is the same)
 *   grad_weight = sum over rows of grad_out * h * rstd                     (fp32, fixed order; overwritten)
 * grad_residual: the gradient that reaches residual_out, or NULL.  grad_x is contiguous [n_rows, dim] and may be
 * grad_out or grad_residual itself when that is contiguous.  weight NULL: ones; grad_weight may be NULL.
 * n_rows == 0 writes zeros to grad_weight.
 */
CSA_API int csa_rms_norm_bwd(const void *h, int64_t h_stride, const void *grad_out, int64_t grad_out_stride,
                     const void *grad_residual, int64_t grad_residual_stride, const float *weight,
                     const float *rstd, int64_t n_rows, int32_t dim, int32_t dtype, void *grad_x,
                     float *grad_weight, void *stream);

/*
 * Layer norm with the residual's addition:
 *   h = round(x + residual)    rounded to dtype (h = x when residual is NULL)
 *   mean = mean(h),  rstd = 1 / sqrt(mean((h - mean)^2) + eps),  out = round((h - mean) * rstd * weight + bias)   in fp32
 *
 * x, residual: [n_rows, dim] of dtype (BF16, F16 or F32), row strides in elements, at least dim.  weight, bias: fp32 [dim]
 * or NULL (ones, zeros).  residual_out (h, contiguous), mean and rstd (fp32 [n_rows]) may be NULL.  out and residual_out may
 * be x or residual themselves (same stride); otherwise outputs overlap no input.  dim in [1, 16384]; any alignment of the
 * elements, faster where rows are 16-byte aligned.
 */
CSA_API int csa_layer_norm_fwd(const void *x, int64_t x_stride, const void *residual, int64_t residual_stride,
                       const float *weight, const float *bias, int64_t n_rows, int32_t dim, float eps, int32_t dtype,
                       void *out, int64_t out_stride, void *residual_out, float *mean, float *rstd, void *stream);

/*
 * Gradient of csa_layer_norm_fwd, from h (residual_out, or x without a residual), mean and rstd, with
 * u = (h - mean) * rstd and g = weight * grad_out:
 *   grad_x = rstd * (g - mean_of(g) - u * mean_of(g * u)) + grad_residual     (the residual's gradient is the same)
 *   grad_weight = sum over rows of grad_out * u,  grad_bias = sum over rows of grad_out   (fp32, fixed order; overwritten)
 * grad_residual: the gradient that reaches residual_out, or NULL.  grad_x is contiguous [n_rows, dim] and may be
 * grad_out or grad_residual itself when that is contiguous.  weight NULL: ones; grad_weight and grad_bias may be NULL.
 * n_rows == 0 writes zeros to them.
 */
CSA_API int csa_layer_norm_bwd(const void *h, int64_t h_stride, const void *grad_out, int64_t grad_out_stride,
                       const void *grad_residual, int64_t grad_residual_stride, const float *weight, const float *mean,
                       const float *rstd, int64_t n_rows, int32_t dim, int32_t dtype, void *grad_x, float *grad_weight,
                       float *grad_bias, void *stream);

/*
 * Rows appended to a paged cache, their last rot_dim columns rotated by the row's position, and queries rotated beside them.
 * A row is rows[i] with the rotated columns last, or, with rotary, rows[i] (row_dim columns) followed by the rotation of
 * rotary[i] (rot_dim columns); width = row_dim, or row_dim + rot_dim.  The columns to rotate are rot_dim / 2 pairs (a, b),
 * pair i columns (2 i, 2 i + 1) when interleaved, else (i, i + rot_dim / 2):
 *   (a, b) -> (a cos - b sin, a sin + b cos)      in fp32, one rounding
 * with cos = rotation[position][i] and sin = rotation[position][rot_dim / 2 + i].
 *
 * rows, rotary, q: dtype (BF16, F16 or F32); row strides in elements.  positions: int32 [n_rows]; a position outside
 * [0, n_positions) makes the rotated columns NaN.  rotation: fp32 [n_positions, rot_dim], contiguous.  slots: int64 [n_rows];
 * row i goes to row slots[i] of out and nowhere when that is outside [0, n_slots) (distinct rows need distinct slots).
 * out: [n_slots, width], dtype or E4M3; with E4M3 scales fp32 [n_slots] gets max|row| / 448 and out e4m3(row / scale) (a row of
 * zeros has scale 0, one with a NaN scale NaN; the quotient as in csa_rms_norm_fwd).
 * q: n_tokens tokens of n_heads heads, rot_dim columns each, element (token, head, c) at token * q_token_stride +
 * head * q_head_stride + c; rotated to q_out (strides of its own; q itself when the strides agree) by q_positions int32
 * [n_tokens].  n_rows 0 or n_tokens 0: nothing of that kind is done.  Otherwise outputs overlap no input.
 * rot_dim even in [2, 1024], width at most 1024, n_tokens * n_heads < 2^31.  Any alignment of the elements; faster where rows
 * are 16-byte aligned and halves (interleaved: parts) are whole 16-byte vectors.
 */
CSA_API int csa_append_rows(const void *rows, int64_t row_stride, int32_t row_dim, const void *rotary, int64_t rotary_stride,
                    int32_t rot_dim, const int32_t *positions, int64_t n_rows, int32_t dtype, const float *rotation,
                    int64_t n_positions, int32_t interleaved, const int64_t *slots, int64_t n_slots, void *out,
                    int64_t out_stride, int32_t out_dtype, float *scales, const void *q, int64_t q_token_stride,
                    int64_t q_head_stride, const int32_t *q_positions, int64_t n_tokens, int32_t n_heads, void *q_out,
                    int64_t q_out_token_stride, int64_t q_out_head_stride, void *stream);

/*
 * The rotation of csa_append_rows alone, over n_heads heads of n_tokens tokens, or with inverse its inverse (by the negated
 * angle): what an attention's output takes whose values were rotated with the keys, and the rotation's gradient.  out may be
 * x itself when the strides agree.
 */
CSA_API int csa_rotate(const void *x, int64_t x_token_stride, int64_t x_head_stride, const int32_t *positions, int64_t n_tokens,
               int32_t n_heads, int32_t rot_dim, int32_t dtype, const float *rotation, int64_t n_positions, int32_t interleaved,
               int32_t inverse, void *out, int64_t out_token_stride, int64_t out_head_stride, void *stream);

/*
 * Block tables, offsets and slots of a paged cache of compressed rows.  Request r goes from before[r] to after[r]
 * tokens, that is from floor(before/ratio) to floor(after/ratio) rows (never fewer than before), in pages of
 * page_size rows:
 *   table_out [n_req, width]  the pages of r: those it holds (copied from table), then free_pages[taken ...] in
 *                             request order, -1 past its need and where free pages run out
 *   cu_rows   [n_req + 1]     offsets of the requests' new rows, in order
 *   slots     int64 [capacity] page * page_size + offset of each new row, -1 where it has no page and past the last
 *   counts    [4]             new rows, pages taken, pages short, the most pages that a request needs
 * taken: device int32 or NULL, the entries of free_pages [n_free] that are already used.  table: [n_req, width] with
 * row stride table_stride; table_out is contiguous and may be table itself when table_stride == width.  All arrays
 * are int32 unless said otherwise.  Negative lengths count as 0.  n_req <= 14000.  Sums of rows and of pages are held at
 * 2^31 - 1.
 *
 * A table narrower than a need (counts[3] > width) holds none of the pages past its columns, although counts[1] counts
 * them and later requests get the entries of free_pages behind them: such a result is not to be kept.  Call again with a
 * table of counts[3] columns or more (those past the pages that a request holds may have anything in them) and the same
 * taken, which gives what the wider table would have given at once, after a call in place too.
 */
CSA_API int csa_page_tables(const int32_t *before, const int32_t *after, int32_t n_req, int32_t ratio, int32_t page_size,
                    const int32_t *free_pages, int32_t n_free, const int32_t *taken, const int32_t *table,
                    int64_t table_stride, int32_t width, int64_t capacity, int32_t *table_out, int32_t *cu_rows,
                    int64_t *slots, int32_t *counts, void *stream);

/*
 * Attention whose keys and values are one shared row a position (the Compressor's rows) of a paged cache, for all
 * query heads: with k_j the cache rows of the token's request and v_j their first v_dim columns,
 *   s_j = scale * q . k_j,   out = sum_j exp(s_j) v_j / (sum_j exp(s_j) + exp(sink)),
 *   lse = log(sum_j exp(s_j) + exp(sink))
 * (evaluated relative to the running maximum).  Token i of the nq new tokens of request r sees the first
 *   floor((seq_lens[r] - nq + i + 1) / ratio)
 * rows, that is the blocks that it completes or that lie before it, at most width * page_size; seq_lens counts the
 * request's tokens, the new ones among them.  A token that sees no row gives out = 0 and lse = sink (-inf without).
 *
 * q          bf16, element (token, head, c) at token * q_token_stride + head * q_head_stride + c
 * cu_q       int32 [n_req + 1], tokens [cu_q[r], cu_q[r+1]) of q belong to r; tokens past cu_q[n_req] are left alone
 * cache      [n_pages, page_size, head_dim], row stride cache_stride in elements; BF16, or E4M3 with
 * row_scales fp32 [n_pages * page_size]: a row's values are e4m3 * scale
 * block_table int32 [n_req, width], row stride table_stride; an entry outside [0, n_pages) hides its rows
 * sink       fp32 [n_heads], finite or -inf, or NULL
 * out        bf16 [n_tokens, n_heads, v_dim] contiguous;  lse fp32 [n_tokens, n_heads] or NULL
 *
 * n_req <= 14000, n_heads <= 4096, n_tokens * n_heads < 2^31; n_pages * page_size and width * page_size at most
 * 2^31 - 128.  head_dim: a multiple of 8 in [8, 1024], v_dim a multiple of 8 in [8, head_dim].  Multiples of 64 up to head_dim 576
 * and v_dim 512 run on the tensor cores; other widths on the fp32 units.  q and cache bases and strides are multiples
 * of 16 bytes (CSA_ERR_MISALIGNED).  Products take bf16 operands (an 8-bit value is exact in bf16; its scale is
 * applied in fp32) and fp32 sums; on the tensor cores the weights exp(s - m) are rounded to bf16 for the second
 * product.  Values that no token sees are never read into a result: cache memory past a request's rows may hold
 * anything.
 */
CSA_API int csa_latent_attention(const void *q, int64_t q_token_stride, int64_t q_head_stride, const int32_t *cu_q,
                         int32_t n_req, int64_t n_tokens, int32_t n_heads, int32_t head_dim, int32_t v_dim,
                         const void *cache, int64_t cache_stride, int32_t cache_dtype, const float *row_scales,
                         int64_t n_pages, int32_t page_size, const int32_t *block_table, int64_t table_stride,
                         int32_t width, const int32_t *seq_lens, int32_t ratio, float scale, const float *sink,
                         void *out, float *lse, void *stream);

/*
 * csa_latent_attention for a batch whose requests share prefixes: requests [cu_groups[g], cu_groups[g+1]) have their first
 * shared_rows[g] rows in common (a system prompt, a document), which are read once for the group instead of once for each
 * request.  The result is csa_latent_attention's of the same arguments.  block_table lists each request's pages from its first
 * row on, as there: for the shared rows the same pages, or pages with equal contents (the rows of any one of them may be
 * the ones that are read).
 *
 * cu_groups int32 [n_groups + 1], not decreasing, within [0, n_req]; requests outside of all groups share nothing.
 * shared_rows int32 [n_groups].  Rows that some token of the group does not see are not shared, whatever shared_rows says.
 * What is read once is whole pages of the first request of a group that has new tokens, up to its first table entry outside the
 * cache; none in a group with a request of more rows than its table lists.  Rows of 128 to 576 columns in multiples of 64 with
 * v_dim 128, 256, 384 or 512 are shared, in calls that can gain from it: the host, which does not see the lengths, goes by the query rows
 * and by width * page_size, so that a table much wider than its requests need sends a small batch the way of a large one (5 requests of 16
 * heads behind 2048 rows 25.5 us with a table for 131072 rows, 18.6 with a narrow view of it or by csa_latent_attention).  Others are read by request.
 * Memory: fp32 sums of every query row, 4 GiB at most; for 8-bit rows and pages that are no multiples of 8 rows bf16 copies of the
 * groups' prefixes, with room for the lesser of a table's and the cache's rows each and 1 GiB for all groups (prefix rows past that
 * are read by request).  Where the device has no such memory the call is read by request.
 * Everything else, and every limit, as in csa_latent_attention; n_groups <= 14000.
 */
CSA_API int csa_shared_attention(const void *q, int64_t q_token_stride, int64_t q_head_stride, const int32_t *cu_q,
                         int32_t n_req, int64_t n_tokens, int32_t n_heads, int32_t head_dim, int32_t v_dim,
                         const void *cache, int64_t cache_stride, int32_t cache_dtype, const float *row_scales,
                         int64_t n_pages, int32_t page_size, const int32_t *block_table, int64_t table_stride,
                         int32_t width, const int32_t *seq_lens, const int32_t *cu_groups, const int32_t *shared_rows,
                         int32_t n_groups, int32_t ratio, float scale, const float *sink, void *out, float *lse,
                         void *stream);

#ifdef __cplusplus
}
#endif

#endif /* CSA_SERVING_H_ */
