/*
 * dan_cache.h -- C ABI of the paged key/value cache operators (sm_103a).
 *
 *   dan_qk_norm_rope_cache  per-head RMSNorm + RoPE of Q and K at given
 *                           positions; K and V stored into a paged cache
 *   dan_window_attention    attention of ragged sequences over that cache,
 *                           with a sliding window, first tokens that stay
 *                           visible, and causality by chunks
 *
 * They continue the QK epilogue of dan.h for models that generate step by
 * step (token by token, or chunk of tokens by chunk) and keep the keys and
 * values of earlier steps.  Status codes, the device status word and the
 * conventions of dan.h hold here: device pointers owned by the caller,
 * nothing allocated or synchronised, launches asynchronous on `stream` with
 * programmatic dependent launch, invalid arguments refused without side
 * effects, 16-byte alignment.  Integer arrays are int32 in device memory,
 * 4-byte aligned, and are read by the kernels only.
 *
 * The cache.  k_cache and v_cache are [num_pages, kv_heads, page_size,
 * head_dim] bf16, contiguous: the page_size tokens of one head in one page
 * lie together.  page_size is 16, 32, 64 or 128; head_dim 64 or 128;
 * num_pages * kv_heads * page_size <= 2^31 - 256.  Slot n is token n % page_size
 * of page n / page_size.
 *
 * Index checks on the device.  An index that the arrays hold and that is out
 * of its range cannot be refused before the launch.  Such an entry is never
 * used as an address: the kernel leaves out what is said below and sets bit
 * 8 of the device status word (dan_get_device_status).  A wait that runs out
 * sets bits 1 and 4 as for the other kernels.
 */
#ifndef DAN_CACHE_H
#define DAN_CACHE_H

#include "dan.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------- QK-RMSNorm + RoPE + cache write
 * N tokens, q [N, heads*hd] with row stride q_row_stride and k, v
 * [N, kv_heads*hd] with row stride kv_row_stride (elements, multiples of 8,
 * >= the row; e.g. column slices of one packed projection).  heads is a
 * multiple of kv_heads.  For every token t and head of Q and of K
 *   rstd = rn(1/rn(sqrt(rn(rn(s/hd) + eps)))), s folded as in
 *          dan_qk_norm_rope_epilogue (8 columns in order per logical thread,
 *          then the adjacent-pair tree),
 *   n_j  = rn(rn(x_j * rstd) * w_j)    (fp32, not rounded to bf16)
 *   (out_a, out_b) = (bf16(rn(rn(n_a c_i) - rn(n_b s_i))),
 *                     bf16(rn(rn(n_a s_i) + rn(n_b c_i))))
 * with (a, b) = (2i, 2i+1), or (i, i + hd/2) when neox != 0, and c_i, s_i the
 * fp32 row rope[positions[t]] = [cos_0..cos_{hd/2-1} | sin_0..] of a table of
 * `table_rows` rows.  Unlike the epilogue the normalised value is not rounded
 * before the rotation: each output is rounded once.
 * q_out [N, heads, hd] has row stride qo_row_stride; the K head and the
 * unchanged V head go to slot slots[t] of the caches.  A negative slot stores
 * neither (a padding token); its q row is still written.  Two tokens of one
 * call must not share a slot (which one's heads stay is then not defined).
 * Slots that no token names keep their contents.  positions[t] outside
 * [0, table_rows): the token is left out (q row and slot unchanged), bit 8.
 * slots[t] >= num_pages*page_size: K and V are not stored, bit 8.
 * In place: q_out == q with qo_row_stride == q_row_stride; q, k and v may then
 * still be the columns of one packed projection, in any order. */
int dan_qk_norm_rope_cache(const dan_bf16 *q, const dan_bf16 *k, const dan_bf16 *v, int64_t N,
                           int64_t q_row_stride, int64_t kv_row_stride, int64_t heads,
                           int64_t kv_heads, int64_t head_dim, const dan_bf16 *wq,
                           const dan_bf16 *wk, const float *rope, int64_t table_rows,
                           const int32_t *positions, const int32_t *slots, float eps, int neox,
                           dan_bf16 *q_out, int64_t qo_row_stride, dan_bf16 *k_cache,
                           dan_bf16 *v_cache, int64_t num_pages, int64_t page_size, void *stream);
int dan_can_use_qk_norm_rope_cache(const dan_bf16 *q, const dan_bf16 *k, const dan_bf16 *v,
                                   int64_t N, int64_t q_row_stride, int64_t kv_row_stride,
                                   int64_t heads, int64_t kv_heads, int64_t head_dim,
                                   const dan_bf16 *wq, const dan_bf16 *wk, const float *rope,
                                   int64_t table_rows, const int32_t *positions,
                                   const int32_t *slots, float eps, int neox,
                                   const dan_bf16 *q_out, int64_t qo_row_stride,
                                   const dan_bf16 *k_cache, const dan_bf16 *v_cache,
                                   int64_t num_pages, int64_t page_size);

/* ------------------------------------------------ attention over the cache
 * S sequences; sequence s has the query rows q_start[s] .. q_start[s+1]-1 of
 * q [N, heads, hd] (row stride q_row_stride), n_s of them, and kv_len[s] keys
 * in the cache, key j in page page_table[s][j / page_size] (int32 rows of
 * table_stride entries, max_pages of them used), offset j % page_size.  The
 * queries are the sequence's last tokens: row i has position
 * p = kv_len[s] - n_s + i, and with
 *   p0 = p - p % chunk,  hi = min(kv_len[s], p0 + chunk),  lo = p0 + 1 - window
 * it sees the keys j < hi with j < sinks or j >= lo: its own chunk of `chunk`
 * tokens whole, the `window` tokens up to its chunk's first, and the first
 * `sinks` tokens.  chunk == 1 is plain causal attention in which a token sees
 * itself and the window - 1 tokens before it.  window == 0: the first
 * `sinks` tokens only.
 *   out_i = sum_j softmax_j(scale * q_i . k_j) v_j    bf16 [N, heads, hd]
 *   lse_i = ln sum_j exp(scale * q_i . k_j)           fp32 [N, heads]
 * query head h reads key head h / (heads / kv_heads).  lse may be NULL.  A row
 * that sees no key (also one with p < 0) gives out 0 and lse -infinity.  Rows
 * of q outside every sequence are not looked at, and out and lse keep theirs.
 * A row whose scores are all -infinity counts as one that sees no key.
 * Key slots that no query of their sequence sees are not used: they may hold
 * anything (NaN included), and page-table entries that cover only such slots
 * may be anything (e.g. -1).  A value row that some query of the call sees
 * must be finite, of magnitude at most 2^99 (2^94 where kv_len > 2^24): the
 * sums are divided after they are taken, and larger values may take them past
 * fp32's range.  Keys may hold anything (a query that sees a NaN key, or one
 * whose score is +infinity, gives NaN).
 *
 * Arithmetic: products of bf16 values summed in fp32; the softmax statistics
 * in fp32; each probability rounded to bf16 for its product with V, the sum
 * that divides taken before that rounding.  Unlike the operations of dan.h
 * the bits are not those of a written-out order of sums.  They are batch
 * invariant all the same: a row's bits depend on its own sequence (its n_s,
 * kv_len, queries and visible keys) and on window, sinks, chunk, scale and the
 * head counts, never on the other sequences, N, S, max_q, the page size or
 * where the pages lie.
 *
 * max_q: an upper bound on every n_s that the caller knows (N when none is):
 * a smaller one launches less.  A sequence with more than max_q rows is left
 * out, bit 8.  q_start entries that descend or leave [0, N]: the sequence is
 * left out, bit 8.  kv_len outside [0, max_pages*page_size]: taken as the
 * nearest bound, bit 8.  A page id outside [0, num_pages) for a visible key:
 * zeros in place of the page's keys and values, bit 8.  Sequences may share
 * pages and q rows must not be shared: a sequence with n_s * heads / kv_heads
 * > 16 that begins before an earlier one's end is left out, bit 8; where a
 * shorter one overlaps another, the rows of both are not defined in out and
 * lse (other rows are not touched).
 *
 * workspace: dan_window_attention_workspace(...) bytes of device memory,
 * 16-byte aligned, used by this call alone until it has completed (0 bytes:
 * may be NULL).  The count follows from its arguments alone: a call passes the
 * same ones.  A window that lets a query see little of a long table asks for
 * less, and for none where no sequence can be split.  Two calls that may run
 * at the same time, or two captured graphs that may, need one each.
 * Limits: S <= 2^20, heads <= 1024, heads / kv_heads <= 128, q_row_stride < 2^39,
 * N * heads <= 2^30, max_pages*page_size <= 2^30, window,
 * sinks, chunk in [0, 2^31 - 1] with chunk >= 1; scale finite and > 0. */
int64_t dan_window_attention_workspace(int64_t N, int64_t S, int64_t heads, int64_t kv_heads,
                                       int64_t head_dim, int64_t max_pages, int64_t page_size,
                                       int64_t window, int64_t sinks, int64_t chunk, int64_t max_q);
int dan_window_attention(const dan_bf16 *q, int64_t N, int64_t q_row_stride,
                         const dan_bf16 *k_cache, const dan_bf16 *v_cache, int64_t num_pages,
                         int64_t page_size, const int32_t *page_table, int64_t table_stride,
                         int64_t max_pages, const int32_t *q_start, const int32_t *kv_len,
                         int64_t S, int64_t heads, int64_t kv_heads, int64_t head_dim,
                         int64_t window, int64_t sinks, int64_t chunk, int64_t max_q, float scale,
                         dan_bf16 *out, float *lse, void *workspace, int64_t workspace_bytes,
                         void *stream);
int dan_can_use_window_attention(const dan_bf16 *q, int64_t N, int64_t q_row_stride,
                                 const dan_bf16 *k_cache, const dan_bf16 *v_cache,
                                 int64_t num_pages, int64_t page_size, const int32_t *page_table,
                                 int64_t table_stride, int64_t max_pages, const int32_t *q_start,
                                 const int32_t *kv_len, int64_t S, int64_t heads, int64_t kv_heads,
                                 int64_t head_dim, int64_t window, int64_t sinks, int64_t chunk,
                                 int64_t max_q, float scale, const dan_bf16 *out, const float *lse,
                                 const void *workspace, int64_t workspace_bytes);

#ifdef __cplusplus
}
#endif

#endif /* DAN_CACHE_H */
