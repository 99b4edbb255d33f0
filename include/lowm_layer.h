/*
 * lowm_layer.h -- C ABI of the decoder-layer operators that stand around the
 * low-M GEMM (lowm_gemm.h) on GB300 (sm_103a): residual norms, rotary
 * positions with the append to a paged key/value cache, attention of a chunk
 * of new tokens over that cache, and a mixture-of-experts layer for at most
 * 128 tokens.  They are exported by the same library and follow the same
 * conventions: bf16 activations, weights and caches as plain device pointers,
 * caller-owned buffers, `stream` a cudaStream_t passed as void*, checks before
 * anything is enqueued, no synchronization, lowm_status_t results, waits of a
 * kernel bounded and reported by lowm_gemm_sync_status.  Strides are in
 * elements; the innermost dimension of every tensor is contiguous.
 *
 * Launches use programmatic dependent launch: every kernel waits for its
 * predecessor on the stream before it touches memory.
 */
#ifndef LOWM_LAYER_H
#define LOWM_LAYER_H

#include <stddef.h>
#include <stdint.h>

#include "lowm_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The norms after and before a block, fused with the block's gate and the
 * residual scale.  For every token t, with RMS(x; w) = w * x / sqrt(mean(x^2) + eps):
 *
 *     r'[t] = scale * residual[t] + gate[t] * RMS(block[t]; post_weight)
 *     out[t] = RMS(r'[t]; pre_weight)
 *
 * r' stays in fp32 between the two lines; out_residual and out are each
 * rounded once.
 *   residual, out_residual  [tokens, hidden], fp32 when residual_f32 else bf16;
 *                 they may be the same buffer.  out may lie between the rows of
 *                 out_residual, but share none of them
 *   block         [tokens, hidden] bf16, or NULL: no block precedes the norm
 *                 (post_weight, gate and out_residual must then be NULL and
 *                 scale 1; out = RMS(residual; pre_weight))
 *   post_weight   [hidden] bf16, or NULL: the block's output is taken as it is
 *   gate          bf16, or NULL for 1.  gate_stride 0: one row [hidden] for
 *                 all tokens, else the row stride of [tokens, hidden]
 *   pre_weight    [hidden] bf16, or NULL for 1
 *   out           [tokens, hidden] bf16
 *   tokens        >= 0 (0: nothing is launched); hidden 1..16384
 * Rows are read and written in 16-byte pieces when hidden and the strides are
 * multiples of 8 (4 for an fp32 residual) and the pointers 16-byte aligned.  With
 * other widths and strides they are, too, where that is faster, from the first
 * 16-byte boundary of a row on, if the pointers of the row tensors are 16-byte
 * aligned and their strides differ by multiples of 8 (hidden at most 15872); else
 * element by element.  Two reductions per row in a fixed order: the same
 * arguments, alignment included, give the same bits.
 */
lowm_status_t lowm_residual_norm(const void *residual, int residual_f32, int64_t residual_stride,
                                 const void *block, int64_t block_stride, const void *post_weight,
                                 const void *gate, int64_t gate_stride, const void *pre_weight,
                                 void *out_residual, int64_t out_residual_stride, void *out, int64_t out_stride,
                                 int tokens, int hidden, float scale, float eps, void *stream);

/*
 * Rotary positions for the new tokens' queries and keys, and the append of
 * their keys and values to a paged cache.
 *   q             [tokens, heads, dim], k, v [tokens, kv_heads, dim] bf16, by
 *                 token and head stride (slices of one projection will do)
 *   cos_sin       fp32 [table_rows, rotary]: cosines of the rotary / 2 pairs,
 *                 then their sines; 16-byte aligned
 *   positions     int64 [axes, tokens] by positions_stride: the table row of a
 *                 token on each axis (1 to 3: time, height, width)
 *   section0, section1  pairs that turn by axis 0 and axis 1 (pair j < section0:
 *                 axis 0; next section1: axis 1; the rest: axis 2).  With one
 *                 axis section0 = rotary / 2
 *   interleaved   0: pair j is (j, j + rotary / 2); 1: (2j, 2j + 1).  Elements
 *                 from `rotary` on are copied
 *   slots         int64 [tokens]: page * page_size + place in the page; a
 *                 negative one appends nothing (padding)
 *   q_out         [tokens, heads, dim] bf16 by strides; may be q itself
 *   k_cache, v_cache  [num_pages, page_size, kv_heads, dim] bf16, by page,
 *                 place and head strides; offsets are 64-bit
 * A position outside the table gives NaN (in the elements of q_out that turn)
 * and appends nothing; a slot outside the cache appends nothing.  Two tokens with one slot: one of them is
 * kept, element by element unspecified.  q, k and v are rounded once.
 *   dim, rotary   1..1024, 0..dim, rotary even
 */
lowm_status_t lowm_rope_append(const void *q, int64_t q_token_stride, int64_t q_head_stride,
                               const void *k, int64_t k_token_stride, int64_t k_head_stride,
                               const void *v, int64_t v_token_stride, int64_t v_head_stride,
                               const float *cos_sin, int64_t table_rows,
                               const int64_t *positions, int64_t positions_stride, int axes,
                               int section0, int section1, int interleaved, const int64_t *slots,
                               void *q_out, int64_t q_out_token_stride, int64_t q_out_head_stride,
                               void *k_cache, int64_t k_page_stride, int64_t k_place_stride, int64_t k_cache_head_stride,
                               void *v_cache, int64_t v_page_stride, int64_t v_place_stride, int64_t v_cache_head_stride,
                               int64_t num_pages, int page_size,
                               int tokens, int heads, int kv_heads, int dim, int rotary, void *stream);

/*
 * Attention of each sequence's newest tokens over its paged keys and values.
 * Sequence b has kv_lens[b] tokens in the cache, the last of which are its
 * cu_q[b+1] - cu_q[b] new ones (rows cu_q[b].. of q); new token i stands at
 * position p = kv_len - q_len + i and sees keys j <= p, and j > p - window when
 * window > 0.  Query head h reads key/value head h / (heads / kv_heads).
 *
 *     out[i, h] = sum_j softmax_j(scale * q[i, h] . k[j]) v[j]
 *
 * A row that sees no key (p < 0) gets zeros and lse = -inf.
 *   q, out        [q_tokens, heads, dim] bf16 by token and head stride
 *   k_cache, v_cache  as in lowm_rope_append; base 16-byte aligned, strides
 *                 multiples of 8 (of a dimension of one they may be anything)
 *   page_table    int32 [batch, table_width] by page_table_stride: the pages of
 *                 a sequence in order.  An entry outside the cache reads as zeros
 *   kv_lens       int32 [batch]; taken as at most table_width * page_size
 *   cu_q          int32 [batch + 1], non-decreasing from 0 to q_tokens
 *   lse           NULL, or fp32 [q_tokens, heads]: log of the sum of exponentials
 *   dim           64 or 128; page_size a power of two from 8 to 1024; heads a
 *                 multiple of kv_heads with heads / kv_heads <= 128; batch >= 0
 *   workspace     lowm_paged_attention_workspace(...) bytes, 16-byte aligned;
 *                 contents need not survive between calls
 * What a page holds past a sequence's length or before its window does not
 * matter, NaN included, and a value of a token that is not finite reaches the
 * rows that see the token and no others (where only some rows of a chunk see
 * it, at the price of a walk over at most 254 keys a row, some milliseconds
 * whatever the lengths).  The result is deterministic.
 */
lowm_status_t lowm_paged_attention(const void *q, int64_t q_token_stride, int64_t q_head_stride,
                                   const void *k_cache, int64_t k_page_stride, int64_t k_place_stride,
                                   int64_t k_cache_head_stride,
                                   const void *v_cache, int64_t v_page_stride, int64_t v_place_stride,
                                   int64_t v_cache_head_stride, int64_t num_pages, int page_size,
                                   const int32_t *page_table, int64_t page_table_stride, int table_width,
                                   const int32_t *kv_lens, const int32_t *cu_q,
                                   void *out, int64_t out_token_stride, int64_t out_head_stride, float *lse,
                                   int batch, int q_tokens, int heads, int kv_heads, int dim,
                                   float scale, int window,
                                   void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of workspace lowm_paged_attention needs (0 for sizes it refuses). */
size_t lowm_paged_attention_workspace(int batch, int q_tokens, int heads, int kv_heads, int dim);

#define LOWM_MOE_SOFTMAX 0
#define LOWM_MOE_SIGMOID 1

/*
 * A whole mixture-of-experts layer for 1..128 tokens:
 *
 *     l = x . router^T                              fp32 [tokens, experts]
 *     p = softmax(l) or sigmoid(l)
 *     e_1..e_k = the top_k largest of p + bias      (ties: the lowest index)
 *     w_s = scale * p[e_s]  (/ sum_s p[e_s] when renormalize)
 *     out = sum_s w_s * down[e_s] . (silu(gate[e_s] . x) * (up[e_s] . x))
 *
 *   x, out        [tokens, hidden] bf16 by row stride (at least hidden)
 *   router        [experts, hidden] bf16
 *   bias          NULL, or fp32 [experts]: enters the choice only
 *   gate_up       [experts, 2 * inner, hidden] bf16, gate rows before up rows
 *   down          [experts, hidden, inner] bf16
 *   hidden, inner multiples of 8 (16-byte rows), at most 32768
 *   experts       1..1024; top_k 1..min(16, experts)
 *   workspace     lowm_moe_workspace(...) bytes, 16-byte aligned; contents need
 *                 not survive between calls
 * Weights contiguous, 16-byte aligned.  Sums, softmax and the weighted sum of
 * the experts are fp32, in a fixed order: the result is deterministic.
 */
lowm_status_t lowm_moe(const void *x, int64_t x_stride, const void *router, const float *bias,
                       const void *gate_up, const void *down, void *out, int64_t out_stride,
                       int tokens, int hidden, int inner, int experts, int top_k,
                       int scoring, int renormalize, float scale,
                       void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of workspace lowm_moe needs (0 for sizes it refuses). */
size_t lowm_moe_workspace(int tokens, int hidden, int inner, int experts, int top_k);

#ifdef __cplusplus
}
#endif
#endif
