/*
 * lowm_fp8.h -- C ABI of the 8-bit forms of the low-M GEMM (lowm_gemm.h) and of
 * the paged cache (lowm_layer.h) on GB300 (sm_103a).  Codes are e4m3 (4 exponent
 * and 3 mantissa bits, largest value 448, no infinities) and stand for code *
 * scale with fp32 scales by block.  The conventions are those of lowm_layer.h:
 * plain device pointers, caller-owned buffers, strides in elements with the
 * innermost dimension contiguous, checks before anything is enqueued, no
 * synchronization, bounded waits reported by lowm_gemm_sync_status.
 *
 * The scale that the operators give a block is the smallest power of two, 2^-100
 * at least, that brings its largest finite magnitude to 448 or less: dividing by
 * it rounds nothing.  Codes are rounded to nearest, ties to even.  What is not
 * finite becomes NaN.
 */
#ifndef LOWM_FP8_H
#define LOWM_FP8_H

#include <stddef.h>
#include <stdint.h>

#include "lowm_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Codes and scales of a bf16 matrix, a scale for each `block_rows` rows (1:
 * activations; 128: weights) and 128 columns.
 *   x             [rows, cols] bf16 by row stride
 *   codes         [rows, cols] e4m3, contiguous
 *   scales        [ceil(rows / block_rows), ceil(cols / 128)] fp32, contiguous
 *   rows >= 0, cols >= 1
 */
lowm_status_t lowm_quantize_fp8(const void *x, int64_t x_stride, void *codes, float *scales,
                                int rows, int cols, int block_rows, void *stream);

/*
 * C[M,N] = A[M,K] . W[N,K]^T with A and W in 8 bits:
 *
 *     C[m,n] = sum_b a_scale[m,b] w_scale[n / 128, b] sum_{k in block b} A[m,k] W[n,k]
 *
 * over the blocks of 128 along K.  Products of a block are summed by the tensor
 * cores, blocks in fp32 in a fixed order (the two scales are multiplied in fp32); C is
 * rounded once: the result is deterministic.
 *   A             [M, K] e4m3, contiguous; a_scale fp32 [M, ceil(K / 128)]
 *   W             [N, K] e4m3, contiguous; w_scale fp32 [ceil(N / 128), ceil(K / 128)]
 *   C             [M, N] bf16, contiguous
 *   M             1..128; N >= 1; K >= 16, a multiple of 16
 *   flags         0, or LOWM_FLAG_W_BEFORE_PDL_WAIT: the kernel that precedes this
 *                 launch on the stream does not write W
 * A and W 16-byte aligned.
 */
lowm_status_t lowm_gemm_fp8(const void *A, const float *a_scale, const void *W, const float *w_scale, void *C,
                            int M, int N, int K, unsigned flags, void *stream);

/*
 * lowm_gemm_fp8 of bf16 activations, which are quantised on the way as by
 * lowm_quantize_fp8 with block_rows 1.
 *   x             [M, K] bf16 by row stride
 *   workspace     lowm_gemm_fp8_bf16_workspace(M, K) bytes, 16-byte aligned; contents
 *                 need not survive between calls
 */
lowm_status_t lowm_gemm_fp8_bf16(const void *x, int64_t x_stride, const void *W, const float *w_scale, void *C,
                                 int M, int N, int K, unsigned flags, void *workspace, size_t workspace_bytes,
                                 void *stream);

/* Bytes of workspace lowm_gemm_fp8_bf16 needs (0 for sizes it refuses). */
size_t lowm_gemm_fp8_bf16_workspace(int M, int K);

/*
 * lowm_rope_append for a cache of codes.  k_cache and v_cache are e4m3
 * [num_pages, page_size, kv_heads, dim], k_scale and v_scale fp32 [num_pages,
 * page_size / block, kv_heads], all by strides.  A block is `block` places of a
 * page; its scale covers the tokens of one head in it.
 *
 * Tokens that share a block are to be neighbouring tokens of the call with rising
 * places, as a sequence's are; fewer than `block` tokens that are not appended may
 * lie between two of them.  The first of them says what the block holds: at
 * the block's first place the block begins anew, else the tokens at the places
 * before it stay, and when the new ones need a larger scale their codes are moved
 * to it (code * old / new, rounded).  What lies behind the last new token is of no
 * sequence and may hold anything.  A block that two such runs of one call write
 * holds one or the other, element by element unspecified.
 *   block         a power of two, at most page_size
 *   dim           1..256 (q, k, v and positions as in lowm_rope_append)
 * q_out is rounded once to bf16; k is quantised from the fp32 rotation, v from v.
 */
lowm_status_t lowm_rope_append_fp8(const void *q, int64_t q_token_stride, int64_t q_head_stride,
                                   const void *k, int64_t k_token_stride, int64_t k_head_stride,
                                   const void *v, int64_t v_token_stride, int64_t v_head_stride,
                                   const float *cos_sin, int64_t table_rows,
                                   const int64_t *positions, int64_t positions_stride, int axes,
                                   int section0, int section1, int interleaved, const int64_t *slots,
                                   void *q_out, int64_t q_out_token_stride, int64_t q_out_head_stride,
                                   void *k_cache, int64_t k_page_stride, int64_t k_place_stride,
                                   int64_t k_cache_head_stride,
                                   void *v_cache, int64_t v_page_stride, int64_t v_place_stride,
                                   int64_t v_cache_head_stride,
                                   float *k_scale, int64_t ks_page_stride, int64_t ks_block_stride,
                                   int64_t ks_head_stride,
                                   float *v_scale, int64_t vs_page_stride, int64_t vs_block_stride,
                                   int64_t vs_head_stride,
                                   int64_t num_pages, int page_size, int block,
                                   int tokens, int heads, int kv_heads, int dim, int rotary, void *stream);

/*
 * lowm_paged_attention over a cache of codes with their scales (as in
 * lowm_rope_append_fp8): key j counts as k_scale * k[j], its value as v_scale * v[j].
 *   k_cache, v_cache  base 16-byte aligned, strides multiples of 16 (of a dimension
 *                 of one they may be anything)
 *   k_scale       any fp32 numbers
 *   v_scale       0 .. 2^50, where less than 2^-50 counts as 2^-50; another one makes
 *                 the rows that see its tokens NaN
 *   block         a power of two, at most page_size
 * The other arguments, their limits and what a row that sees nothing gets are
 * those of lowm_paged_attention.  A length that the table has no room for counts as
 * the table's room.  What a page or a scale holds past a sequence's length or before
 * its window does not matter, NaN included; a NaN code reaches the rows that see its
 * token and no others.  An element of q that is not finite makes its row NaN, or
 * zeros where it makes all of the row's scores -inf.  The result is deterministic.
 */
lowm_status_t lowm_paged_attention_fp8(const void *q, int64_t q_token_stride, int64_t q_head_stride,
                                       const void *k_cache, int64_t k_page_stride, int64_t k_place_stride,
                                       int64_t k_cache_head_stride,
                                       const void *v_cache, int64_t v_page_stride, int64_t v_place_stride,
                                       int64_t v_cache_head_stride,
                                       const float *k_scale, int64_t ks_page_stride, int64_t ks_block_stride,
                                       int64_t ks_head_stride,
                                       const float *v_scale, int64_t vs_page_stride, int64_t vs_block_stride,
                                       int64_t vs_head_stride,
                                       int64_t num_pages, int page_size, int block,
                                       const int32_t *page_table, int64_t page_table_stride, int table_width,
                                       const int32_t *kv_lens, const int32_t *cu_q,
                                       void *out, int64_t out_token_stride, int64_t out_head_stride, float *lse,
                                       int batch, int q_tokens, int heads, int kv_heads, int dim,
                                       float scale, int window,
                                       void *workspace, size_t workspace_bytes, void *stream);

/*
 * Bytes of workspace lowm_paged_attention_fp8 needs (0 for sizes it refuses), 1.1 GiB
 * at most.  Calls with 96 rows a sequence and head and much room in the table take a
 * bf16 copy of what their rows see into it, for some sequences and heads at a time
 * where it has no room for all; weights meet values rounded to bf16 then, else to
 * fp16.
 */
size_t lowm_paged_attention_fp8_workspace(int batch, int q_tokens, int heads, int kv_heads, int dim, int page_size,
                                          int table_width);

#ifdef __cplusplus
}
#endif
#endif
