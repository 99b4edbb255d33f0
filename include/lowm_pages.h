/*
 * lowm_pages.h -- C ABI of the bookkeeping of a paged cache (lowm_layer.h,
 * lowm_fp8.h) on the device: rows that share pages, fork, grow and end, and pages
 * that move.  Nothing here synchronizes or needs a number from the device, so a
 * decoding step with its cache can be captured in a graph.
 *
 * A row of `page_table` (int32 [rows, width], by row stride) lists the pages of a
 * sequence of lens[row] tokens: ceil(lens / page_size) entries count, at most
 * `width`.  refs[page] (int32 [num_pages]) is how many rows list the page; 0: it is
 * free.  Entries outside [0, num_pages) are passed over.  Free pages are taken in
 * rising order, so results do not depend on timing.  Conventions as in lowm_layer.h.
 *
 * Counts that come from outside of the table keep a page from being taken, not from
 * being written: the row that has it as its unfinished last page goes on in it, and
 * appending to 8 bits may move its codes to a larger scale.  Keep whole pages so.
 */
#ifndef LOWM_PAGES_H
#define LOWM_PAGES_H

#include <stddef.h>
#include <stdint.h>

#include "lowm_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Row i of the new table continues row parents[i] of the old one; a parent outside
 * [0, rows) gives an empty row.  refs gives up the old rows' pages and counts the
 * new rows'.  Whole pages are shared.  Rows whose last page is unfinished and is the
 * unfinished last page of an earlier new row, too, get a page of their own: src[i]
 * and dst[i] say what to copy there (-1: nothing).  Where no page is free the page
 * stays shared, src[i] and dst[i] are -1, and missing[0] counts it.
 *   parents       int32 [new_rows]
 *   new_table     int32 [new_rows, width] by row stride, no memory of the old one;
 *                 entries that do not count are set to -1
 *   new_lens, src, dst  int32 [new_rows]; missing int32 [1]
 *   rows, new_rows  0..8192
 */
lowm_status_t lowm_fork_pages(const int32_t *page_table, int64_t table_stride, const int32_t *lens, int rows,
                              const int32_t *parents, int new_rows, int width, int32_t *refs, int num_pages,
                              int page_size, int32_t *new_table, int64_t new_table_stride, int32_t *new_lens,
                              int32_t *src, int32_t *dst, int32_t *missing, void *stream);

/*
 * Room for new tokens: row b grows by cu_new[b+1] - cu_new[b] of them, on its last
 * page and on free pages.  page_table, lens and refs are updated in place.
 *   cu_new        int32 [rows + 1], non-decreasing from 0 to tokens
 *   positions     int64 [tokens]: a new token's position in its sequence
 *   slots         int64 [tokens]: page * page_size + place, for lowm_rope_append; -1
 *                 where the table is full or no page was left
 *   missing       int32 [1]: pages that were not to be had (their entries become -1)
 *   workspace     lowm_extend_pages_workspace(num_pages) bytes, 4-byte aligned
 *   rows          0..8192
 * An unfinished last page that other rows list as the same entry (lowm_fork_pages found
 * none free, or a row was cut back) goes on in the longest of them, of equal ones the
 * first; in the others the tokens that would lie in it have slot -1, and missing counts
 * a page for each such row.
 */
lowm_status_t lowm_extend_pages(int32_t *page_table, int64_t table_stride, int32_t *lens, int rows, int width,
                                const int32_t *cu_new, int tokens, int32_t *refs, int num_pages, int page_size,
                                int64_t *positions, int64_t *slots, int32_t *missing,
                                void *workspace, size_t workspace_bytes, void *stream);
size_t lowm_extend_pages_workspace(int num_pages);

/*
 * Brings the `used` pages that are not free together at 0 .. used - 1: those behind
 * move, in order, to the free ones before.  page_table and refs are updated in place;
 * src and dst list the moves for lowm_copy_pages, in order, then -1.  Entries of this
 * table that count follow their pages; those of another table on the same pool, or
 * behind lens, do not: every sequence of the pool is to be a row of the one table.
 *   src, dst      int32 [num_pages / 2]; used int32 [1]
 *   workspace     lowm_compact_pages_workspace(num_pages) bytes, 4-byte aligned
 */
lowm_status_t lowm_compact_pages(int32_t *page_table, int64_t table_stride, const int32_t *lens, int rows, int width,
                                 int32_t *refs, int num_pages, int page_size, int32_t *src, int32_t *dst, int32_t *used,
                                 void *workspace, size_t workspace_bytes, void *stream);
size_t lowm_compact_pages_workspace(int num_pages);

/* One tensor of a cache: page i is the page_bytes bytes at base + i * page_stride. */
typedef struct {
    void *base;
    int64_t page_stride;
    int64_t page_bytes;
} lowm_page_span_t;

/*
 * Copies page src[i] to page dst[i] in each of `count` tensors (keys, values and
 * scales of all layers), for i < pairs; pairs with an index outside [0, num_pages)
 * are passed over.  No page may be a destination twice or a source and a
 * destination (the lists of the operators above are such); its contents are
 * unspecified then.
 *   spans         on the host, read before the call returns
 *   src, dst      int32 [pairs] on the device
 */
lowm_status_t lowm_copy_pages(const lowm_page_span_t *spans, int count, const int32_t *src, const int32_t *dst, int pairs,
                              int num_pages, void *stream);

#ifdef __cplusplus
}
#endif
#endif
