// Bookkeeping of a paged cache on the device (lowm_pages.h): fork, extend and
// compact page tables, and copy pages.
//
// The tables are whole numbers and small; what these kernels cost is the chain of
// launches and memory latencies, so each operator is one launch where it is small, three at most.
// Reference counts change by integer atomics, whose order does not matter; free
// pages are ranked by scans over the counts, in rising order, by one CTA (fork,
// extend: it stops at the last page it needs) or by chunks (compact).  Copies are
// bound by bandwidth.  A fork with its copies and growth: 8 rows on 149 pages, 16
// tensors 13 us, 128 rows, 32 tensors 25; a pool of 4096 pages brought together 58,
// 46 of them its copies (250 MB, 5.4 TB/s).
#include <algorithm>
#include <climits>

#include "../../include/lowm_pages.h"
#include "layer_host.h"
#include "ptx.cuh"

namespace lowm {
namespace {

constexpr int kPageThreads = 1024;           // of the CTA that ranks free pages
constexpr int kMaxRows = 8192;
constexpr int kFewRows = 64;                 // that one CTA forks, two a warp

struct Table {
    int32_t *entries;
    int64_t stride;
    const int32_t *lens;
    int rows, width;
};

struct Pool {
    int32_t *refs;
    int pages, page_size;
};

__device__ __forceinline__ int pages_of(int64_t tokens, int page_size)
{
    return (int)((tokens + page_size - 1) / page_size);
}

// Entries of a row that count.
__device__ __forceinline__ int used_of(int len, const Pool &pool, int width)
{
    return len <= 0 ? 0 : min(pages_of(len, pool.page_size), width);
}

__device__ __forceinline__ bool in_pool(int page, const Pool &pool) { return page >= 0 && page < pool.pages; }

// Exclusive prefix sum over the CTA's threads in order, and the total.
__device__ __forceinline__ int scan_block(int x, int &total)
{
    __shared__ int sums[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int upto = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o)
            upto += y;
    }
    if (lane == 31)
        sums[warp] = upto;
    __syncthreads();
    if (warp == 0) {
        int s = lane < warps ? sums[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o)
                s += y;
        }
        sums[lane] = s;
    }
    __syncthreads();
    total = sums[warps - 1];
    const int before = (warp > 0 ? sums[warp - 1] : 0) + upto - x;
    __syncthreads();
    return before;
}

// Calls found(rank, page) for the first `want` free pages, in rising order; returns how many there were.  The whole CTA.
template <typename Found>
__device__ __forceinline__ int free_pages(const Pool &pool, int want, Found found)
{
    constexpr int kEach = 8;                 // pages a thread looks at, at once
    int have = 0;
    for (int64_t p0 = 0; p0 < pool.pages && have < want; p0 += kEach * kPageThreads) {
        const int64_t first = p0 + kEach * threadIdx.x;
        int r[kEach], n = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            r[i] = first + i < pool.pages ? pool.refs[first + i] : 1;
            n += r[i] == 0;
        }
        if (!__syncthreads_or(n))
            continue;
        int total;
        int rank = have + scan_block(n, total);
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if (r[i] == 0) {
                if (rank < want)
                    found(rank, (int)(first + i));
                ++rank;
            }
        have += total;
    }
    return min(have, want);
}

// ------------------------------------------------------------------ fork
// An old row's pages are given up, a new row's counted and listed, by threads first, first + step, ... of the row.
__device__ __forceinline__ void fork_row(const Table &old, const int32_t *parents, const Table &next, int32_t *new_lens, const Pool &pool,
                                         int row, int first, int step)
{
    const bool gone = row < old.rows;
    const int i = gone ? row : row - old.rows;
    const int from = gone ? row : parents[i];
    const int len = from >= 0 && from < old.rows ? old.lens[from] : 0;
    const int used = used_of(len, pool, old.width);
    const int32_t *src = old.entries + from * old.stride;
    for (int j = first; j < (gone ? used : old.width); j += step) {
        const int page = j < used ? src[j] : -1;
        if (!gone)
            next.entries[i * next.stride + j] = page;
        if (in_pool(page, pool))
            atomicAdd(pool.refs + page, gone ? -1 : 1);
    }
    if (!gone && first == 0)
        new_lens[i] = len;
}

__global__ void __launch_bounds__(128) fork_rows_kernel(const Table old, const int32_t *parents, const Table next, int32_t *new_lens,
                                                        const Pool pool)
{
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    fork_row(old, parents, next, new_lens, pool, (int)blockIdx.x, threadIdx.x, blockDim.x);
}

// The unfinished last pages that several new rows have: the first of the rows keeps it.
// With `old`, the rows themselves come first, a warp each (few of them: a launch less).
__global__ void __launch_bounds__(kPageThreads) fork_tails_kernel(const Table old, const int32_t *parents, const Table next,
                                                                  int32_t *new_lens, const Pool pool, int32_t *src, int32_t *dst,
                                                                  int32_t *missing, int rows_first)
{
    extern __shared__ int32_t tails[];       // [rows]
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    if (rows_first) {
        for (int row = threadIdx.x >> 5; row < old.rows + next.rows; row += kPageThreads / 32)
            fork_row(old, parents, next, new_lens, pool, row, threadIdx.x & 31, 32);
        __syncthreads();
    }
    const int each = (next.rows + kPageThreads - 1) / kPageThreads, row0 = threadIdx.x * each;
    auto tail_at = [&](int i) { return next.entries + i * next.stride + used_of(next.lens[i], pool, next.width) - 1; };
    for (int i = threadIdx.x; i < next.rows; i += kPageThreads) {
        const int len = next.lens[i];
        const bool unfinished = used_of(len, pool, next.width) > 0 && pages_of(len, pool.page_size) <= next.width && len % pool.page_size;
        const int page = unfinished ? *tail_at(i) : -1;
        tails[i] = in_pool(page, pool) ? page : -1;
        src[i] = dst[i] = -1;
    }
    __syncthreads();
    unsigned again = 0;                      // of this thread's rows, in order
    for (int k = 0; k < each && row0 + k < next.rows; ++k) {
        const int page = tails[row0 + k];
        if (page < 0 || pool.refs[page] < 2)
            continue;
        for (int i = 0; i < row0 + k; ++i)
            if (tails[i] == page) {
                again |= 1u << k;
                break;
            }
    }
    int want;
    int rank = scan_block(__popc(again), want);
    __syncthreads();
    // Row of each rank, over the tails (all have been looked at).
    for (int k = 0; k < each; ++k)
        if (again >> k & 1) {
            src[row0 + k] = tails[row0 + k];
        }
    __syncthreads();
    for (int k = 0; k < each; ++k)
        if (again >> k & 1)
            tails[rank++] = row0 + k;
    __syncthreads();
    const int have = free_pages(pool, want, [&](int r, int page) {
        const int i = tails[r];
        dst[i] = page;
        *tail_at(i) = page;
    });
    __syncthreads();                         // the counts have been read
    for (int r = threadIdx.x; r < want; r += kPageThreads) {
        const int i = tails[r];
        if (r < have) {
            pool.refs[dst[i]] = 1;
            atomicAdd(pool.refs + src[i], -1);
        } else {
            src[i] = -1;
        }
    }
    if (threadIdx.x == 0)
        *missing = want - have;
}

// ------------------------------------------------------------------ extend
struct NewTokens {
    const int32_t *cu;
    int tokens;
    int64_t *positions, *slots;
};

// Whether another row has page `page`, entry j of a row of `len` tokens, and goes on in it in that row's place: a longer one,
// or an equally long one before it.  (Rare: a fork found no free page, or a row was cut back.)  lens are the new ones.
__device__ __noinline__ bool is_anothers(const Table &table, const Pool &pool, const NewTokens &fresh, int row, int len, int j, int page)
{
    for (int r = 0; r < table.rows; ++r) {
        const int old = table.lens[r] - max(fresh.cu[r + 1] - fresh.cu[r], 0);
        if (r != row && old >= len && (old > len || r < row) && used_of(old, pool, table.width) > j && table.entries[r * table.stride + j] == page)
            return true;
    }
    return false;
}

// Positions and slots of tokens `first`, first + step, ...; lens are the rows' new ones.  `missing` counts the rows that cannot
// go on in a page that they share.
__device__ __forceinline__ void place_tokens(const Table &table, const Pool &pool, const NewTokens &fresh, int32_t *missing, int first,
                                             int step)
{
    for (int t = first; t < fresh.tokens; t += step) {
        int lo = 0, hi = table.rows;         // the last row that begins at t or before
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (fresh.cu[mid + 1] <= t)
                lo = mid + 1;
            else
                hi = mid;
        }
        int64_t position = 0, slot = -1;
        if (lo < table.rows && fresh.cu[lo] <= t) {
            position = (int64_t)table.lens[lo] - (fresh.cu[lo + 1] - t);
            const int64_t j = position / pool.page_size;
            const int page = j < table.width ? table.entries[lo * table.stride + j] : -1;
            if (in_pool(page, pool)) {
                slot = (int64_t)page * pool.page_size + position % pool.page_size;
                const int len = table.lens[lo] - (fresh.cu[lo + 1] - fresh.cu[lo]);
                if (j * pool.page_size < len && pool.refs[page] > 1 && is_anothers(table, pool, fresh, lo, len, (int)j, page)) {
                    slot = -1;
                    if (t == fresh.cu[lo])
                        atomicAdd(missing, 1);
                }
            }
        }
        fresh.positions[t] = position;
        fresh.slots[t] = slot;
    }
}

__global__ void __launch_bounds__(kPageThreads) extend_kernel(const Table table, int32_t *lens, const Pool pool, const NewTokens fresh,
                                                              int32_t *missing, int32_t *list, int place_here)
{
    extern __shared__ int32_t starts[];      // [rows + 1]: ranks of the rows' new pages
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int each = (table.rows + kPageThreads - 1) / kPageThreads, row0 = threadIdx.x * each;
    // New entries [before, after) of a row.
    auto span = [&](int i, int &before, int &after) {
        const int64_t len = max(lens[i], 0), n = max(fresh.cu[i + 1] - fresh.cu[i], 0);
        before = min(pages_of(len, pool.page_size), table.width);
        after = min(pages_of(len + n, pool.page_size), table.width);
    };
    int n = 0, beyond = 0;                   // pages, and pages behind the table's end
    for (int k = 0; k < each && row0 + k < table.rows; ++k) {
        const int i = row0 + k;
        int before, after;
        span(i, before, after);
        starts[i] = n;                       // (of this thread's rows)
        n += after - before;
        const int64_t len = max(lens[i], 0), grown = len + max(fresh.cu[i + 1] - fresh.cu[i], 0);
        beyond += max(pages_of(grown, pool.page_size), table.width) - max(pages_of(len, pool.page_size), table.width);
    }
    int want, lost;
    const int base = scan_block(n, want);
    (void)scan_block(beyond, lost);
    for (int k = 0; k < each && row0 + k < table.rows; ++k)
        starts[row0 + k] += base;
    if (threadIdx.x == 0)
        starts[table.rows] = want;
    __syncthreads();
    const int have = free_pages(pool, min(want, pool.pages), [&](int r, int page) { list[r] = page; });
    __syncthreads();
    for (int r = threadIdx.x; r < want; r += kPageThreads) {
        int lo = 0, hi = table.rows;         // the last row that begins at r or before
        while (lo + 1 < hi) {
            const int mid = (lo + hi) / 2;
            if (starts[mid] <= r)
                lo = mid;
            else
                hi = mid;
        }
        int before, after;
        span(lo, before, after);
        const int page = r < have ? list[r] : -1;
        table.entries[lo * table.stride + before + r - starts[lo]] = page;
        if (page >= 0)
            pool.refs[page] = 1;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < table.rows; i += kPageThreads)
        lens[i] = max(lens[i], 0) + max(fresh.cu[i + 1] - fresh.cu[i], 0);
    if (threadIdx.x == 0)
        *missing = want - have + lost;
    __syncthreads();
    if (place_here)
        place_tokens(table, pool, fresh, missing, threadIdx.x, kPageThreads);
}

__global__ void __launch_bounds__(256) place_kernel(const Table table, const Pool pool, const NewTokens fresh, int32_t *missing)
{
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    place_tokens(table, pool, fresh, missing, (int)(blockIdx.x * 256 + threadIdx.x), (int)(gridDim.x * 256));
}

// ------------------------------------------------------------------ compact
constexpr int kChunk = 4096;                 // pages of a CTA
constexpr int kChunkThreads = 512, kChunkEach = kChunk / kChunkThreads;

__global__ void __launch_bounds__(kChunkThreads) count_used_kernel(const Pool pool, int32_t *counts)
{
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    int n = 0;
    for (int k = 0; k < kChunkEach; ++k) {
        const int64_t i = (int64_t)blockIdx.x * kChunk + k * kChunkThreads + threadIdx.x;
        n += i < pool.pages && pool.refs[i] != 0;
    }
    int total;
    (void)scan_block(n, total);
    if (threadIdx.x == 0)
        counts[blockIdx.x] = total;
}

// Pages in use before page `end`: whole chunks, then one by one.
__device__ __forceinline__ int used_before(const Pool &pool, const int32_t *counts, int end)
{
    int n = 0, total;
    const int whole = end / kChunk;
    for (int c = threadIdx.x; c < whole; c += kChunkThreads)
        n += counts[c];
    for (int64_t i = (int64_t)whole * kChunk + threadIdx.x; i < end; i += kChunkThreads)
        n += pool.refs[i] != 0;
    (void)scan_block(n, total);
    return total;
}

__global__ void __launch_bounds__(kChunkThreads) rank_pages_kernel(const Pool pool, const int32_t *counts, int32_t *ranks, int32_t *src,
                                                                   int32_t *dst, int32_t *used)
{
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int chunks = (int)gridDim.x;
    int n = 0, total, unused;
    for (int c = threadIdx.x; c < chunks; c += kChunkThreads)
        n += counts[c];
    (void)scan_block(n, total);              // pages in use
    const int stay = used_before(pool, counts, total), moves = total - stay;
    const int before = used_before(pool, counts, (int)blockIdx.x * kChunk);
    const int64_t first = (int64_t)blockIdx.x * kChunk + threadIdx.x * kChunkEach;
    bool full[kChunkEach];
    n = 0;
    for (int k = 0; k < kChunkEach; ++k) {
        full[k] = first + k < pool.pages && pool.refs[first + k] != 0;
        n += full[k];
    }
    int rank = before + scan_block(n, unused);
    for (int k = 0; k < kChunkEach; ++k) {
        const int i = (int)(first + k);
        if (first + k >= pool.pages)
            break;
        if (full[k] && i >= total) {
            ranks[i] = rank - stay;
            src[rank - stay] = i;
        } else if (!full[k] && i < total) {
            dst[i - rank] = i;
        }
        rank += full[k];
    }
    for (int64_t i = moves + (int64_t)blockIdx.x * kChunkThreads + threadIdx.x; i < pool.pages / 2; i += (int64_t)chunks * kChunkThreads)
        src[i] = dst[i] = -1;
    if (blockIdx.x == 0 && threadIdx.x == 0)
        *used = total;
}

// The entries first, first + step, ... of a row, whose pages may have moved.
__device__ __forceinline__ void move_row(const Table &table, const Pool &pool, const int32_t *ranks, const int32_t *src,
                                         const int32_t *dst, int total, int row, int first, int step)
{
    const int n = used_of(table.lens[row], pool, table.width);
    for (int j = first; j < n; j += step) {
        int32_t *e = table.entries + row * table.stride + j;
        // (a page that no count knows has no place to go to)
        if (*e >= total && *e < pool.pages) {
            const int r = ranks[*e];
            if (r >= 0 && r < pool.pages / 2 && src[r] == *e)
                *e = dst[r];
        }
    }
}

// The first `rows` CTAs have a row of the table each, the others the counts of the pages that move.
__global__ void __launch_bounds__(128) move_entries_kernel(const Table table, const Pool pool, const int32_t *ranks, const int32_t *src,
                                                           const int32_t *dst, const int32_t *used)
{
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int row = (int)blockIdx.x;
    if (row < table.rows) {
        move_row(table, pool, ranks, src, dst, *used, row, threadIdx.x, 128);
        return;
    }
    for (int64_t i = (int64_t)(row - table.rows) * 128 + threadIdx.x; i < pool.pages / 2; i += (int64_t)(gridDim.x - table.rows) * 128) {
        const int from = src[i];
        if (from < 0)
            break;
        pool.refs[dst[i]] = pool.refs[from];
        pool.refs[from] = 0;
    }
}

// A small pool and table: all of it by one CTA, whose threads have kHereEach pages each.  us, one launch and three: 8 rows of 25
// on 200 pages 3.5, 6.6; 64 of 64 on 1000 5.1, 7.2; 64 of 128 on 1000 6.7, 7.2, on 2000 7.2, 7.8, on 4000 8.3, 8.9; 96 of 128 on
// 4000 10.0, 9.1; 128 of 256 17.4, 10.0.  Eight pages a thread would take pools of 8000 (32 of 128 9.1, 10.3) and cost the
// others: 200 pages 4.2, 4000 with 64 of 128 9.2.
constexpr int kHereEach = 4, kHerePages = kHereEach * kPageThreads, kHereEntries = 8192;

__global__ void __launch_bounds__(kPageThreads) compact_here_kernel(const Table table, const Pool pool, int32_t *ranks, int32_t *src,
                                                                    int32_t *dst, int32_t *used)
{
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int first = threadIdx.x * kHereEach;
    bool full[kHereEach];
    int n = 0, total, stay;
#pragma unroll
    for (int k = 0; k < kHereEach; ++k) {
        full[k] = first + k < pool.pages && pool.refs[first + k] != 0;
        n += full[k];
    }
    int rank = scan_block(n, total), before = 0;
#pragma unroll
    for (int k = 0; k < kHereEach; ++k)
        before += full[k] && first + k < total;
    (void)scan_block(before, stay);
    const int moves = total - stay;
#pragma unroll
    for (int k = 0; k < kHereEach; ++k) {
        const int i = first + k;
        if (i >= pool.pages)
            break;
        if (full[k] && i >= total) {
            ranks[i] = rank - stay;
            src[rank - stay] = i;
        } else if (!full[k] && i < total) {
            dst[i - rank] = i;
        }
        rank += full[k];
    }
    for (int i = moves + threadIdx.x; i < pool.pages / 2; i += kPageThreads)
        src[i] = dst[i] = -1;
    if (threadIdx.x == 0)
        *used = total;
    __syncthreads();
    for (int row = threadIdx.x >> 5; row < table.rows; row += kPageThreads / 32)
        move_row(table, pool, ranks, src, dst, total, row, threadIdx.x & 31, 32);
    for (int i = threadIdx.x; i < moves; i += kPageThreads) {
        const int from = src[i];
        pool.refs[dst[i]] = pool.refs[from];
        pool.refs[from] = 0;
    }
}

// ------------------------------------------------------------------ copy
constexpr int kSpans = 128;                  // of a launch: 3 KiB of parameters
struct Spans {
    lowm_page_span_t at[kSpans];
};
constexpr int kCopyThreads = 256;

template <typename T>
__device__ __forceinline__ void copy_page(const uint8_t *from, uint8_t *to, int64_t bytes)
{
    const int64_t n = bytes / (int64_t)sizeof(T);
    const T *a = reinterpret_cast<const T *>(from);
    T *b = reinterpret_cast<T *>(to);
    int64_t i = threadIdx.x;
    for (; i + 3 * kCopyThreads < n; i += 4 * kCopyThreads) {
        T x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            x[k] = a[i + k * kCopyThreads];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            b[i + k * kCopyThreads] = x[k];
    }
    for (; i < n; i += kCopyThreads)
        b[i] = a[i];
}

__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ Spans spans, int count, const int32_t *src,
                                                                  const int32_t *dst, int pairs, int num_pages)
{
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    for (int64_t task = blockIdx.x; task < (int64_t)pairs * count; task += gridDim.x) {
        const int i = (int)(task / count);
        const lowm_page_span_t &s = spans.at[task - (int64_t)i * count];
        const int from = src[i], to = dst[i];
        if (from < 0 || from >= num_pages || to < 0 || to >= num_pages || from == to)
            continue;
        const uint8_t *a = static_cast<const uint8_t *>(s.base) + from * s.page_stride;
        uint8_t *b = static_cast<uint8_t *>(s.base) + to * s.page_stride;
        const uintptr_t all = reinterpret_cast<uintptr_t>(s.base) | (uintptr_t)s.page_stride | (uintptr_t)s.page_bytes;
        if (!(all & 15))
            copy_page<uint4>(a, b, s.page_bytes);
        else if (!(all & 3))
            copy_page<uint32_t>(a, b, s.page_bytes);
        else
            copy_page<uint8_t>(a, b, s.page_bytes);
    }
}

bool table_ok(const void *entries, int64_t stride, const void *lens, int rows, int width)
{
    return rows >= 0 && width >= 0 && stride >= 0 && (rows == 0 || (lens && (width == 0 || entries))) &&
           (rows <= 1 || stride >= width);
}

// Whether two tables have memory in common.  (Of tables that lie in one another's range only columns of one buffer are known to
// have none.)
bool tables_meet(const int32_t *a, int64_t a_stride, int a_rows, const int32_t *b, int64_t b_stride, int b_rows, int width)
{
    if (a_rows <= 0 || b_rows <= 0 || width <= 0)
        return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a) / 4, b0 = reinterpret_cast<uintptr_t>(b) / 4;
    const uintptr_t a1 = a0 + (uintptr_t)(a_rows - 1) * a_stride + width, b1 = b0 + (uintptr_t)(b_rows - 1) * b_stride + width;
    if (a1 <= b0 || b1 <= a0)
        return false;
    const uintptr_t stride = a_rows > 1 ? a_stride : b_stride, apart = b0 > a0 ? b0 - a0 : a0 - b0;
    if ((a_rows > 1 && b_rows > 1 && a_stride != b_stride) || stride < (uintptr_t)width)
        return true;
    return apart % stride < (uintptr_t)width || apart % stride + width > stride;
}

}  // namespace
}  // namespace lowm

extern "C" lowm_status_t lowm_fork_pages(const int32_t *page_table, int64_t table_stride, const int32_t *lens, int rows,
                                         const int32_t *parents, int new_rows, int width, int32_t *refs, int num_pages,
                                         int page_size, int32_t *new_table, int64_t new_table_stride, int32_t *new_lens,
                                         int32_t *src, int32_t *dst, int32_t *missing, void *stream)
{
    using namespace lowm;
    if (!table_ok(page_table, table_stride, lens, rows, width) || !table_ok(new_table, new_table_stride, new_lens, new_rows, width) ||
        num_pages <= 0 || page_size <= 0 || !refs || !missing || (new_rows && (!parents || !src || !dst)))
        return LOWM_ERR_INVALID_ARGUMENT;
    if (rows > kMaxRows || new_rows > kMaxRows)
        return LOWM_ERR_UNSUPPORTED_SHAPE;
    const void *all[] = {page_table, lens, parents, refs, new_table, new_lens, src, dst, missing};
    for (const void *x : all)
        if (!is_aligned(x, 4))
            return LOWM_ERR_MISALIGNED;
    if (tables_meet(page_table, table_stride, rows, new_table, new_table_stride, new_rows, width))
        return LOWM_ERR_INVALID_ARGUMENT;
    int sms = 0;
    lowm_status_t st = host_check_device(&sms);
    if (st != LOWM_OK)
        return st;
    const Table old = {const_cast<int32_t *>(page_table), table_stride, lens, rows, width};
    const Table next = {new_table, new_table_stride, new_lens, new_rows, width};
    const Pool pool = {refs, num_pages, page_size};
    const bool few = rows + new_rows <= kFewRows;
    if (!few &&
        (st = launch_pdl(fork_rows_kernel, dim3((unsigned)(rows + new_rows)), dim3(128), 0, stream, old, parents, next, new_lens,
                         pool)) != LOWM_OK)
        return st;
    return launch_pdl(fork_tails_kernel, dim3(1), dim3(kPageThreads), (size_t)new_rows * 4, stream, old, parents, next, new_lens, pool,
                      src, dst, missing, (int)few);
}

extern "C" size_t lowm_extend_pages_workspace(int num_pages) { return num_pages > 0 ? (size_t)num_pages * 4 : 0; }

extern "C" lowm_status_t lowm_extend_pages(int32_t *page_table, int64_t table_stride, int32_t *lens, int rows, int width,
                                           const int32_t *cu_new, int tokens, int32_t *refs, int num_pages, int page_size,
                                           int64_t *positions, int64_t *slots, int32_t *missing, void *workspace,
                                           size_t workspace_bytes, void *stream)
{
    using namespace lowm;
    if (!table_ok(page_table, table_stride, lens, rows, width) || num_pages <= 0 || page_size <= 0 || tokens < 0 || !refs || !missing ||
        (rows && !cu_new) || (tokens && (!positions || !slots)) || !workspace ||
        workspace_bytes < lowm_extend_pages_workspace(num_pages))
        return LOWM_ERR_INVALID_ARGUMENT;
    if (rows > kMaxRows)
        return LOWM_ERR_UNSUPPORTED_SHAPE;
    const void *all[] = {page_table, lens, cu_new, refs, missing, workspace};
    for (const void *x : all)
        if (!is_aligned(x, 4))
            return LOWM_ERR_MISALIGNED;
    if (!is_aligned(positions, 8) || !is_aligned(slots, 8))
        return LOWM_ERR_MISALIGNED;
    int sms = 0;
    lowm_status_t st = host_check_device(&sms);
    if (st != LOWM_OK)
        return st;
    const Table table = {page_table, table_stride, lens, rows, width};
    const Pool pool = {refs, num_pages, page_size};
    const NewTokens fresh = {cu_new, tokens, positions, slots};
    const bool here = tokens <= 4 * kPageThreads;
    st = launch_pdl(extend_kernel, dim3(1), dim3(kPageThreads), (size_t)(rows + 1) * 4, stream, table, lens, pool, fresh, missing,
                    static_cast<int32_t *>(workspace), (int)here);
    if (st == LOWM_OK && !here)
        st = launch_pdl(place_kernel, dim3((unsigned)std::min((tokens + 255) / 256, 8 * sms)), dim3(256), 0, stream, table, pool, fresh,
                        missing);
    return st;
}

extern "C" size_t lowm_compact_pages_workspace(int num_pages)
{
    return num_pages > 0 ? ((size_t)num_pages + (num_pages - 1) / lowm::kChunk + 1) * 4 : 0;
}

extern "C" lowm_status_t lowm_compact_pages(int32_t *page_table, int64_t table_stride, const int32_t *lens, int rows, int width,
                                            int32_t *refs, int num_pages, int page_size, int32_t *src, int32_t *dst, int32_t *used,
                                            void *workspace, size_t workspace_bytes, void *stream)
{
    using namespace lowm;
    if (!table_ok(page_table, table_stride, lens, rows, width) || num_pages <= 0 || page_size <= 0 || !refs || !used ||
        (num_pages > 1 && (!src || !dst)) || !workspace || workspace_bytes < lowm_compact_pages_workspace(num_pages))
        return LOWM_ERR_INVALID_ARGUMENT;
    const void *all[] = {page_table, lens, refs, src, dst, used, workspace};
    for (const void *x : all)
        if (!is_aligned(x, 4))
            return LOWM_ERR_MISALIGNED;
    int sms = 0;
    lowm_status_t st = host_check_device(&sms);
    if (st != LOWM_OK)
        return st;
    const Table table = {page_table, table_stride, lens, rows, width};
    const Pool pool = {refs, num_pages, page_size};
    int32_t *ranks = static_cast<int32_t *>(workspace), *counts = ranks + num_pages;
    if (num_pages <= kHerePages && (int64_t)rows * width <= kHereEntries)
        return launch_pdl(compact_here_kernel, dim3(1), dim3(kPageThreads), 0, stream, table, pool, ranks, src, dst, used);
    const unsigned chunks = (unsigned)((num_pages - 1) / kChunk + 1);
    if ((st = launch_pdl(count_used_kernel, dim3(chunks), dim3(kChunkThreads), 0, stream, pool, counts)) != LOWM_OK ||
        (st = launch_pdl(rank_pages_kernel, dim3(chunks), dim3(kChunkThreads), 0, stream, pool, counts, ranks, src, dst, used)) != LOWM_OK)
        return st;
    const int movers = std::min((num_pages / 2 + 127) / 128, 2 * sms);
    if (rows + movers == 0)
        return LOWM_OK;
    return launch_pdl(move_entries_kernel, dim3((unsigned)(rows + movers)), dim3(128), 0, stream, table, pool, ranks, src, dst, used);
}

extern "C" lowm_status_t lowm_copy_pages(const lowm_page_span_t *spans, int count, const int32_t *src, const int32_t *dst, int pairs,
                                         int num_pages, void *stream)
{
    using namespace lowm;
    if (count < 0 || pairs < 0 || num_pages < 0 || (count && !spans))
        return LOWM_ERR_INVALID_ARGUMENT;
    for (int i = 0; i < count; ++i)
        if (spans[i].page_bytes < 0 || spans[i].page_stride < 0 || (num_pages > 1 && spans[i].page_stride < spans[i].page_bytes) ||
            (!spans[i].base && spans[i].page_bytes))
            return LOWM_ERR_INVALID_ARGUMENT;
    if (count == 0 || pairs == 0 || num_pages == 0)
        return LOWM_OK;
    if (!src || !dst)
        return LOWM_ERR_INVALID_ARGUMENT;
    if (!is_aligned(src, 4) || !is_aligned(dst, 4))
        return LOWM_ERR_MISALIGNED;
    int sms = 0;
    lowm_status_t st = host_check_device(&sms);
    if (st != LOWM_OK)
        return st;
    for (int first = 0; first < count && st == LOWM_OK; first += kSpans) {
        Spans s;
        const int n = std::min(kSpans, count - first);
        std::copy(spans + first, spans + first + n, s.at);
        const int64_t tasks = (int64_t)pairs * n;
        st = launch_pdl(copy_pages_kernel, dim3((unsigned)std::min<int64_t>(tasks, 8 * sms)), dim3(kCopyThreads), 0, stream, s, n, src,
                        dst, pairs, num_pages);
    }
    return st;
}
