// The line of work that the attention kernels over a paged cache cut into equal
// shares (paged_attention.cu, paged_attention_fp8.cu).  An item is a tile of
// rows (a sequence's queries of one key/value head, token by token and head of
// the group by head) and the tiles of 64 keys that any of them sees; all items,
// sequence after sequence, head after head, form the line.
#pragma once

#include <cstdint>

namespace lowm {

constexpr int kTileKeys = 64;
constexpr int kMaxKeys = 1 << 30;            // of a sequence

// What the line follows from.  ROWS: rows of an item; COST: what an item costs
// beside its tiles, in tiles; MINIMUM: tiles of the smallest share.
template <int ROWS, int COST, int MINIMUM>
struct LineParams {
    static constexpr int kRows = ROWS, kCost = COST, kMinimum = MINIMUM;
    const int32_t *kv_lens, *cu_q;
    int batch, q_tokens, kv_heads, group, window;
    int capacity;                            // keys a sequence can have: table_width * page_size
};

// The item that begins in a CTA's share and ends in a later one, for the join.
struct CutItem {
    int parts;                               // shares it lies in; 0: there is none
    int q0, q_len, head, q_tile;
};

// ------------------------------------------------------------------ the line of tiles
struct Item {
    int b, head, q_tile;                     // sequence, key/value head, tile of P::kRows rows
    int q0, q_len, kv;                       // the sequence's first row of q, new tokens, keys
    int first_tile, tiles;                   // tiles of 64 keys
    int start;                               // the item's place on the line: its cost, then its tiles
};

template <class P>
__device__ __forceinline__ void load_sequence(const P &p, int b, int &q0, int &q_len, int &kv)
{
    q0 = min(max(p.cu_q[b], 0), p.q_tokens);
    q_len = min(max(p.cu_q[b + 1], q0), p.q_tokens) - q0;
    kv = min(max(p.kv_lens[b], 0), p.capacity);
}

// Tiles that the rows of row tile q_tile of a sequence see.  Rows that
// see nothing still form one (fully masked) tile, so that they are written.
template <class P>
__device__ __forceinline__ void tile_range(const P &p, int q_len, int kv, int q_tile, int &first, int &tiles)
{
    const int t0 = q_tile * P::kRows / p.group, t1 = min(q_len - 1, (q_tile * P::kRows + P::kRows - 1) / p.group);
    const int hi = max(0, kv - q_len + t1 + 1);
    const int lo = p.window > 0 ? max(0, kv - q_len + t0 - p.window + 1) : 0;
    first = lo < hi ? lo / kTileKeys : 0;
    tiles = lo < hi ? (hi + kTileKeys - 1) / kTileKeys - first : 1;
}

template <class P>
__device__ __forceinline__ int q_tiles_of(const P &p, int q_len)
{
    return (q_len * p.group + P::kRows - 1) / P::kRows;
}

// Units of one key/value head of sequence b (all its row tiles).
template <class P>
__device__ __forceinline__ int head_units(const P &p, int b)
{
    int q0, q_len, kv, first, n, sum = 0;
    load_sequence(p, b, q0, q_len, kv);
    for (int t = 0; t < q_tiles_of(p, q_len); ++t) {
        tile_range(p, q_len, kv, t, first, n);
        sum += n + P::kCost;
    }
    return sum;
}

// The line as one warp sees it: lane l holds the units of a head of sequence l
// and of all heads of sequences 0..l (of the first 32), and everyone the total.
// The host refuses calls whose line could pass 2^31.
struct Line {
    int head, upto, total;
};

__device__ __forceinline__ int scan32(int x)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if ((threadIdx.x & 31) >= o)
            x += y;
    }
    return x;
}

template <class P>
__device__ __forceinline__ Line make_line(const P &p)
{
    const int lane = threadIdx.x & 31;
    Line l;
    l.head = lane < p.batch ? head_units(p, lane) : 0;
    l.upto = scan32(l.head * p.kv_heads);
    l.total = __shfl_sync(0xffffffffu, l.upto, 31);
    if (p.batch > 32) {
        int sum = 0;
        for (int b = 32 + lane; b < p.batch; b += 32)
            sum += head_units(p, b);
        l.total += __reduce_add_sync(0xffffffffu, sum) * p.kv_heads;
    }
    return l;
}

// The item that unit u of the line belongs to (one warp; u below the total).
template <class P>
__device__ __forceinline__ Item locate(const P &p, Line line, int u)
{
    const int lane = threadIdx.x & 31;
    Item it;
    int before = 0;
    for (int b0 = 0;; b0 += 32) {
        const unsigned past = __ballot_sync(0xffffffffu, before + line.upto > u);
        if (past || b0 + 32 >= p.batch) {
            const int l = past ? __ffs(past) - 1 : 31;
            it.b = min(b0 + l, p.batch - 1);
            const int per_head = max(__shfl_sync(0xffffffffu, line.head, l), 1);
            before += __shfl_sync(0xffffffffu, line.upto, l) - per_head * p.kv_heads;
            it.head = (u - before) / per_head;
            it.start = before + it.head * per_head;
            break;
        }
        before += __shfl_sync(0xffffffffu, line.upto, 31);
        line.head = b0 + 32 + lane < p.batch ? head_units(p, b0 + 32 + lane) : 0;
        line.upto = scan32(line.head * p.kv_heads);
    }
    load_sequence(p, it.b, it.q0, it.q_len, it.kv);
    for (it.q_tile = 0;; ++it.q_tile) {
        tile_range(p, it.q_len, it.kv, it.q_tile, it.first_tile, it.tiles);
        if (u < it.start + P::kCost + it.tiles || it.q_tile + 1 >= q_tiles_of(p, it.q_len))
            return it;
        it.start += P::kCost + it.tiles;
    }
}

// The item behind `it` on the line.
template <class P>
__device__ __forceinline__ void advance(const P &p, Item &it)
{
    it.start += P::kCost + it.tiles;
    if (++it.q_tile >= q_tiles_of(p, it.q_len)) {
        it.q_tile = 0;
        if (++it.head == p.kv_heads) {
            it.head = 0;
            do {                             // sequences without new tokens have no items
                ++it.b;
                load_sequence(p, it.b, it.q0, it.q_len, it.kv);
            } while (it.q_len == 0 && it.b + 1 < p.batch);
        }
    }
    tile_range(p, it.q_len, it.kv, it.q_tile, it.first_tile, it.tiles);
}

template <class P>
__device__ __forceinline__ int share_of(const P &, int line, int ctas)
{
    return max((line + ctas - 1) / ctas, P::kMinimum);
}

// A CTA's part of one item: tiles [from, to) of it, at least one.
struct Piece {
    Item it;
    int from, to;
};

template <class P>
__device__ __forceinline__ void cut(const P &, Piece &c, int u, int end)
{
    const int first = c.it.start + P::kCost;          // the item's first tile on the line
    c.from = max(u - first, 0);
    c.to = min(end - first, c.it.tiles);
}

// The first piece of the share [begin, end); false when it has none.
template <class P>
__device__ __forceinline__ bool next_piece(const P &p, Piece &c, int end)
{
    for (;;) {
        const int u = c.it.start + P::kCost + c.it.tiles;
        if (u >= end)
            return false;
        advance(p, c.it);
        cut(p, c, u, end);
        if (c.from < c.to)
            return true;
    }
}

template <class P>
__device__ __forceinline__ bool first_piece(const P &p, Piece &c, const Line &line, int begin, int end)
{
    c.it = locate(p, line, begin);
    cut(p, c, begin, end);
    return c.from < c.to || next_piece(p, c, end);
}

// Row r of the item belongs to token r / group, query head head * group + r % group.
struct Row {
    bool valid;
    int token, q_head;                       // token: index into q
    int hi, lo;                              // keys lo..hi are seen
};

template <class P>
__device__ __forceinline__ Row row_of(const P &p, const Item &it, int r)
{
    Row w;
    const int row = it.q_tile * P::kRows + r;
    const int t = row / p.group;
    w.valid = t < it.q_len;
    w.token = it.q0 + t;
    w.q_head = it.head * p.group + row % p.group;
    w.hi = it.kv - it.q_len + t;
    w.lo = p.window > 0 ? w.hi - p.window + 1 : 0;
    return w;
}

// Keys that all rows of an item see, [all_lo, all_hi] (none when all_lo > all_hi),
// and those that some row sees, [lo, end).
struct Seen {
    int all_lo, all_hi, lo, end;
    __device__ bool mixed() const { return all_hi + 1 < end; }   // the rows' tokens differ, and so do their keys
};

template <class P>
__device__ __forceinline__ Seen seen_by(const P &p, const Item &it)
{
    const int first = it.q_tile * P::kRows / p.group;
    const int last = min(it.q_len - 1, (it.q_tile * P::kRows + P::kRows - 1) / p.group);
    Seen s;
    s.all_hi = it.kv - it.q_len + first;
    s.end = it.kv - it.q_len + last + 1;
    s.all_lo = p.window > 0 ? s.end - p.window : 0;
    s.lo = p.window > 0 ? s.all_hi - p.window + 1 : 0;
    return s;
}

}  // namespace lowm
