// Attention of each sequence's newest tokens over its paged keys and values
// (lowm_layer.h), on the tensor cores.
//
// Work.  The rows of one key/value head are its queries of one sequence, token
// by token and head of the group by head (row = token * group + g), so a key is
// read once for all heads that share it.  An item is up to 128 such rows (one
// MMA M) and the tiles of 64 keys that any of them sees.  All items' tiles,
// sequence after sequence, form one line that is cut into equal shares, one
// for each CTA of a grid of two per SM: a CTA's time does not depend on how
// the lengths are spread over the batch.  The host knows no length; every warp
// finds its share from cu_q and kv_lens by itself.  A share that begins or
// ends inside an item leaves its rows' sum, maximum and weighted values (fp32)
// in the workspace, and a second small kernel joins the parts in order.
//
// A CTA has four softmax warps (a thread owns a row = a TMEM lane), a warp
// that feeds a ring of 64-key tiles by TMA, page by page, and two warps that
// issue the MMAs: S = Q K^T into one of two TMEM buffers, and O += P V with P
// (bf16, written over its S) from TMEM and V as the transposed operand.  The
// second of them, while it waits for P, also clears from V what some rows must
// not meet, weight 0 or not (in the softmax warps 2 to 7 % slower).
// S of the next tile is computed while the softmax of this one runs, and the
// two CTAs of an SM fill each other's gaps.  O is rescaled only when a row's
// maximum has grown by 2^8 (the weights stay below 256, and bf16 and fp32 are
// relative), so most tiles leave O alone.
//
// What bounds it.  Decode: the cache's bandwidth (24 sequences of up to 16384
// keys, 1.0 GB: 157 us, 6.4 TB/s).  Chunks: the MMA issue, the loads and the
// softmax of two CTAs an SM, none of them alone (2048 tokens over 16384 keys: 364
// us, 1.41 PFLOP/s, to 392 from box to box; without the exponentials, with half of
// the loads or with one page for all 3 to 5 % less each; the scores' MMAs of N 64
// read more shared memory than their arithmetic hides).  One CTA an SM with 256
// rows and tiles of 128 keys halves the loads and has MMAs of N 128, but one S for
// each 128 rows: the chain S, softmax, O of one half is not hidden by the other
// (453 us).  Few keys: the chain of launch, schedule, first tile and join (4 x 1000
// keys: 12.6 us).
//
// Rounding: weights meet V in bf16 (the type of the tensor cores' operand);
// their sum, which divides, adds the unrounded fp32 weights.
#include <cuda_bf16.h>
#include <math_constants.h>

#include <algorithm>
#include <climits>

#include "layer_host.h"
#include "layer_device.cuh"

namespace lowm {
namespace {

constexpr int kTileKeys = 64;
constexpr int kTileRows = 128;
constexpr int kAttnThreads = 224;            // softmax warps 0-3, TMA warp 4, MMA warps 5 (Q K^T) and 6 (P V)
constexpr int kMaxAttnCtas = 320;            // two per SM, and a bound for the workspace
constexpr int kMaxKeys = 1 << 30;            // of a sequence
// The line counts time in tiles.  An item costs kItemCost tiles beside its own
// (its queries' way in, its rows' way out); without it the CTAs with short
// items ended 20 % after the others (chunks of 1537 tokens: 209 us at 5, 200 at
// 7, 198.5 at 8, 199.5 at 10, 202 at 12).
constexpr int kItemCost = 8;
// Smaller shares cost more in the join than they save, larger ones wait longer
// (4 x 1000 keys: 13.6 us at 3, 13.2 at 4, 12.6 at 5, 13.2 at 6).
constexpr int kMinShare = 5;
constexpr float kRescaleLog2 = 8.f;
constexpr uint32_t kSColumns = 64;           // one S buffer; P takes its first 32 columns

// Bits of the device status word (above those of the GEMM).
enum : uint32_t {
    kErrAttnRing = 1u << 12,
    kErrAttnFull = 1u << 13,
    kErrAttnScores = 1u << 14,
    kErrAttnWeights = 1u << 15,
    kErrAttnOutput = 1u << 16,
    kErrAttnBase = 1u << 17,                 // dynamic shared memory not on a 1024-byte boundary
};

struct AttnParams {
    const __nv_bfloat16 *q, *k, *v;
    __nv_bfloat16 *out;
    float *lse;
    int64_t q_ts, q_hs, o_ts, o_hs, table_stride, num_pages;
    int64_t k_page, k_place, k_head, v_page, v_place, v_head;
    const int32_t *table, *kv_lens, *cu_q;
    int page_size, page_shift, batch, q_tokens, heads, kv_heads, group, window, slot_rows;
    int capacity;                            // keys a sequence can have: table_width * page_size
    float scale_log2;                        // |scale| * log2(e); the sign is in Q
    float q_sign;
    bool q_vec, out_vec;                     // 16-byte rows
    float4 *parts;                           // [2 * ctas][dim / 4][slot_rows] sums, rows side by side as the lanes hold
                                             // them, then [2 * ctas][slot_rows] (max, sum) pairs
    struct CutItem *cuts;                    // [ctas]
    unsigned int *status;
};

// The item that begins in a CTA's share and ends in a later one, for the join.
struct CutItem {
    int parts;                               // shares it lies in; 0: there is none
    int q0, q_len, head, q_tile;
};

// ------------------------------------------------------------------ the line of tiles
struct Item {
    int b, head, q_tile;                     // sequence, key/value head, tile of 128 rows
    int q0, q_len, kv;                       // the sequence's first row of q, new tokens, keys
    int first_tile, tiles;                   // tiles of 64 keys
    int start;                               // the item's place on the line: kItemCost units, then its tiles
};

__device__ __forceinline__ void load_sequence(const AttnParams &p, int b, int &q0, int &q_len, int &kv)
{
    q0 = min(max(p.cu_q[b], 0), p.q_tokens);
    q_len = min(max(p.cu_q[b + 1], q0), p.q_tokens) - q0;
    kv = min(max(p.kv_lens[b], 0), p.capacity);
}

// Tiles that rows [128 q_tile, 128 q_tile + 128) of a sequence see.  Rows that
// see nothing still form one (fully masked) tile, so that they are written.
__device__ __forceinline__ void tile_range(const AttnParams &p, int q_len, int kv, int q_tile, int &first, int &tiles)
{
    const int t0 = q_tile * kTileRows / p.group, t1 = min(q_len - 1, (q_tile * kTileRows + kTileRows - 1) / p.group);
    const int hi = max(0, kv - q_len + t1 + 1);
    const int lo = p.window > 0 ? max(0, kv - q_len + t0 - p.window + 1) : 0;
    first = lo < hi ? lo / kTileKeys : 0;
    tiles = lo < hi ? (hi + kTileKeys - 1) / kTileKeys - first : 1;
}

__device__ __forceinline__ int q_tiles_of(const AttnParams &p, int q_len)
{
    return (q_len * p.group + kTileRows - 1) / kTileRows;
}

// Units of one key/value head of sequence b (all its row tiles).
__device__ __forceinline__ int head_units(const AttnParams &p, int b)
{
    int q0, q_len, kv, first, n, sum = 0;
    load_sequence(p, b, q0, q_len, kv);
    for (int t = 0; t < q_tiles_of(p, q_len); ++t) {
        tile_range(p, q_len, kv, t, first, n);
        sum += n + kItemCost;
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

__device__ __forceinline__ Line make_line(const AttnParams &p)
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
__device__ __forceinline__ Item locate(const AttnParams &p, Line line, int u)
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
        if (u < it.start + kItemCost + it.tiles || it.q_tile + 1 >= q_tiles_of(p, it.q_len))
            return it;
        it.start += kItemCost + it.tiles;
    }
}

// The item behind `it` on the line.
__device__ __forceinline__ void advance(const AttnParams &p, Item &it)
{
    it.start += kItemCost + it.tiles;
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

__device__ __forceinline__ int share_of(int line, int ctas)
{
    return max((line + ctas - 1) / ctas, kMinShare);
}

// A CTA's part of one item: tiles [from, to) of it, at least one.
struct Piece {
    Item it;
    int from, to;
};

__device__ __forceinline__ void cut(Piece &c, int u, int end)
{
    const int first = c.it.start + kItemCost;          // the item's first tile on the line
    c.from = max(u - first, 0);
    c.to = min(end - first, c.it.tiles);
}

// The first piece of the share [begin, end); false when it has none.
__device__ __forceinline__ bool next_piece(const AttnParams &p, Piece &c, int end)
{
    for (;;) {
        const int u = c.it.start + kItemCost + c.it.tiles;
        if (u >= end)
            return false;
        advance(p, c.it);
        cut(c, u, end);
        if (c.from < c.to)
            return true;
    }
}

__device__ __forceinline__ bool first_piece(const AttnParams &p, Piece &c, const Line &line, int begin, int end)
{
    c.it = locate(p, line, begin);
    cut(c, begin, end);
    return c.from < c.to || next_piece(p, c, end);
}

// ------------------------------------------------------------------ PTX of this kernel
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 values in one register pair: one instruction for both.
__device__ __forceinline__ uint64_t pack2(float x, float y)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}

__device__ __forceinline__ uint64_t pack2(uint32_t x, uint32_t y)
{
    return pack2(__uint_as_float(x), __uint_as_float(y));
}

__device__ __forceinline__ float2 unpack2(uint64_t v)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void *tmap, int x, int y, int z, int w, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}

// D[tmem] (+)= A[tmem] . B[smem desc], bf16 operands, fp32 accumulator.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_ld_x32(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_st_x32(uint32_t taddr, const uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

// Descriptor of V as the MMA's B operand, N (the head's elements) contiguous:
// 128-byte swizzled atoms of 64 elements x 8 keys; the leading offset leads to
// the next 64 elements, the stride offset to the next 8 keys.
__device__ __forceinline__ uint64_t make_sw128_nmajor_desc(uint32_t saddr, uint32_t next_64)
{
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(next_64 >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// ------------------------------------------------------------------ shared memory
template <int DIM>
struct AttnSmem {
    static constexpr uint32_t kHalves = DIM / 64;                       // 128-byte wide pieces of a row
    static constexpr uint32_t kQ = 0;                                   // [halves][128 rows][64]
    static constexpr uint32_t kTileBytes = kTileKeys * DIM * 2;
    static constexpr uint32_t kRing = kTileRows * DIM * 2;              // [stages][halves][64 keys][64]
    static constexpr uint32_t kStages = DIM == 128 ? 5 : 10;            // 80 KiB: two CTAs fill an SM's 227 KiB
    // A wait for a full stage passes too early when the load before it in that stage has not landed yet: the
    // barrier's parity is then still that of the phase before.  Loads (K0, K1, V0, K2, V1, ..., V of the last tile, then
    // the next item's) may land in any order, so it must follow from what the waiting warp has seen.  At K of tile g
    // that is K up to g - 1 and, by the O of g - 3, V up to there: not V of g - 1 and g - 2, which are among the three
    // loads before.  At V of tile g it is V up to g - 1 and, by the weights of g - 1, K up to there: not K of g and
    // g + 1, among the three loads before as well.
    static_assert(kStages >= 4, "a warp would wait for a stage whose previous load may be under way");
    static constexpr uint32_t kBars = kRing + kStages * kTileBytes;     // full, empty [stages]; q; s, p, o [2]; edges; drain
    static constexpr uint32_t kNumBars = 2 * kStages + 9;
    static constexpr uint32_t kSlot = kBars + kNumBars * 8;             // TMEM address, edge word
    static constexpr uint32_t kBytes = kSlot + 16;                      // 112.2 KiB: two CTAs an SM
};

// Row r of the item belongs to token r / group, query head head * group + r % group.
struct Row {
    bool valid;
    int token, q_head;                       // token: index into q
    int hi, lo;                              // keys lo..hi are seen
};

__device__ __forceinline__ Row row_of(const AttnParams &p, const Item &it, int r)
{
    Row w;
    const int row = it.q_tile * kTileRows + r;
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

__device__ __forceinline__ Seen seen_by(const AttnParams &p, const Item &it)
{
    const int first = it.q_tile * kTileRows / p.group;
    const int last = min(it.q_len - 1, (it.q_tile * kTileRows + kTileRows - 1) / p.group);
    Seen s;
    s.all_hi = it.kv - it.q_len + first;
    s.end = it.kv - it.q_len + last + 1;
    s.all_lo = p.window > 0 ? s.end - p.window : 0;
    s.lo = p.window > 0 ? s.all_hi - p.window + 1 : 0;
    return s;
}

template <int DIM>
__device__ __forceinline__ void store_row(const AttnParams &p, const Row &w, int col, const float (&v)[32])
{
    __nv_bfloat16 *o = p.out + w.token * p.o_ts + w.q_head * p.o_hs + col;
    if (p.out_vec) {
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
            uint4 u;
            __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&u);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                h[j] = __floats2bfloat162_rn(v[i + 2 * j], v[i + 2 * j + 1]);
            *reinterpret_cast<uint4 *>(o + i) = u;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            o[i] = __float2bfloat16_rn(v[i]);
    }
}

constexpr int kCleanKeys = 16;                       // looked at at once: all loads before the first use

// x * 0 + sum for two bf16: 0 while x is finite, else NaN.
__device__ __forceinline__ uint32_t times_zero(uint32_t x, uint32_t sum)
{
    asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(sum) : "r"(x), "r"(0u));
    return sum;
}

// Clears the values that are not finite of this lane's part of 16 keys from
// `key` on, where only some rows see them.
template <int DIM>
__device__ __noinline__ void take_out(uint4 *at, const Seen &seen, int key)
{
    key += (threadIdx.x & 31) >> 3;
#pragma unroll 1
    for (int i = 0; i < kCleanKeys / 4; ++i, key += 4)
#pragma unroll 1
        for (int half = 0; half < DIM / 64; ++half) {
            if (key >= seen.all_lo && key <= seen.all_hi)
                continue;
            uint32_t *words = reinterpret_cast<uint32_t *>(at + half * (kTileKeys * 8) + i * 32);
#pragma unroll 1
            for (int w = 0; w < 4; ++w) {
                const uint32_t sign = ((words[w] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;   // exponent all ones
                words[w] &= ~(sign | (sign - (sign >> 15)));                                    // and the 15 bits below
            }
        }
}

// Makes a tile of V (keys key0.., 128-byte swizzled) fit to meet the weights of
// all rows, by one warp: a weight of 0 does not silence what is not finite.  Keys
// that no row of the item sees may hold anything (the rest of a sequence's last
// page, pages that a window has left behind) and are cleared.  Of keys that some
// rows see and others do not, the values that are not finite are taken out, to be
// added to the rows that see them at the item's end; true when there were any.
template <int DIM>
__device__ __forceinline__ bool clean_values(uint8_t *tile, const Seen &seen, int key0)
{
    const int lane = threadIdx.x & 31;
    uint32_t found = 0;
#pragma unroll 1
    for (int k0 = 0; k0 < kTileKeys; k0 += kCleanKeys) {
        if (key0 + k0 >= seen.all_lo && key0 + k0 + kCleanKeys - 1 <= seen.all_hi)
            continue;
        uint4 *at = reinterpret_cast<uint4 *>(tile + k0 * 128) + lane;   // 4 keys of 64 elements a step
        uint4 x[kCleanKeys / 4][DIM / 64];
#pragma unroll
        for (int i = 0; i < kCleanKeys / 4; ++i)
#pragma unroll
            for (int half = 0; half < DIM / 64; ++half)
                x[i][half] = at[half * (kTileKeys * 8) + i * 32];
        uint32_t bad = 0;
#pragma unroll
        for (int i = 0; i < kCleanKeys / 4; ++i) {
            const int key = key0 + k0 + 4 * i + (lane >> 3);
            uint32_t here = 0;                       // stays 0 (or -0) while all are finite
#pragma unroll
            for (int half = 0; half < DIM / 64; ++half) {
                here = times_zero(x[i][half].x, here);
                here = times_zero(x[i][half].y, here);
                here = times_zero(x[i][half].z, here);
                here = times_zero(x[i][half].w, here);
            }
            if (key < seen.lo || key >= seen.end) {
#pragma unroll
                for (int half = 0; half < DIM / 64; ++half)
                    at[half * (kTileKeys * 8) + i * 32] = make_uint4(0, 0, 0, 0);
            } else if (key < seen.all_lo || key > seen.all_hi) {
                bad |= here & 0x7fff7fffu;
            }
        }
        if (bad)
            take_out<DIM>(at, seen, key0 + k0);
        found |= bad;
    }
    ptx::fence_proxy_async_shared();
    return __any_sync(0xffffffffu, found != 0);
}

// Adds the values that are not finite of keys that only some rows of the item
// see, which were taken out of V for the MMA: for each row of this warp whose bit
// is set in `rows`, those of the keys key_begin..key_end - 1 that it sees, times
// their weight (2^(score - shift), in bf16 as in the MMA) and `factor`, onto `out`
// or the row's part.  The whole warp is on a row.  An item has at most 128 tokens,
// so these keys are among the last 127 that a row sees, or the first 127 of its
// window; among them are keys that all rows see, whose infinities are in O already
// and change nothing a second time.  A warp's 32 rows take some milliseconds at
// worst, whatever the lengths (3 ms an item with nothing but NaN in V): far below
// the limit of the other warps' waits.
template <int DIM>
__device__ __noinline__ void add_edge_values(const AttnParams &p, unsigned rows, int sequence, const Row &mine, int key_begin,
                                             int key_end, float shift, float factor, int64_t slot, int r)
{
    constexpr int E = DIM / 32;
    const int lane = threadIdx.x & 31, r0 = r - lane;
    __syncwarp();
    while (rows) {
        const int l = __ffs(rows) - 1;
        rows &= rows - 1;
        const int token = __shfl_sync(0xffffffffu, mine.token, l), head = __shfl_sync(0xffffffffu, mine.q_head, l);
        const int lo = __shfl_sync(0xffffffffu, mine.lo, l), hi = __shfl_sync(0xffffffffu, mine.hi, l);
        const float base = __shfl_sync(0xffffffffu, shift, l), f = __shfl_sync(0xffffffffu, factor, l);
        const int g = head / p.group;
        float acc[E] = {};
        bool any = false;
        const int first_end = p.window > 0 ? lo + kTileRows - 2 : -1, last_begin = max(lo, hi - kTileRows + 2);
#pragma unroll 1
        for (int key = max(max(lo, 0), key_begin); key <= hi && key < key_end; ++key) {
            if (key > first_end && key < last_begin) {
                key = last_begin - 1;
                continue;
            }
            const int64_t page = p.table[sequence * p.table_stride + (key >> p.page_shift)];
            const int64_t place = key & (p.page_size - 1);
            if (page < 0 || page >= p.num_pages)     // reads as zeros
                continue;
            float v[E];
            bool bad = false;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                v[e] = __bfloat162float(p.v[page * p.v_page + place * p.v_place + g * p.v_head + lane * E + e]);
                bad = bad || !(fabsf(v[e]) < CUDART_INF_F);
            }
            if (!__any_sync(0xffffffffu, bad))
                continue;
            any = true;
            float s = 0.f;
            for (int e = 0; e < E; ++e)
                s = fmaf(__bfloat162float(p.q[token * p.q_ts + head * p.q_hs + lane * E + e]),
                         __bfloat162float(p.k[page * p.k_page + place * p.k_place + g * p.k_head + lane * E + e]), s);
            for (int o = 16; o > 0; o >>= 1)
                s += __shfl_xor_sync(0xffffffffu, s, o);
            // (a weight too small for a float still carries an infinity)
            const float a = s == -p.q_sign * CUDART_INF_F
                                ? 0.f
                                : fmaxf(__bfloat162float(__float2bfloat16_rn(ex2(fmaf(p.q_sign * s, p.scale_log2, -base)))), 1e-30f);
            for (int e = 0; e < E; ++e)
                if (!(fabsf(v[e]) < CUDART_INF_F))
                    acc[e] = fmaf(a, v[e], acc[e]);
        }
        for (int e = 0; e < E && any; ++e) {
            const int d = lane * E + e;
            if (slot < 0) {
                __nv_bfloat16 *o = p.out + token * p.o_ts + head * p.o_hs + d;
                *o = __float2bfloat16_rn(fmaf(acc[e], f, __bfloat162float(*o)));
            } else {
                reinterpret_cast<float *>(p.parts + (slot * (DIM / 4) + d / 4) * p.slot_rows + r0 + l)[d & 3] += acc[e];
            }
        }
    }
}

template <int DIM>
__global__ void __launch_bounds__(kAttnThreads, 2)
    paged_attention_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                           const AttnParams p)
{
    using L = AttnSmem<DIM>;
    constexpr uint32_t kColumns = 256;       // two S buffers and O (192 or 256 columns), a power of two
    constexpr uint32_t kOColumn = 2 * kSColumns;
    // The swizzle repeats every 1024 bytes, so the base must be a multiple; rounding it up at run time
    // would cost the KiB that the second CTA of the SM needs.
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = ptx::smem_u32(smem);
    const uint32_t bar_full = sbase + L::kBars, bar_empty = bar_full + 8 * L::kStages;
    const uint32_t bar_q = bar_empty + 8 * L::kStages, bar_s = bar_q + 8, bar_p = bar_s + 16, bar_o = bar_p + 16,
                   bar_edges = bar_o + 16, bar_drain = bar_edges + 8;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (sbase & 1023u) {
        if (threadIdx.x == 0)
            atomicOr(p.status, kErrAttnBase);
        return;
    }

    if (threadIdx.x == 0) {
        for (uint32_t s = 0; s < L::kStages; ++s) {
            ptx::mbar_init(bar_full + 8 * s, 1);
            ptx::mbar_init(bar_empty + 8 * s, 1);
        }
        ptx::mbar_init(bar_q, 4);                // softmax warps
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(bar_s + 8 * i, 1);
            ptx::mbar_init(bar_p + 8 * i, 4);
            ptx::mbar_init(bar_o + 8 * i, 1);
        }
        ptx::mbar_init(bar_edges, 1);
        ptx::mbar_init(bar_drain, 2);
        ptx::fence_mbarrier_init_cluster();
        ptx::fence_proxy_async_shared();
    }
    if (warp == 5) {
        ptx::tmem_alloc(sbase + L::kSlot, kColumns);
        ptx::tmem_relinquish_alloc_permit();
        ptx::tcgen05_fence_before_thread_sync();
    }
    __syncthreads();
    ptx::tcgen05_fence_after_thread_sync();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + L::kSlot);

    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    const Line line = make_line(p);
    const int share = share_of(line.total, gridDim.x);
    const int begin = (int)min((int64_t)share * blockIdx.x, (int64_t)line.total), end = min(share, line.total - begin) + begin;

    if (threadIdx.x == 0)
        p.cuts[blockIdx.x].parts = 0;        // until this thread finds one
    Piece c;
    if (begin < end && first_piece(p, c, line, begin, end)) {
        const Item &it = c.it;
        if (warp == 4) {
            // -------------------------------------------------------- TMA: K0, K1, V0, K2, V1, ...
            const int box_keys = min(p.page_size, kTileKeys), boxes = kTileKeys / box_keys;
            const int mine = lane / (int)L::kHalves, half = lane % (int)L::kHalves;   // this lane's box and half
            uint32_t i = 0;
            bool ok = true;
            do {
                const int from = c.from, n = c.to - c.from;
                const int32_t *pages = p.table + it.b * p.table_stride;
                // Table entries of this lane's box for the newest K tile and the V tile behind it.
                auto entry = [&](int tile) {
                    const int key = (it.first_tile + tile) * kTileKeys + mine * box_keys;
                    return mine < boxes && key < it.kv ? pages[key >> p.page_shift] : -1;
                };
                int page_k = entry(from), page_v = page_k, page_next = n > 1 ? entry(from + 1) : -1;
                auto load = [&](const CUtensorMap *map, int tile, int page) {
                    const uint32_t s = i % L::kStages;
                    if (ok && !wait_short(bar_empty + 8 * s, ((i / L::kStages) & 1) ^ 1)) {
                        ok = false;
                        atomicOr(p.status, kErrAttnRing);
                    }
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok)
                        return;
                    const int key0 = (it.first_tile + tile) * kTileKeys;
                    // Pages past the sequence's end are not requested.
                    const int used = min(boxes, max(1, (it.kv - key0 + box_keys - 1) / box_keys));
                    if (lane == 0)
                        ptx::mbar_arrive_expect_tx(bar_full + 8 * s, (uint32_t)used * box_keys * DIM * 2);
                    __syncwarp();
                    if (mine < used)
                        tma_load_4d(sbase + L::kRing + s * L::kTileBytes + half * (kTileKeys * 128) + mine * box_keys * 128,
                                    map, half * 64, key0 & (p.page_size - 1), it.head, page, bar_full + 8 * s);
                    ++i;
                };
                load(&map_k, from, page_k);
                for (int j = 0; j < n; ++j) {
                    page_v = page_k;
                    if (j + 1 < n) {
                        page_k = page_next;
                        if (j + 2 < n)
                            page_next = entry(from + j + 2);
                        load(&map_k, from + j + 1, page_k);
                    }
                    load(&map_v, from + j, page_v);
                }
            } while (ok && next_piece(p, c, end));
            // No copy may land after the CTA has ended: normally all were consumed long ago.
            for (uint32_t j = i > L::kStages ? i - L::kStages : 0; j < i; ++j)
                (void)wait_short(bar_full + 8 * (j % L::kStages), (j / L::kStages) & 1);
        } else if (warp >= 5) {
            // -------------------------------------------------------- MMA: one warp for S, one for O
            // A tile's 12 MMAs, 4 commits and 3 waits in one thread took 2100
            // cycles, more than its softmax; two run them side by side.  The warps
            // stay converged and elect the issuing thread, and the compiler knows
            // that the operands are the same in all lanes: from a branch for lane 0
            // the 8 MMAs of S took 765 cycles to issue, this way 580 (2048 tokens over
            // 16384 keys: 395 -> 364 us).
            constexpr uint32_t kIdescS = make_idesc_bf16(kTileRows, kTileKeys);
            constexpr uint32_t kIdescO = make_idesc_bf16(kTileRows, DIM) | (1u << 16);   // B: N contiguous
            const bool first = uniform(warp) == 5;
            const uint32_t base = uniform(tmem);
            uint32_t i = 0, g = 0, items = 0;                           // ring stages passed, tiles, items
            bool ok = true;
            auto wait = [&](uint32_t bar, uint32_t parity, uint32_t err) {
                if (!wait_short(bar, parity)) {
                    ok = false;
                    atomicOr(p.status, err);
                }
                ok = __all_sync(0xffffffffu, ok);
            };
            do {
                const int n = uniform(c.to - c.from);
                if (first) {
                    wait(bar_q, items & 1, kErrAttnWeights);
                    for (int j = 0; j < n && ok; ++j, ++g) {            // S[g & 1] = Q . K^T
                        const uint32_t at = i + (j == 0 ? 0 : 2 * j - 1), s = at % L::kStages;
                        wait(bar_full + 8 * s, (at / L::kStages) & 1, kErrAttnFull);
                        if (g > 1)                                      // the weights that lay there have met V
                            wait(bar_o + 8 * (g & 1), ((g >> 1) & 1) ^ 1, kErrAttnOutput);
                        ptx::tcgen05_fence_after_thread_sync();
                        if (!ok)
                            break;
                        const uint64_t a0 = make_sw128_kmajor_desc(sbase + L::kQ);
                        const uint64_t b0 = make_sw128_kmajor_desc(sbase + L::kRing + s * L::kTileBytes);
                        if (ptx::elect_one_sync()) {
#pragma unroll
                            for (uint32_t k = 0; k < 4 * L::kHalves; ++k)
                                ptx::mma_bf16_ss(base + (g & 1) * kSColumns, a0 + (k >> 2) * (kTileRows * 8) + 2 * (k & 3),
                                                 b0 + (k >> 2) * (kTileKeys * 8) + 2 * (k & 3), kIdescS, k > 0);
                            ptx::tcgen05_commit(bar_s + 8 * (g & 1));
                            ptx::tcgen05_commit(bar_empty + 8 * s);
                        }
                        __syncwarp();
                    }
                } else {
                    const Seen seen = seen_by(p, c.it);
                    bool edges = false;
                    for (int j = 0; j < n && ok; ++j, ++g) {            // O (+)= P . V
                        const uint32_t at = i + (j + 1 < n ? 2 * j + 2 : 2 * j + 1), s = at % L::kStages;
                        wait(bar_full + 8 * s, (at / L::kStages) & 1, kErrAttnFull);
                        // (while the softmax warps are at the tile's weights)
                        const int key0 = (c.it.first_tile + c.from + j) * kTileKeys;
                        if (ok && (key0 < seen.all_lo || key0 + kTileKeys - 1 > seen.all_hi))
                            edges |= clean_values<DIM>(smem + L::kRing + s * L::kTileBytes, seen, key0);
                        wait(bar_p + 8 * (g & 1), (g >> 1) & 1, kErrAttnWeights);
                        ptx::tcgen05_fence_after_thread_sync();
                        if (!ok)
                            break;
                        const uint64_t b0 = make_sw128_nmajor_desc(sbase + L::kRing + s * L::kTileBytes, kTileKeys * 128);
                        if (ptx::elect_one_sync()) {
#pragma unroll
                            for (uint32_t k = 0; k < kTileKeys / 16; ++k)    // 16 keys: 2 KiB of V, 8 columns of P
                                mma_bf16_ts(base + kOColumn, base + (g & 1) * kSColumns + 8 * k, b0 + 128 * k, kIdescO,
                                            j > 0 || k > 0);
                            ptx::tcgen05_commit(bar_o + 8 * (g & 1));
                            ptx::tcgen05_commit(bar_empty + 8 * s);
                        }
                        __syncwarp();
                    }
                    if (ok && lane == 0) {
                        *reinterpret_cast<volatile uint32_t *>(smem + L::kSlot + 4) = edges;
                        ptx::mbar_arrive(bar_edges);
                    }
                    __syncwarp();
                }
                i += 2 * n;
                ++items;
            } while (ok && uniform(next_piece(p, c, end)));
            if (ptx::elect_one_sync())
                ptx::tcgen05_commit(bar_drain);
            __syncwarp();
            (void)wait_short(bar_drain, 0);                             // nothing reads or writes TMEM any more
        } else {
            // -------------------------------------------------------- softmax: thread = row = TMEM lane
            const uint32_t lane_base = tmem + ((uint32_t)(32 * warp) << 16);
            const int r = threadIdx.x;
            uint32_t g = 0, items = 0;
            bool ok = true;
            auto wait = [&](uint32_t bar, uint32_t parity, uint32_t err) {
                if (!wait_short(bar, parity)) {
                    ok = false;
                    atomicOr(p.status, err);
                }
                ok = __all_sync(0xffffffffu, ok);
                ptx::tcgen05_fence_after_thread_sync();
            };
            // A warp's 32 rows of Q into the swizzled K-major tile (16-byte chunk c of
            // row r at c ^ (r & 7)), a row's chunks by neighbouring lanes, all loads
            // before the first store.
            auto load_q = [&](const Item &item) {
                constexpr int kChunks = DIM / 8, kRowsAtOnce = 32 / kChunks, kLoads = 32 / kRowsAtOnce;
                const Row row = row_of(p, item, r);
                const int64_t at = row.valid ? row.token * p.q_ts + row.q_head * p.q_hs : -1;
                const uint32_t flip = p.q_sign < 0.f ? 0x80008000u : 0u;
                const int c = lane % kChunks, q0 = lane / kChunks;
                uint4 x[kLoads];
                if (p.q_vec) {
#pragma unroll
                    for (int i = 0; i < kLoads; ++i) {
                        const int64_t from = __shfl_sync(0xffffffffu, at, i * kRowsAtOnce + q0);
                        x[i] = from >= 0 ? *reinterpret_cast<const uint4 *>(p.q + from + 8 * c) : make_uint4(0, 0, 0, 0);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < kLoads; ++i) {
                        const int64_t from = __shfl_sync(0xffffffffu, at, i * kRowsAtOnce + q0);
                        __nv_bfloat16 *e = reinterpret_cast<__nv_bfloat16 *>(&x[i]);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            e[j] = from >= 0 ? p.q[from + 8 * c + j] : __float2bfloat16_rn(0.f);
                    }
                }
#pragma unroll
                for (int i = 0; i < kLoads; ++i) {
                    const int q = i * kRowsAtOnce + q0;
                    *reinterpret_cast<uint4 *>(smem + L::kQ + (c >> 3) * (kTileRows * 128) + (32 * warp + q) * 128 +
                                               (((c & 7) ^ (q & 7)) << 4)) =
                        make_uint4(x[i].x ^ flip, x[i].y ^ flip, x[i].z ^ flip, x[i].w ^ flip);
                }
                ptx::fence_proxy_async_shared();
                ptx::tcgen05_fence_before_thread_sync();
                __syncwarp();
                if (lane == 0)
                    ptx::mbar_arrive(bar_q);
            };
            load_q(it);
            for (bool more = true; more;) {
                const int from = c.from, n = c.to - c.from;
                const Row w = row_of(p, it, r);
                const bool warp_has_rows = __any_sync(0xffffffffu, w.valid);
                const Seen seen = seen_by(p, it);
                const int all_lo = seen.all_lo, all_hi = seen.all_hi;   // no mask inside
                float m = -CUDART_INF_F, l = 0.f;                       // maximum (raw score) and sum of this row
                for (int j = 0; j < n; ++j, ++g) {
                    wait(bar_s + 8 * (g & 1), (g >> 1) & 1, kErrAttnScores);
                    if (!ok)
                        break;
                    const int key0 = (it.first_tile + from + j) * kTileKeys;
                    uint32_t s0[32], s1[32];
                    const uint32_t s_addr = lane_base + (g & 1) * kSColumns;
                    if (warp_has_rows) {
                        tmem_ld_x32(s_addr, s0);
                        tmem_ld_x32(s_addr + 32, s1);
                        ptx::tmem_wait_ld();
                        if (key0 < all_lo || key0 + kTileKeys - 1 > all_hi) {
                            const int hi = w.valid ? w.hi - key0 : -1, lo = w.lo - key0;
#pragma unroll
                            for (int k = 0; k < 32; ++k) {
                                if (k > hi || k < lo)
                                    s0[k] = 0xff800000u;
                                if (k + 32 > hi || k + 32 < lo)
                                    s1[k] = 0xff800000u;
                            }
                        }
                        float t[4] = {m, m, m, m};
#pragma unroll
                        for (int k = 0; k < 32; k += 4)
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                t[c] = fmaxf(fmaxf(t[c], __uint_as_float(s0[k + c])), __uint_as_float(s1[k + c]));
                        const float top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
                        if (j == 0) {
                            m = top;
                        } else if (__any_sync(0xffffffffu, (top - m) * p.scale_log2 > kRescaleLog2)) {
                            // O of the tiles so far is complete once PV of the previous tile is.
                            wait(bar_o + 8 * ((g - 1) & 1), ((g - 1) >> 1) & 1, kErrAttnOutput);
                            if (!ok)
                                break;
                            const float a = m == top ? 1.f : ex2((m - top) * p.scale_log2);
                            l *= a;
                            m = top;
#pragma unroll
                            for (int c = 0; c < DIM; c += 8) {
                                uint32_t o[8];
                                ptx::tmem_ld_32x32b_x8(lane_base + kOColumn + c, o);
                                ptx::tmem_wait_ld();
#pragma unroll
                                for (int k = 0; k < 8; ++k)
                                    o[k] = __float_as_uint(__uint_as_float(o[k]) * a);
                                ptx::tmem_st_32x32b_x8(lane_base + kOColumn + c, o);
                            }
                        }
                        const float ms = m == -CUDART_INF_F ? 0.f : m * p.scale_log2;
                        const uint64_t scale2 = pack2(p.scale_log2, p.scale_log2), shift2 = pack2(-ms, -ms);
                        uint64_t sum0 = 0, sum1 = 0;
                        uint32_t pk[32];
#pragma unroll
                        for (int k = 0; k < 32; k += 2) {
                            const float2 x = unpack2(fma2(pack2(s0[k], s0[k + 1]), scale2, shift2));
                            const float2 y = unpack2(fma2(pack2(s1[k], s1[k + 1]), scale2, shift2));
                            const float a = ex2(x.x), b = ex2(x.y), c = ex2(y.x), d = ex2(y.y);
                            sum0 = add2(sum0, pack2(a, b));
                            sum1 = add2(sum1, pack2(c, d));
                            const __nv_bfloat162 ab = __floats2bfloat162_rn(a, b), cd = __floats2bfloat162_rn(c, d);
                            pk[k / 2] = *reinterpret_cast<const uint32_t *>(&ab);
                            pk[16 + k / 2] = *reinterpret_cast<const uint32_t *>(&cd);
                        }
                        const float2 sums = unpack2(add2(sum0, sum1));
                        l += sums.x + sums.y;
                        tmem_st_x32(s_addr, pk);
                        ptx::tmem_wait_st();
                    }
                    ptx::tcgen05_fence_before_thread_sync();
                    __syncwarp();
                    if (lane == 0)
                        ptx::mbar_arrive(bar_p + 8 * (g & 1));
                }
                if (!ok)
                    break;
                // The next item's queries before this one's rows: every S of this one is complete, and the
                // first products of the next run while its rows are written.
                const bool whole = n == it.tiles;
                const int64_t slot = 2 * (int64_t)blockIdx.x + (from == 0 ? 1 : 0);
                if (r == 0 && from == 0 && !whole)
                    p.cuts[blockIdx.x] = {(it.start + kItemCost + it.tiles - 1) / share - (int)blockIdx.x + 1, it.q0, it.q_len,
                                          it.head, it.q_tile};
                const int sequence = it.b, key_begin = (it.first_tile + from) * kTileKeys, key_end = key_begin + n * kTileKeys;
                const bool mixed = seen.mixed();
                more = next_piece(p, c, end);
                if (more)
                    load_q(it);
                wait(bar_o + 8 * ((g - 1) & 1), ((g - 1) >> 1) & 1, kErrAttnOutput);
                if (!ok)
                    break;
                // Values were taken out of this item's V.  (The word is written again only after this warp's weights of the
                // next item's last tile.)
                bool edges = false;
                if (mixed) {
                    wait(bar_edges, items & 1, kErrAttnOutput);
                    if (!ok)
                        break;
                    edges = ptx::ld_volatile_shared(sbase + L::kSlot + 4) != 0;
                }
                ++items;
                // The item's rows: finished here, or a part for the join.
                const float inv = l == 0.f ? 0.f : 1.f / l;
                if (warp_has_rows) {
#pragma unroll
                    for (int c = 0; c < DIM; c += 32) {
                        uint32_t o[32];
                        tmem_ld_x32(lane_base + kOColumn + c, o);
                        ptx::tmem_wait_ld();
                        if (!w.valid)
                            continue;
                        if (whole) {
                            float v[32];
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                v[k] = l == 0.f ? 0.f : __uint_as_float(o[k]) * inv;
                            store_row<DIM>(p, w, c, v);
                        } else {
                            float4 *dst = p.parts + (slot * (DIM / 4) + c / 4) * p.slot_rows + r;
#pragma unroll
                            for (int k = 0; k < 32; k += 4)
                                dst[k / 4 * p.slot_rows] = make_float4(__uint_as_float(o[k]), __uint_as_float(o[k + 1]),
                                                         __uint_as_float(o[k + 2]), __uint_as_float(o[k + 3]));
                        }
                    }
                    if (w.valid && whole && p.lse)
                        p.lse[(int64_t)w.token * p.heads + w.q_head] =
                            l == 0.f ? -CUDART_INF_F : (m * p.scale_log2 + log2f(l)) * CUDART_LN2_F;
                    if (w.valid && !whole) {
                        float2 *ml = reinterpret_cast<float2 *>(p.parts + 2 * (int64_t)gridDim.x * p.slot_rows * (DIM / 4));
                        ml[slot * p.slot_rows + r] = make_float2(m * p.scale_log2, l);
                    }
                    if (edges)
                        add_edge_values<DIM>(p, __ballot_sync(0xffffffffu, w.valid), sequence, w, key_begin, key_end,
                                             m == -CUDART_INF_F ? 0.f : m * p.scale_log2, whole ? inv : 1.f,
                                             whole ? -1 : slot, r);
                }
            }
        }
    }
    ptx::tcgen05_fence_before_thread_sync();
    __syncthreads();
    if (warp == 5) {
        ptx::tcgen05_fence_after_thread_sync();
        ptx::tmem_dealloc(tmem, kColumns);
    }
}

// Joins the parts of the items that shares cut: CTA c owns the one that begins
// in share c and ends in a later one.  A thread owns 16 elements of a row;
// neighbouring threads own neighbouring rows, as the parts lie in memory.
// Part i counts 2^(its maximum - the largest maximum), and the parts add in the
// order of the keys.  The kernel is a few memory latencies long: the item, the
// maxima, then all sums of up to four parts at once.
constexpr int kJoinThreads = 256, kJoinSplit = 4;   // kJoinSplit CTAs an item: 128 rows of 128 are a task a thread

template <int DIM>
__global__ void __launch_bounds__(kJoinThreads) join_parts_kernel(const AttnParams p, int ctas)
{
    constexpr int kGroups = DIM / 16;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    if (blockIdx.x == 0 && blockIdx.y == 0) {   // rows of no sequence
        const int first = p.batch > 0 ? min(max(p.cu_q[0], 0), p.q_tokens) : p.q_tokens;
        const int last = p.batch > 0 ? min(max(p.cu_q[p.batch], 0), p.q_tokens) : p.q_tokens;
        for (int t = threadIdx.x >> 5; t < p.q_tokens; t += kJoinThreads / 32)
            if (t < first || t >= last)
                for (int h = 0; h < p.heads; ++h) {
                    for (int d = threadIdx.x & 31; d < DIM; d += 32)
                        p.out[t * p.o_ts + h * p.o_hs + d] = __float2bfloat16_rn(0.f);
                    if ((threadIdx.x & 31) == 0 && p.lse)
                        p.lse[(int64_t)t * p.heads + h] = -CUDART_INF_F;
                }
    }
    if (p.batch == 0)
        return;
    const CutItem cut = p.cuts[blockIdx.x];
    const int parts = cut.parts;
    if (parts == 0)
        return;
    const float2 *ml = reinterpret_cast<const float2 *>(p.parts + 2 * (int64_t)ctas * p.slot_rows * (DIM / 4));
    const int rows = min(kTileRows, cut.q_len * p.group - cut.q_tile * kTileRows);
    auto slot = [&](int i) { return 2 * (int64_t)(blockIdx.x + i) + (i == 0 ? 1 : 0); };
    for (int c = threadIdx.x + blockIdx.y * kJoinThreads; c < rows * kGroups; c += kJoinSplit * kJoinThreads) {
        const int r = c % rows, e = c / rows * 4;
        const int row = cut.q_tile * kTileRows + r, t = cut.q0 + row / p.group, h = cut.head * p.group + row % p.group;
        float top = -CUDART_INF_F;
#pragma unroll 4
        for (int i = 0; i < parts; ++i)
            top = fmaxf(top, ml[slot(i) * p.slot_rows + r].x);
        const float base = top == -CUDART_INF_F ? 0.f : top;
        float4 acc[4] = {};
        float l = 0.f;
#pragma unroll 4
        for (int i = 0; i < parts; ++i) {
            const float2 x = ml[slot(i) * p.slot_rows + r];
            const float4 *src = p.parts + (slot(i) * (DIM / 4) + e) * p.slot_rows + r;
            const float a = ex2(x.x - base);
            l = fmaf(x.y, a, l);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float4 o = src[k * p.slot_rows];
                acc[k].x = fmaf(o.x, a, acc[k].x);
                acc[k].y = fmaf(o.y, a, acc[k].y);
                acc[k].z = fmaf(o.z, a, acc[k].z);
                acc[k].w = fmaf(o.w, a, acc[k].w);
            }
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        alignas(16) __nv_bfloat162 v[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (l == 0.f)
                acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            v[2 * k] = __floats2bfloat162_rn(acc[k].x * inv, acc[k].y * inv);
            v[2 * k + 1] = __floats2bfloat162_rn(acc[k].z * inv, acc[k].w * inv);
        }
        __nv_bfloat16 *o = p.out + t * p.o_ts + h * p.o_hs + 4 * e;
        if (p.out_vec) {
            reinterpret_cast<uint4 *>(o)[0] = *reinterpret_cast<const uint4 *>(v);
            reinterpret_cast<uint4 *>(o)[1] = *reinterpret_cast<const uint4 *>(v + 4);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                o[2 * k] = v[k].x;
                o[2 * k + 1] = v[k].y;
            }
        }
        if (p.lse && e == 0)
            p.lse[(int64_t)t * p.heads + h] = l == 0.f ? -CUDART_INF_F : (base + log2f(l)) * CUDART_LN2_F;
    }
}

bool attention_shape_ok(int batch, int q_tokens, int heads, int kv_heads, int dim)
{
    return batch >= 0 && q_tokens >= 0 && heads > 0 && kv_heads > 0 && heads % kv_heads == 0 &&
           heads / kv_heads <= kTileRows && (dim == 64 || dim == 128) && (int64_t)q_tokens * heads < INT_MAX / 2;
}

// Rows a part can have: a tile's, or all there are.
int slot_rows_of(int q_tokens, int heads, int kv_heads)
{
    return (int)std::min<int64_t>(kTileRows, std::max<int64_t>(1, (int64_t)q_tokens * (heads / kv_heads)));
}

// (dim, place, head, page) view of a cache; a box is one head's 64 elements of
// up to 64 places of a page, zeros outside.
lowm_status_t encode_cache(const void *base, int64_t page_stride, int64_t place_stride, int64_t head_stride,
                           int64_t num_pages, int page_size, int kv_heads, int dim, CUtensorMap *map)
{
    EncodeTiledFn enc = host_encode_fn();
    if (!enc)
        return LOWM_ERR_CUDA;
    // A dimension of one never uses its stride, but the encoder checks it.
    const cuuint64_t unit = 16;
    const cuuint64_t dims[4] = {(cuuint64_t)dim, (cuuint64_t)page_size, (cuuint64_t)kv_heads, (cuuint64_t)num_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)place_stride * 2, kv_heads > 1 ? (cuuint64_t)head_stride * 2 : unit,
                                   num_pages > 1 ? (cuuint64_t)page_stride * 2 : unit};
    const cuuint32_t box[4] = {64, (cuuint32_t)std::min(page_size, kTileKeys), 1, 1};
    const cuuint32_t step[4] = {1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, step,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? LOWM_OK
               : LOWM_ERR_CUDA;
}

template <int DIM>
lowm_status_t launch_attention(const CUtensorMap &map_k, const CUtensorMap &map_v, const AttnParams &p, int sms,
                               void *stream)
{
    static SmemOptIn opt_in;
    if (!opt_in.set(reinterpret_cast<const void *>(paged_attention_kernel<DIM>), AttnSmem<DIM>::kBytes))
        return LOWM_ERR_CUDA;
    const int ctas = std::min(2 * sms, kMaxAttnCtas);
    if (p.batch > 0) {
        const lowm_status_t st = launch_pdl(paged_attention_kernel<DIM>, dim3((unsigned)ctas), dim3(kAttnThreads),
                                            AttnSmem<DIM>::kBytes, stream, map_k, map_v, p);
        if (st != LOWM_OK)
            return st;
    }
    return launch_pdl(join_parts_kernel<DIM>, dim3((unsigned)ctas, kJoinSplit), dim3(kJoinThreads), 0, stream, p, ctas);
}

}  // namespace
}  // namespace lowm

extern "C" size_t lowm_paged_attention_workspace(int batch, int q_tokens, int heads, int kv_heads, int dim)
{
    using namespace lowm;
    if (!attention_shape_ok(batch, q_tokens, heads, kv_heads, dim))
        return 0;
    return (size_t)2 * kMaxAttnCtas * slot_rows_of(q_tokens, heads, kv_heads) * (dim + 2) * sizeof(float) +
           kMaxAttnCtas * sizeof(CutItem);
}

extern "C" lowm_status_t lowm_paged_attention(
    const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *k_cache, int64_t k_page_stride,
    int64_t k_place_stride, int64_t k_cache_head_stride, const void *v_cache, int64_t v_page_stride,
    int64_t v_place_stride, int64_t v_cache_head_stride, int64_t num_pages, int page_size, const int32_t *page_table,
    int64_t page_table_stride, int table_width, const int32_t *kv_lens, const int32_t *cu_q, void *out,
    int64_t out_token_stride, int64_t out_head_stride, float *lse, int batch, int q_tokens, int heads, int kv_heads,
    int dim, float scale, int window, void *workspace, size_t workspace_bytes, void *stream)
{
    using namespace lowm;
    if (batch < 0 || q_tokens < 0 || heads <= 0 || kv_heads <= 0 || dim <= 0 || num_pages <= 0 || num_pages > INT_MAX || page_size <= 0 ||
        table_width < 0 || window < 0 || !(scale == scale))
        return LOWM_ERR_INVALID_ARGUMENT;
    if (!attention_shape_ok(batch, q_tokens, heads, kv_heads, dim) || page_size < 8 || page_size > 1024 ||
        (page_size & (page_size - 1)))
        return LOWM_ERR_UNSUPPORTED_SHAPE;
    if (q_tokens == 0)
        return LOWM_OK;
    if (!q || !k_cache || !v_cache || !cu_q || !out || !workspace || (batch && !kv_lens) ||
        (batch && table_width && !page_table))
        return LOWM_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < lowm_paged_attention_workspace(batch, q_tokens, heads, kv_heads, dim))
        return LOWM_ERR_INVALID_ARGUMENT;
    const int64_t cache_strides[] = {k_page_stride, k_place_stride, k_cache_head_stride,
                                     v_page_stride, v_place_stride, v_cache_head_stride};
    const int64_t extents[] = {num_pages, page_size, kv_heads, num_pages, page_size, kv_heads};
    for (int i = 0; i < 6; ++i) {
        if (extents[i] == 1)                     // the stride of a single one is not used
            continue;
        if (cache_strides[i] < 0)
            return LOWM_ERR_INVALID_ARGUMENT;
        if (cache_strides[i] & 7)
            return LOWM_ERR_MISALIGNED;
    }
    if (q_token_stride < 0 || q_head_stride < 0 || out_token_stride < 0 || out_head_stride < 0 || page_table_stride < 0)
        return LOWM_ERR_INVALID_ARGUMENT;
    if (!is_aligned(k_cache, 16) || !is_aligned(v_cache, 16) || !is_aligned(workspace, 16) || !is_aligned(q, 2) ||
        !is_aligned(out, 2) || !is_aligned(page_table, 4) || !is_aligned(kv_lens, 4) || !is_aligned(cu_q, 4) ||
        !is_aligned(lse, 4))
        return LOWM_ERR_MISALIGNED;
    // The tensor maps take strides below 2^40 bytes, and no stride of 0 where it is used.
    for (int i = 0; i < 6; ++i)
        if (extents[i] > 1 && (cache_strides[i] == 0 || cache_strides[i] >= ((int64_t)1 << 39)))
            return LOWM_ERR_INVALID_ARGUMENT;
    // Tile counts are 32-bit in the kernels, rounding up to equal shares included.
    const int64_t capacity = std::min<int64_t>((int64_t)table_width * page_size, kMaxKeys);
    const int64_t q_tiles = (int64_t)q_tokens * (heads / kv_heads) / kTileRows + batch;
    if ((double)q_tiles * kv_heads * (double)(capacity / kTileKeys + 2 + kItemCost) > (double)(INT_MAX - kMaxAttnCtas))
        return LOWM_ERR_UNSUPPORTED_SHAPE;
    int sms = 0;
    lowm_status_t st = host_check_device(&sms);
    if (st != LOWM_OK)
        return st;

    AttnParams p;
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.lse = lse;
    p.q_ts = q_token_stride;
    p.q_hs = q_head_stride;
    p.o_ts = out_token_stride;
    p.o_hs = out_head_stride;
    p.table_stride = page_table_stride;
    p.k = static_cast<const __nv_bfloat16 *>(k_cache);
    p.v = static_cast<const __nv_bfloat16 *>(v_cache);
    p.num_pages = num_pages;
    p.k_page = k_page_stride;
    p.k_place = k_place_stride;
    p.k_head = k_cache_head_stride;
    p.v_page = v_page_stride;
    p.v_place = v_place_stride;
    p.v_head = v_cache_head_stride;
    p.table = page_table;
    p.kv_lens = kv_lens;
    p.cu_q = cu_q;
    p.page_size = page_size;
    p.page_shift = 0;
    while ((1 << p.page_shift) < page_size)
        ++p.page_shift;
    p.batch = batch;
    p.q_tokens = q_tokens;
    p.heads = heads;
    p.kv_heads = kv_heads;
    p.group = heads / kv_heads;
    p.window = window < kMaxKeys ? window : 0;
    p.slot_rows = slot_rows_of(q_tokens, heads, kv_heads);
    p.capacity = (int)capacity;
    // Never 0, so that a masked score (-inf) stays one.
    p.scale_log2 = std::max((scale < 0.f ? -scale : scale) * 1.44269504088896340736f, 1e-30f);
    p.q_sign = scale < 0.f ? -1.f : 1.f;
    p.q_vec = is_aligned(q, 16) && !((q_token_stride | q_head_stride) & 7);
    p.out_vec = is_aligned(out, 16) && !((out_token_stride | out_head_stride) & 7);
    p.parts = static_cast<float4 *>(workspace);
    p.cuts = reinterpret_cast<CutItem *>(static_cast<uint8_t *>(workspace) +
                                         (size_t)2 * kMaxAttnCtas * p.slot_rows * (dim + 2) * sizeof(float));
    p.status = host_status_word();
    if (!p.status)
        return LOWM_ERR_CUDA;
    CUtensorMap map_k, map_v;
    if ((st = encode_cache(k_cache, k_page_stride, k_place_stride, k_cache_head_stride, num_pages, page_size, kv_heads,
                           dim, &map_k)) != LOWM_OK ||
        (st = encode_cache(v_cache, v_page_stride, v_place_stride, v_cache_head_stride, num_pages, page_size, kv_heads,
                           dim, &map_v)) != LOWM_OK)
        return st;
    return dim == 64 ? launch_attention<64>(map_k, map_v, p, sms, stream)
                     : launch_attention<128>(map_k, map_v, p, sms, stream);
}
