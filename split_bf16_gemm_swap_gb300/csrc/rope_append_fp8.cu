// Rotary positions for new queries and keys, and the append of keys and values
// to a paged cache of e4m3 codes with a scale for each block of tokens and head
// (lowm_fp8.h).
//
// A block's scale depends on all of its tokens, so the unit of work is a run: the
// neighbouring tokens of the call that lie in one block.  For one head of a run, of k
// or of v, a warp finds the run's largest magnitude, the block's scale, moves the
// block's older codes to it where it has grown, and writes the new ones.  q's rows are
// turned by warps of the same launch.  Two kernels: of heads of 64, 128 or 256 elements
// and 16-byte rows in 16-byte pieces, else element by element.
#include <cuda_bf16.h>
#include <math_constants.h>

#include <algorithm>
#include <climits>

#include "../../include/lowm_fp8.h"
#include "fp8_device.cuh"
#include "layer_host.h"
#include "ptx.cuh"

namespace lowm {
namespace {

struct Rope8Params {
    const __nv_bfloat16 *q, *k, *v;
    __nv_bfloat16 *q_out;
    uint8_t *k_cache, *v_cache;
    float *k_scale, *v_scale;
    int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, qo_ts, qo_hs;
    int64_t kc_page, kc_place, kc_head, vc_page, vc_place, vc_head;
    int64_t ks_page, ks_block, ks_head, vs_page, vs_block, vs_head;
    const float *cos_sin;
    const int64_t *positions, *slots;
    int64_t table_rows, positions_stride, capacity;
    int page_size, block, block_shift, axes, section0, section1, interleaved;
    int tokens, heads, kv_heads, dim, rotary;
};

constexpr int kRopeThreads = 256;

struct Position {
    const float *rows[3];                    // the table's rows by axis
    bool known;
};

__device__ __forceinline__ Position position_of(const Rope8Params &p, int64_t t)
{
    Position at;
    at.known = true;
    for (int a = 0; a < 3; ++a) {
        const int64_t pos = p.positions[a < p.axes ? a * p.positions_stride + t : t];
        at.known = at.known && pos >= 0 && pos < p.table_rows;
        at.rows[a] = p.cos_sin + pos * p.rotary;
    }
    return at;
}

// Turns pair j of a row: elements e0 and e1 of x.
__device__ __forceinline__ float2 turned(const Rope8Params &p, const Position &at, const __nv_bfloat16 *x, int j, int e0, int e1)
{
    const float *row = j < p.section0 ? at.rows[0] : (j < p.section0 + p.section1 ? at.rows[1] : at.rows[2]);
    const float c = at.known ? row[j] : CUDART_NAN_F, s = at.known ? row[p.rotary / 2 + j] : CUDART_NAN_F;
    const float a = __bfloat162float(x[e0]), b = __bfloat162float(x[e1]);
    return make_float2(a * c - b * s, a * s + b * c);
}

// Calls put(e0, value, e1, value) for this lane's pairs of a row, and put(e, value, -1, 0) for its other elements.
template <typename Put>
__device__ __forceinline__ void each(const Rope8Params &p, bool turns, const Position &at, const __nv_bfloat16 *x, Put put)
{
    const int lane = threadIdx.x & 31, half = turns ? p.rotary / 2 : 0;
    for (int j = lane; j < half; j += 32) {
        const int e0 = p.interleaved ? 2 * j : j, e1 = p.interleaved ? 2 * j + 1 : j + half;
        const float2 y = turned(p, at, x, j, e0, e1);
        put(e0, y.x, e1, y.y);
    }
    for (int e = 2 * half + lane; e < p.dim; e += 32)
        put(e, __bfloat162float(x[e]), -1, 0.f);
}

// A run: the tokens of one block, each with a higher slot than the one before it, fewer than `block` tokens of the call apart
// (those between them are not appended).  slot_of(t) is the slot of token t, -1 where it is not appended or not one.  The
// tokens from t to the last one of the run that begins there; 0 when none begins.
template <typename SlotOf>
__device__ __forceinline__ int64_t run_at(const Rope8Params &p, int64_t t, SlotOf slot_of)
{
    const int64_t slot = slot_of(t), block = slot >> p.block_shift;
    if (slot < 0)
        return 0;
    for (int back = 1; back < p.block && back <= t; ++back) {
        const int64_t before = slot_of(t - back);
        if (before >= 0) {
            if (before < slot && before >> p.block_shift == block)
                return 0;                    // it is part of that token's
            break;
        }
    }
    int64_t last = t, highest = slot;
    for (int64_t next = t + 1; next - last < p.block && next < p.tokens; ++next) {
        const int64_t at = slot_of(next);
        if (at < 0)
            continue;
        if (at <= highest || at >> p.block_shift != block)
            break;
        last = next;
        highest = at;
    }
    return last - t + 1;
}

__global__ void __launch_bounds__(kRopeThreads) rope_append_fp8_kernel(const Rope8Params p)
{
    const int lane = threadIdx.x & 31;
    const int per_token = 2 * p.kv_heads + p.heads;
    const int64_t at = (int64_t)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
    const int64_t t = at / per_token;
    const int head = (int)(at - t * per_token);
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    if (t >= p.tokens)
        return;
    if (head >= 2 * p.kv_heads) {
        const int h = head - 2 * p.kv_heads;
        __nv_bfloat16 *out = p.q_out + t * p.qo_ts + h * p.qo_hs;
        each(p, true, position_of(p, t), p.q + t * p.q_ts + h * p.q_hs, [&](int e0, float a, int e1, float b) {
            out[e0] = __float2bfloat16_rn(a);
            if (e1 >= 0)
                out[e1] = __float2bfloat16_rn(b);
        });
        return;
    }
    // The slot of a token that is appended, or -1.
    auto slot_of = [&](int64_t i) {
        if (i < 0 || i >= p.tokens)
            return (int64_t)-1;
        const int64_t slot = p.slots[i];
        return slot >= 0 && slot < p.capacity && position_of(p, i).known ? slot : (int64_t)-1;
    };
    const int64_t n = run_at(p, t, slot_of), slot = slot_of(t);
    if (n == 0)
        return;
    const bool is_k = head < p.kv_heads;
    const int h = is_k ? head : head - p.kv_heads;
    const __nv_bfloat16 *x = is_k ? p.k + t * p.k_ts + h * p.k_hs : p.v + t * p.v_ts + h * p.v_hs;
    const int64_t step = is_k ? p.k_ts : p.v_ts, place_step = is_k ? p.kc_place : p.vc_place;
    const int64_t page = slot / p.page_size;
    const int place = (int)(slot - page * p.page_size), first = place >> p.block_shift << p.block_shift;
    uint8_t *cells = is_k ? p.k_cache + page * p.kc_page + h * p.kc_head : p.v_cache + page * p.vc_page + h * p.vc_head;
    float *scale = is_k ? p.k_scale + page * p.ks_page + (place >> p.block_shift) * p.ks_block + h * p.ks_head
                        : p.v_scale + page * p.vs_page + (place >> p.block_shift) * p.vs_block + h * p.vs_head;

    float amax = 0.f;
    for (int64_t i = 0; i < n; ++i)
        if (slot_of(t + i) >= 0)
            each(p, is_k, position_of(p, t + i), x + i * step,
                 [&](int, float a, int, float b) { amax = fmaxf(amax, fmaxf(finite_magnitude(a), finite_magnitude(b))); });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    float now = power_of_two(scale_exponent(amax));
    if (place > first) {
        const float before = *scale;
        now = before > now ? before : now;   // (a scale that is not a number is replaced)
        if (now != before) {
            const float ratio = before / now;
            for (int l = first; l < place; ++l)
                for (int e = lane; e < p.dim; e += 32) {
                    uint8_t *c = cells + l * place_step + e;
                    *c = (uint8_t)to_e4m3x2(__low2float(e4m3x2_to_half2(*c)) * ratio, 0.f);
                }
        }
    }
    for (int64_t i = 0; i < n; ++i) {
        const int64_t at = slot_of(t + i);
        if (at < 0)
            continue;
        uint8_t *to = cells + (at - page * p.page_size) * place_step;
        each(p, is_k, position_of(p, t + i), x + i * step, [&](int e0, float a, int e1, float b) {
            const uint32_t w = to_e4m3x2(nan_unless_finite(a) / now, nan_unless_finite(b) / now);
            to[e0] = (uint8_t)w;
            if (e1 >= 0)
                to[e1] = (uint8_t)(w >> 8);
        });
    }
    __syncwarp();                            // every lane has read the old scale
    if (lane == 0)
        *scale = now;
}

// ------------------------------------------------------------------ 16-byte pieces
// A lane has a unit of 16 elements of a token: eight pairs of the rotation, or what lies behind them; DIM / 16 lanes have a
// token, so a warp has 512 / DIM tokens at a time.  The first CTAs of the grid have k and v: each looks at kTokens tokens of
// the call and has the runs that begin among them, for some of the heads: of a run of one token (decoding) such a group of
// lanes has a head, of a longer one a warp.  What they need of the slots and the table comes into shared memory first, all
// at once (one by one these were chains of latencies), the table's rows while one warp finds the runs.  The other CTAs turn q.
// Chunks of 1501 tokens (3831 in all, 88 MB, 32 / 8 heads of 128): 22.8 us, 3.9 TB/s; k and v alone 18, whose CTAs are a chain
// of five latencies (slots, table, runs, values, codes) and of instructions that four warps a scheduler hide in part; q alone
// 15.  With 16 tokens a CTA 26, with three CTAs an SM, which spill, 31, with the values loaded one after another 36.
constexpr int kTokens = 32, kWideWarps = 8, kWideThreads = 32 * kWideWarps;
constexpr int kWideBlock = 128;              // the longest run
__host__ __device__ constexpr int angle_tokens(int dim) { return dim == 256 ? kTokens : 2 * kTokens; }    // whose angles are kept: 32 KiB at most
constexpr int kAtHand = 4;                   // units a thread loads at once

template <int DIM, bool INTERLEAVED>
struct RopeUnit {
    static constexpr int kLanes = DIM / 16, kAtOnce = 32 / kLanes;
    int e0, e1, j0;                          // the unit's two runs of eight elements; its first pair
    bool turns;

    __device__ RopeUnit(const Rope8Params &p, bool turned)
    {
        const int u = threadIdx.x % kLanes, half = p.rotary / 2;
        turns = turned && 8 * u < half;
        j0 = 8 * u;
        e0 = !turned ? 16 * u : (turns ? (INTERLEAVED ? 16 * u : 8 * u) : p.rotary + 2 * (8 * u - half));
        e1 = turns && !INTERLEAVED ? e0 + half : e0 + 8;
    }

    // The cosines and sines of a unit that turns, from a row kept in shared memory.
    __device__ __forceinline__ void kept_angles(const Rope8Params &p, const float *kept, float (&c)[8], float (&s)[8]) const
    {
        const int half = p.rotary / 2;
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            const float4 x = *reinterpret_cast<const float4 *>(kept + j0 + i), y = *reinterpret_cast<const float4 *>(kept + half + j0 + i);
            c[i] = x.x, c[i + 1] = x.y, c[i + 2] = x.z, c[i + 3] = x.w;
            s[i] = y.x, s[i + 1] = y.y, s[i + 2] = y.z, s[i + 3] = y.w;
        }
    }

    // Those of token t from the table.
    __device__ __forceinline__ void angles(const Rope8Params &p, int64_t t, float (&c)[8], float (&s)[8]) const
    {
        const int half = p.rotary / 2;
        const Position at = position_of(p, t);
        const int end1 = p.section0 + p.section1;
        const int axis0 = j0 < p.section0 ? 0 : (j0 < end1 ? 1 : 2), axis1 = j0 + 7 < p.section0 ? 0 : (j0 + 7 < end1 ? 1 : 2);
        if (axis0 == axis1 && at.known) {
            const float *row = (axis0 == 0 ? at.rows[0] : (axis0 == 1 ? at.rows[1] : at.rows[2])) + j0;
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
                const float4 x = *reinterpret_cast<const float4 *>(row + i), y = *reinterpret_cast<const float4 *>(row + half + i);
                c[i] = x.x, c[i + 1] = x.y, c[i + 2] = x.z, c[i + 3] = x.w;
                s[i] = y.x, s[i + 1] = y.y, s[i + 2] = y.z, s[i + 3] = y.w;
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int j = j0 + i;
            const float *row = j < p.section0 ? at.rows[0] : (j < end1 ? at.rows[1] : at.rows[2]);
            c[i] = at.known ? row[j] : CUDART_NAN_F;
            s[i] = at.known ? row[half + j] : CUDART_NAN_F;
        }
    }

    __device__ __forceinline__ void load(const __nv_bfloat16 *x, uint4 (&v)[2]) const
    {
        v[0] = *reinterpret_cast<const uint4 *>(x + e0);
        v[1] = *reinterpret_cast<const uint4 *>(x + e1);
    }

    __device__ __forceinline__ void turn(const uint4 (&v)[2], const float (&c)[8], const float (&s)[8], float (&y)[16]) const
    {
        const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            y[2 * i] = __uint_as_float(w[i] << 16);
            y[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
        if (!turns)
            return;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float &a = y[INTERLEAVED ? 2 * i : i], &b = y[INTERLEAVED ? 2 * i + 1 : 8 + i];
            const float u = a, x = b;
            a = u * c[i] - x * s[i];
            b = u * s[i] + x * c[i];
        }
    }

    // The bits of the largest finite magnitude; whether there are others.
    __device__ __forceinline__ static void largest(const float (&y)[16], uint32_t &top, bool &other)
    {
        uint32_t all = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint32_t m = __float_as_uint(y[i]) & 0x7fffffffu;
            all = max(all, m);
            top = max(top, m < 0x7f800000u ? m : 0u);
        }
        other = other || all >= 0x7f800000u;
    }

    // Codes y / scale; `plain`: all are finite and the scale is a power of two with this inverse.
    __device__ __forceinline__ void store(uint8_t *to, const float (&y)[16], float scale, bool plain, float inverse) const
    {
        uint32_t w[4] = {};
        if (plain) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = to_e4m3x2(y[4 * i] * inverse, y[4 * i + 1] * inverse) |
                       to_e4m3x2(y[4 * i + 2] * inverse, y[4 * i + 3] * inverse) << 16;
        } else {                             // (rare, and kept short)
            float z[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
                z[i] = y[i];
#pragma unroll 1
            for (int i = 15; i >= 0; --i) {
                w[3] = w[3] << 8 | w[2] >> 24;
                w[2] = w[2] << 8 | w[1] >> 24;
                w[1] = w[1] << 8 | w[0] >> 24;
                w[0] = w[0] << 8 | (to_e4m3x2(nan_unless_finite(z[i]) / scale, 0.f) & 0xffu);
            }
        }
        *reinterpret_cast<uint2 *>(to + e0) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2 *>(to + e1) = make_uint2(w[2], w[3]);
    }

    // Moves the unit's codes of a token to another scale.
    __device__ __forceinline__ void move(uint8_t *at, float ratio) const
    {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint2 *c = reinterpret_cast<uint2 *>(at + (half ? e1 : e0));
            uint2 w = *c;
            uint32_t out[2] = {w.x, w.y};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 lo = __half22float2(e4m3x2_to_half2(out[i] & 0xffffu)), hi = __half22float2(e4m3x2_to_half2(out[i] >> 16));
                out[i] = to_e4m3x2(lo.x * ratio, lo.y * ratio) | to_e4m3x2(hi.x * ratio, hi.y * ratio) << 16;
            }
            *c = make_uint2(out[0], out[1]);
        }
    }
};

// (Not in line: few calls come here, and four copies of it would be in the loop.)
template <int DIM, bool INTERLEAVED>
__device__ __noinline__ void far_angles_of(const Rope8Params &p, const RopeUnit<DIM, INTERLEAVED> &unit, int64_t t, float *to)
{
    float c[8], s[8];
    unit.angles(p, t, c, s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        to[i] = c[i];
        to[8 + i] = s[i];
    }
}

template <int DIM, bool INTERLEAVED>
__device__ __forceinline__ void far_angles(const Rope8Params &p, const RopeUnit<DIM, INTERLEAVED> &unit, int64_t t, float (&c)[8],
                                           float (&s)[8])
{
    float both[16];
    far_angles_of(p, unit, t, both);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        c[i] = both[i];
        s[i] = both[8 + i];
    }
}

// One head of k's or v's cache.
struct HeadCache {
    const __nv_bfloat16 *x;
    uint8_t *cells;
    float *scales;
    int64_t step, page, place, s_page, s_block;
};

__device__ __forceinline__ HeadCache head_cache(const Rope8Params &p, int head)
{
    const bool is_k = head < p.kv_heads;
    const int h = is_k ? head : head - p.kv_heads;
    HeadCache c;
    c.x = is_k ? p.k + h * p.k_hs : p.v + h * p.v_hs;
    c.step = is_k ? p.k_ts : p.v_ts;
    c.cells = is_k ? p.k_cache + h * p.kc_head : p.v_cache + h * p.vc_head;
    c.scales = is_k ? p.k_scale + h * p.ks_head : p.v_scale + h * p.vs_head;
    c.page = is_k ? p.kc_page : p.vc_page;
    c.place = is_k ? p.kc_place : p.vc_place;
    c.s_page = is_k ? p.ks_page : p.vs_page;
    c.s_block = is_k ? p.ks_block : p.vs_block;
    return c;
}

// q's rows: `at_once` tokens of the call by as many equal parts of the CTA; a thread has one unit of every so manieth head.
template <int DIM, bool INTERLEAVED>
__device__ __forceinline__ void turn_queries(const Rope8Params &p, int64_t cta, int at_once)
{
    using Unit = RopeUnit<DIM, INTERLEAVED>;
    const int part = kWideThreads / at_once, lanes = part / Unit::kLanes;
    const int64_t t = cta * at_once + threadIdx.x / part;
    if (t >= p.tokens)
        return;
    const Unit unit(p, true);
    int h = threadIdx.x % part / Unit::kLanes;
    if (h >= p.heads)
        return;
    float cosines[8], sines[8];
    for (bool begin = true; h < p.heads; h += kAtHand * lanes, begin = false) {
        uint4 raw[kAtHand][2];
#pragma unroll
        for (int u = 0; u < kAtHand; ++u)
            if (h + u * lanes < p.heads)
                unit.load(p.q + t * p.q_ts + (h + u * lanes) * p.q_hs, raw[u]);
        if (begin && unit.turns)
            unit.angles(p, t, cosines, sines);
#pragma unroll
        for (int u = 0; u < kAtHand; ++u) {
            if (h + u * lanes >= p.heads)
                break;
            float y[16];
            unit.turn(raw[u], cosines, sines, y);
            alignas(16) __nv_bfloat162 v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = __floats2bfloat162_rn(y[2 * j], y[2 * j + 1]);
            __nv_bfloat16 *out = p.q_out + t * p.qo_ts + (h + u * lanes) * p.qo_hs;
            *reinterpret_cast<uint4 *>(out + unit.e0) = reinterpret_cast<const uint4 *>(v)[0];
            *reinterpret_cast<uint4 *>(out + unit.e1) = reinterpret_cast<const uint4 *>(v)[1];
        }
    }
}

template <int DIM, bool INTERLEAVED>
__global__ void __launch_bounds__(kWideThreads, 2)
    rope_append_fp8_wide_kernel(const Rope8Params p, int windows, int kv_ctas, int at_once)
{
    using Unit = RopeUnit<DIM, INTERLEAVED>;
    constexpr int kLanes = Unit::kLanes, kAtOnce = Unit::kAtOnce, kAngleTokens = angle_tokens(DIM);
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    if (blockIdx.x >= kv_ctas) {
        turn_queries<DIM, INTERLEAVED>(p, blockIdx.x - kv_ctas, at_once);
        return;
    }
    extern __shared__ __align__(16) float angles[];     // [kAngleTokens][rotary]
    __shared__ int64_t slots[kTokens + 2 * kWideBlock]; // from token t0 - block on; -1: not appended
    __shared__ int rows[3][kAngleTokens];    // of the table, by axis; -1: not one of its rows
    __shared__ int starts[kTokens], lengths[kTokens], counts[2];    // the runs that begin here, those of one token first
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, group = lane / kLanes;
    const int64_t t0 = (int64_t)(blockIdx.x % windows) * kTokens;
    // The heads of k, then v, in equal parts.
    const int columns = kv_ctas / windows, a_column = (2 * p.kv_heads + columns - 1) / columns;
    const int head0 = (int)(blockIdx.x / windows) * a_column, heads_here = min(a_column, 2 * p.kv_heads - head0);
    const int here = (int)min((int64_t)kTokens, p.tokens - t0);
    const int kept = (int)min((int64_t)min(kAngleTokens, kTokens - 1 + p.block), p.tokens - t0);      // tokens
    const int cached = kTokens + 2 * p.block;
    for (int i = threadIdx.x; i < cached; i += kWideThreads) {
        const int64_t t = t0 - p.block + i;
        int64_t slot = -1;
        if (t >= 0 && t < p.tokens) {
            int64_t at[3];
            slot = p.slots[t];
#pragma unroll
            for (int a = 0; a < 3; ++a)
                at[a] = p.positions[a < p.axes ? a * p.positions_stride + t : t];
            bool known = true;
#pragma unroll
            for (int a = 0; a < 3; ++a)
                known = known && at[a] >= 0 && at[a] < p.table_rows;
            if (i >= p.block && i < p.block + kAngleTokens)
#pragma unroll
                for (int a = 0; a < 3; ++a)
                    rows[a][i - p.block] = known ? (int)at[a] : -1;
            slot = known && slot >= 0 && slot < p.capacity ? slot : -1;
        }
        slots[i] = slot;
    }
    __syncthreads();
    auto slot_of = [&](int64_t t) {          // (what lies further away is of a run with gaps)
        const int64_t i = t - t0 + p.block;
        if (i >= 0 && i < cached)
            return slots[i];
        if (t < 0 || t >= p.tokens)
            return (int64_t)-1;
        const int64_t slot = p.slots[t];
        return slot >= 0 && slot < p.capacity && position_of(p, t).known ? slot : (int64_t)-1;
    };
    if (warp == 0) {                         // a lane a token
        const int n = lane < here ? (int)min(run_at(p, t0 + lane, slot_of), (int64_t)INT_MAX) : 0;
        const unsigned single = __ballot_sync(0xffffffffu, n == 1), longer = __ballot_sync(0xffffffffu, n > 1);
        if (n > 0) {
            const unsigned before = (1u << lane) - 1;
            const int at = n == 1 ? __popc(single & before) : __popc(single) + __popc(longer & before);
            starts[at] = lane;
            lengths[at] = n;
        }
        if (lane == 0) {
            counts[0] = __popc(single);
            counts[1] = __popc(longer);
        }
    } else if (head0 < p.kv_heads) {         // v is not turned
        // A warp a token, a lane an element of its row; loads before stores, to be under way together.
        constexpr int kLoad = 4;
        const int half = p.rotary / 2;
#pragma unroll 1
        for (int token0 = warp - 1; token0 < kept; token0 += kLoad * (kWideWarps - 1)) {
            float x[kLoad][DIM / 32];
#pragma unroll
            for (int u = 0; u < kLoad; ++u)
#pragma unroll
                for (int j = 0; j < DIM / 32; ++j) {
                    const int token = token0 + u * (kWideWarps - 1), e = lane + 32 * j, pair = e < half ? e : e - half;
                    const int row = token < kept ? rows[pair < p.section0 ? 0 : (pair < p.section0 + p.section1 ? 1 : 2)][token] : -1;
                    x[u][j] = row >= 0 && e < p.rotary ? p.cos_sin[(int64_t)row * p.rotary + e] : CUDART_NAN_F;
                }
#pragma unroll
            for (int u = 0; u < kLoad; ++u)
#pragma unroll
                for (int j = 0; j < DIM / 32; ++j) {
                    const int token = token0 + u * (kWideWarps - 1), e = lane + 32 * j;
                    if (token < kept && e < p.rotary)
                        angles[token * p.rotary + e] = x[u][j];
                }
        }
    }
    __syncthreads();
    const int singles = counts[0], longer = counts[1], batches = (singles + kAtOnce - 1) / kAtOnce;
    // Its heads of k and v: the runs' tasks, warp after warp.
    const int a_head = batches + longer, tasks = a_head * heads_here;
#pragma unroll 1
    for (int task = warp; task < tasks; task += kWideWarps) {
        const int nth = task / a_head, work = task - nth * a_head, head = head0 + nth;
        const HeadCache c = head_cache(p, head);
        const Unit unit(p, head < p.kv_heads);
        const bool one = work < batches;         // a batch of runs of one token, a group of lanes each; or a longer run
        const int run = one ? work * kAtOnce + group : singles + work - batches;
        const bool mine = !one || run < singles;
        const int start = mine ? starts[run] : 0;
        const int64_t t = t0 + start, slot = mine ? slots[p.block + start] : 0;
        const int n = mine ? lengths[run] : 0;
        const int64_t page = slot < INT_MAX ? (int)slot / p.page_size : slot / p.page_size;
        const int place = (int)(slot - page * p.page_size), block = place >> p.block_shift, older = place - block * p.block;
        uint8_t *cells = c.cells + page * c.page;
        float *scale = c.scales + page * c.s_page + block * c.s_block;
        const float before = mine && older > 0 ? *scale : 0.f;
        const int first = one ? 0 : group, step = one ? 1 : kAtOnce;      // this group's tokens of the run
        // This group's next tokens of the run, their loads all under way at once; those of a short run stay.
        uint4 raw[kAtHand][2];
        unsigned has = 0;
        auto fetch = [&](int k0) {
            has = 0;
#pragma unroll
            for (int u = 0; u < kAtHand; ++u) {
                const int k = k0 + u * step;
                if (k < n && slot_of(t + k) >= 0) {
                    has |= 1u << u;
                    unit.load(c.x + (t + k) * c.step, raw[u]);
                }
            }
        };
        const bool stays = n <= kAtHand * step;
        if (stays)
            fetch(first);
        uint32_t top = 0;
        bool other = false, plain = false;
        float now = 0.f, inverse = 0.f;
        // First the largest magnitude, then the codes: one loop, whose instructions fit the caches (two copies and a third
        // for what is not finite, and the kernel waited for instructions a third of its time).
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
            for (int k0 = first; k0 < n; k0 += kAtHand * step) {
                if (!stays)
                    fetch(k0);
#pragma unroll
                for (int u = 0; u < kAtHand; ++u) {
                    if (!(has >> u & 1))
                        continue;
                    const int k = k0 + u * step;
                    float cosines[8], sines[8], y[16];
                    if (unit.turns) {
                        if (start + k < kept)
                            unit.kept_angles(p, angles + (start + k) * p.rotary, cosines, sines);
                        else
                            far_angles(p, unit, t + k, cosines, sines);
                    }
                    unit.turn(raw[u], cosines, sines, y);
                    if (pass == 0)
                        Unit::largest(y, top, other);
                    else
                        unit.store(cells + (slot_of(t + k) - page * p.page_size) * c.place, y, now, plain, inverse);
                }
            }
            if (pass == 1)
                break;
            const unsigned others = __ballot_sync(0xffffffffu, other);
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {    // the group's largest, or the warp's
                const uint32_t far = __shfl_xor_sync(0xffffffffu, top, o);
                if (o < kLanes || !one)
                    top = max(top, far);
            }
            if (!mine)
                break;
            now = power_of_two(scale_exponent(__uint_as_float(top)));
            now = before > now ? before : now;   // (a scale that is not a number is replaced)
            if (older > 0 && now != before)
                for (int l = (one ? 0 : group); l < older; l += step)
                    unit.move(cells + (block * p.block + l) * c.place, before / now);
            const unsigned of_run = one ? ((1u << kLanes) - 1) << (group * kLanes) : 0xffffffffu;
            plain = !(others & of_run) && !(__float_as_uint(now) & 0x7fffffu) && now >= power_of_two(kMinScaleExponent) &&
                    now <= power_of_two(kMaxScaleExponent);
            inverse = plain ? 1.f / now : 0.f;
        }
        if (!mine)
            continue;
        if (one ? lane % kLanes == 0 : lane == 0)
            *scale = now;
    }
}

}  // namespace
}  // namespace lowm

extern "C" lowm_status_t lowm_rope_append_fp8(
    const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *k, int64_t k_token_stride,
    int64_t k_head_stride, const void *v, int64_t v_token_stride, int64_t v_head_stride, const float *cos_sin,
    int64_t table_rows, const int64_t *positions, int64_t positions_stride, int axes, int section0, int section1,
    int interleaved, const int64_t *slots, void *q_out, int64_t q_out_token_stride, int64_t q_out_head_stride,
    void *k_cache, int64_t k_page_stride, int64_t k_place_stride, int64_t k_cache_head_stride, void *v_cache,
    int64_t v_page_stride, int64_t v_place_stride, int64_t v_cache_head_stride, float *k_scale, int64_t ks_page_stride,
    int64_t ks_block_stride, int64_t ks_head_stride, float *v_scale, int64_t vs_page_stride, int64_t vs_block_stride,
    int64_t vs_head_stride, int64_t num_pages, int page_size, int block, int tokens, int heads, int kv_heads, int dim,
    int rotary, void *stream)
{
    using namespace lowm;
    if (tokens < 0 || heads <= 0 || kv_heads <= 0 || dim <= 0 || rotary < 0 || table_rows < 0 || num_pages < 0 ||
        page_size <= 0 || block <= 0 || axes < 1 || axes > 3)
        return LOWM_ERR_INVALID_ARGUMENT;
    if (dim > 256 || rotary > dim || (rotary & 1) || (block & (block - 1)) || page_size % block)
        return LOWM_ERR_UNSUPPORTED_SHAPE;
    if (section0 < 0 || section1 < 0 || section0 + section1 > rotary / 2 || (axes == 1 && section0 != rotary / 2) ||
        (axes == 2 && section0 + section1 != rotary / 2))
        return LOWM_ERR_INVALID_ARGUMENT;
    if (tokens == 0)
        return LOWM_OK;
    if (!q || !k || !v || !positions || !slots || !q_out || !k_cache || !v_cache || !k_scale || !v_scale ||
        (rotary && !cos_sin))
        return LOWM_ERR_INVALID_ARGUMENT;
    const int64_t strides[] = {q_token_stride, q_head_stride, k_token_stride, k_head_stride, v_token_stride,
                               v_head_stride, q_out_token_stride, q_out_head_stride, k_page_stride, k_place_stride,
                               k_cache_head_stride, v_page_stride, v_place_stride, v_cache_head_stride, ks_page_stride,
                               ks_block_stride, ks_head_stride, vs_page_stride, vs_block_stride, vs_head_stride};
    for (int64_t s : strides)
        if (s < 0)
            return LOWM_ERR_INVALID_ARGUMENT;
    if (!is_aligned(q, 2) || !is_aligned(k, 2) || !is_aligned(v, 2) || !is_aligned(q_out, 2) || !is_aligned(cos_sin, 16) ||
        !is_aligned(positions, 8) || !is_aligned(slots, 8) || !is_aligned(k_scale, 4) || !is_aligned(v_scale, 4))
        return LOWM_ERR_MISALIGNED;
    const int64_t ctas = ((int64_t)tokens * (2 * kv_heads + heads) + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
    if (ctas > INT_MAX)
        return LOWM_ERR_UNSUPPORTED_SHAPE;
    int sms = 0;
    const lowm_status_t st = host_check_device(&sms);
    if (st != LOWM_OK)
        return st;

    Rope8Params p;
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.k = static_cast<const __nv_bfloat16 *>(k);
    p.v = static_cast<const __nv_bfloat16 *>(v);
    p.q_out = static_cast<__nv_bfloat16 *>(q_out);
    p.k_cache = static_cast<uint8_t *>(k_cache);
    p.v_cache = static_cast<uint8_t *>(v_cache);
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.q_ts = q_token_stride;
    p.q_hs = q_head_stride;
    p.k_ts = k_token_stride;
    p.k_hs = k_head_stride;
    p.v_ts = v_token_stride;
    p.v_hs = v_head_stride;
    p.qo_ts = q_out_token_stride;
    p.qo_hs = q_out_head_stride;
    p.kc_page = k_page_stride;
    p.kc_place = k_place_stride;
    p.kc_head = k_cache_head_stride;
    p.vc_page = v_page_stride;
    p.vc_place = v_place_stride;
    p.vc_head = v_cache_head_stride;
    p.ks_page = ks_page_stride;
    p.ks_block = ks_block_stride;
    p.ks_head = ks_head_stride;
    p.vs_page = vs_page_stride;
    p.vs_block = vs_block_stride;
    p.vs_head = vs_head_stride;
    p.cos_sin = cos_sin;
    p.positions = positions;
    p.slots = slots;
    p.table_rows = table_rows;
    p.positions_stride = positions_stride;
    p.capacity = num_pages * page_size;
    p.page_size = page_size;
    p.block = block;
    p.block_shift = 0;
    while ((1 << p.block_shift) < block)
        ++p.block_shift;
    p.axes = axes;
    p.section0 = section0;
    p.section1 = section1;
    p.interleaved = interleaved;
    p.tokens = tokens;
    p.heads = heads;
    p.kv_heads = kv_heads;
    p.dim = dim;
    p.rotary = rotary;
    int64_t rows = 0, codes = 0;             // strides
    for (int i = 0; i < 8; ++i)
        rows |= strides[i];
    for (int i = 8; i < 14; ++i)
        codes |= strides[i];
    const bool wide = block <= kWideBlock && table_rows <= INT_MAX && (dim == 64 || dim == 128 || dim == 256) && rotary % 16 == 0 && !(rows & 7) && !(codes & 7) && is_aligned(q, 16) &&
                      is_aligned(k, 16) && is_aligned(v, 16) && is_aligned(q_out, 16) && is_aligned(k_cache, 8) && is_aligned(v_cache, 8);
    if (wide) {
        const int windows = (int)(((int64_t)tokens + kTokens - 1) / kTokens);
        // A head a CTA while there are SMs, a head a warp at most.
        const int columns = std::max((2 * kv_heads + kWideWarps - 1) / kWideWarps,
                                     std::min(2 * kv_heads, (sms + windows - 1) / windows));
        // Few tokens: a CTA each, to be done soonest.  Many: fewer threads with more heads, which read the angles once.
        const int at_once = tokens >= 4 * sms ? 4 : 1;
        const int64_t all = (int64_t)windows * columns + ((int64_t)tokens + at_once - 1) / at_once;
        if (all > INT_MAX)
            return LOWM_ERR_UNSUPPORTED_SHAPE;
        auto fn = dim == 64    ? (interleaved ? rope_append_fp8_wide_kernel<64, true> : rope_append_fp8_wide_kernel<64, false>)
                  : dim == 128 ? (interleaved ? rope_append_fp8_wide_kernel<128, true> : rope_append_fp8_wide_kernel<128, false>)
                               : (interleaved ? rope_append_fp8_wide_kernel<256, true> : rope_append_fp8_wide_kernel<256, false>);
        return launch_pdl(fn, dim3((unsigned)all), dim3(kWideThreads), (size_t)angle_tokens(dim) * rotary * sizeof(float), stream, p,
                          windows, windows * columns, at_once);
    }
    return launch_pdl(rope_append_fp8_kernel, dim3((unsigned)ctas), dim3(kRopeThreads), 0, stream, p);
}
