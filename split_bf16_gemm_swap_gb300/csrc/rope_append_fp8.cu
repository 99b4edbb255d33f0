// Rotary positions for new queries and keys, and the append of keys and values
// to a paged cache of e4m3 codes with a scale for each block of tokens and head
// (lowm_fp8.h).
//
// A block's scale depends on all of its tokens, so the unit of work is a run: the
// neighbouring tokens of the call that lie in one block.  A warp has one head of a
// run, of k or of v, a lane every 32nd pair of a row (or element behind the pairs):
// it finds the run's largest magnitude, the block's scale, moves the block's older
// codes to it where it has grown, and writes the new ones.  The rows are turned
// twice rather than kept: a run may be as long as a page.  q's rows are turned by
// further warps of the same launch.
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
    int page_size, block, axes, section0, section1, interleaved;
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
        const int64_t slot = p.slots[i];
        return slot >= 0 && slot < p.capacity && position_of(p, i).known ? slot : -1;
    };
    const int64_t slot = slot_of(t), block = slot / p.block;
    if (slot < 0)
        return;
    if (t > 0) {                             // the token before has the run, if it is part of it
        const int64_t before = slot_of(t - 1);
        if (before >= 0 && before < slot && before / p.block == block)
            return;
    }
    int n = 1;
    for (int64_t last = slot; n < p.block && t + n < p.tokens; ++n) {
        const int64_t next = slot_of(t + n);
        if (next <= last || next / p.block != block)
            break;
        last = next;
    }
    const bool is_k = head < p.kv_heads;
    const int h = is_k ? head : head - p.kv_heads;
    const __nv_bfloat16 *x = is_k ? p.k + t * p.k_ts + h * p.k_hs : p.v + t * p.v_ts + h * p.v_hs;
    const int64_t step = is_k ? p.k_ts : p.v_ts, place_step = is_k ? p.kc_place : p.vc_place;
    const int64_t page = slot / p.page_size;
    const int place = (int)(slot - page * p.page_size), first = place / p.block * p.block;
    uint8_t *cells = is_k ? p.k_cache + page * p.kc_page + h * p.kc_head : p.v_cache + page * p.vc_page + h * p.vc_head;
    float *scale = is_k ? p.k_scale + page * p.ks_page + place / p.block * p.ks_block + h * p.ks_head
                        : p.v_scale + page * p.vs_page + place / p.block * p.vs_block + h * p.vs_head;

    float amax = 0.f;
    for (int i = 0; i < n; ++i)
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
    for (int i = 0; i < n; ++i) {
        uint8_t *to = cells + (p.slots[t + i] - page * p.page_size) * place_step;
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
    p.axes = axes;
    p.section0 = section0;
    p.section1 = section1;
    p.interleaved = interleaved;
    p.tokens = tokens;
    p.heads = heads;
    p.kv_heads = kv_heads;
    p.dim = dim;
    p.rotary = rotary;
    return launch_pdl(rope_append_fp8_kernel, dim3((unsigned)ctas), dim3(kRopeThreads), 0, stream, p);
}
