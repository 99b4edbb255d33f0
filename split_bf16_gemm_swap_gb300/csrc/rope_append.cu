// Rotary positions (one to three axes) for new queries and keys, and the
// append of keys and values to the paged cache (lowm_layer.h).
//
// Element-wise work bound by its bytes (at few tokens by the launch and two
// dependent reads, position then table).  One CTA owns one token; a thread
// owns one group of pairs for several heads, so a token's cosines and sines
// are read once per thread and serve every head it visits.
#include <cuda_bf16.h>

#include <math_constants.h>

#include "layer_host.h"
#include "ptx.cuh"

namespace lowm {
namespace {

struct RopeParams {
    const __nv_bfloat16 *q, *k, *v;
    __nv_bfloat16 *q_out, *k_cache, *v_cache;
    int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, qo_ts, qo_hs;
    int64_t kc_page, kc_place, kc_head, vc_page, vc_place, vc_head;
    const float *cos_sin;
    const int64_t *positions, *slots;
    int64_t table_rows, positions_stride, capacity;
    int page_size, axes, section0, section1;
    int heads, kv_heads, dim, rotary;
};

// GROUP pairs at a time: 8 for the 16-byte form (dim and rotary multiples of
// 16, strides of 8, aligned), 1 for everything else.  A head is dim / 2
// pairs in units of GROUP (and one last single element when dim is odd).
// Rotary units are pairs (j, j + rotary / 2) or (2j, 2j + 1); the units
// behind them copy 2 * GROUP neighbouring elements.
template <int GROUP, bool INTERLEAVED>
__global__ void __launch_bounds__(512) rope_append_kernel(const RopeParams p)
{
    const int64_t t = blockIdx.x;
    const int units = (p.dim + 2 * GROUP - 1) / (2 * GROUP);
    const int u0 = threadIdx.x % units, lane0 = threadIdx.x / units, lanes = blockDim.x / units;
    const int half = p.rotary / 2;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    if (lane0 >= lanes)
        return;

    const int64_t slot = p.slots[t];
    bool append = slot >= 0 && slot < p.capacity;
    const int64_t page = append ? slot / p.page_size : 0, place = append ? slot % p.page_size : 0;
    bool known = true;
    const int64_t pos0 = p.positions[t];
    const int64_t pos1 = p.axes > 1 ? p.positions[p.positions_stride + t] : pos0;
    const int64_t pos2 = p.axes > 2 ? p.positions[2 * p.positions_stride + t] : pos0;
    known = pos0 >= 0 && pos0 < p.table_rows && pos1 >= 0 && pos1 < p.table_rows && pos2 >= 0 && pos2 < p.table_rows;
    append = append && known;

    const bool turns = u0 * GROUP < half;
    float c[GROUP], s[GROUP];
    if (turns) {
#pragma unroll
        for (int i = 0; i < GROUP; ++i) {
            const int j = u0 * GROUP + i;
            const int64_t pos = j < p.section0 ? pos0 : (j < p.section0 + p.section1 ? pos1 : pos2);
            const float *row = p.cos_sin + pos * p.rotary;
            c[i] = known ? row[j] : CUDART_NAN_F;
            s[i] = known ? row[half + j] : CUDART_NAN_F;
        }
    }
    // Offsets of the unit's two runs of GROUP elements (the pair halves, or 2 * GROUP neighbours).
    const int e0 = turns && !INTERLEAVED ? u0 * GROUP : (turns ? 2 * u0 * GROUP : p.rotary + 2 * (u0 * GROUP - half));
    const int e1 = turns && !INTERLEAVED ? e0 + half : e0 + GROUP;
    const bool two = e1 < p.dim;                       // false only for the last element of an odd dim

    struct alignas(GROUP == 8 ? 16 : 2) Run {
        __nv_bfloat16 v[GROUP];
    };
    const int rows = p.heads + 2 * p.kv_heads;
    for (int h = lane0; h < rows; h += lanes) {
        const __nv_bfloat16 *src;
        __nv_bfloat16 *dst;
        bool turn = turns;
        if (h < p.heads) {
            src = p.q + t * p.q_ts + h * p.q_hs;
            dst = p.q_out + t * p.qo_ts + h * p.qo_hs;
        } else if (!append) {
            break;
        } else if (h < p.heads + p.kv_heads) {
            const int g = h - p.heads;
            src = p.k + t * p.k_ts + g * p.k_hs;
            dst = p.k_cache + page * p.kc_page + place * p.kc_place + g * p.kc_head;
        } else {
            const int g = h - p.heads - p.kv_heads;
            src = p.v + t * p.v_ts + g * p.v_hs;
            dst = p.v_cache + page * p.vc_page + place * p.vc_place + g * p.vc_head;
            turn = false;
        }
        Run a, b;
        a = *reinterpret_cast<const Run *>(src + e0);
        if (two)
            b = *reinterpret_cast<const Run *>(src + e1);
        if (turn) {
            Run oa, ob;
#pragma unroll
            for (int i = 0; i < GROUP; ++i) {
                // interleaved: pair i is elements 2i, 2i + 1 of the 2 * GROUP neighbours
                constexpr int kHalfGroup = GROUP / 2 > 0 ? GROUP / 2 : 1;
                const bool lo = i < kHalfGroup || GROUP == 1;
                float x, y;
                if constexpr (INTERLEAVED && GROUP == 8) {
                    x = __bfloat162float(lo ? a.v[(2 * i) & 7] : b.v[(2 * i) & 7]);
                    y = __bfloat162float(lo ? a.v[(2 * i + 1) & 7] : b.v[(2 * i + 1) & 7]);
                } else {
                    x = __bfloat162float(a.v[i]);
                    y = __bfloat162float(b.v[i]);
                }
                const __nv_bfloat16 nx = __float2bfloat16_rn(x * c[i] - y * s[i]);
                const __nv_bfloat16 ny = __float2bfloat16_rn(x * s[i] + y * c[i]);
                if constexpr (INTERLEAVED && GROUP == 8) {
                    (lo ? oa : ob).v[(2 * i) & 7] = nx;
                    (lo ? oa : ob).v[(2 * i + 1) & 7] = ny;
                } else {
                    oa.v[i] = nx;
                    ob.v[i] = ny;
                }
            }
            a = oa;
            b = ob;
        }
        *reinterpret_cast<Run *>(dst + e0) = a;
        if (two)
            *reinterpret_cast<Run *>(dst + e1) = b;
    }
}

}  // namespace
}  // namespace lowm

extern "C" lowm_status_t lowm_rope_append(
    const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *k, int64_t k_token_stride,
    int64_t k_head_stride, const void *v, int64_t v_token_stride, int64_t v_head_stride, const float *cos_sin,
    int64_t table_rows, const int64_t *positions, int64_t positions_stride, int axes, int section0, int section1,
    int interleaved, const int64_t *slots, void *q_out, int64_t q_out_token_stride, int64_t q_out_head_stride,
    void *k_cache, int64_t k_page_stride, int64_t k_place_stride, int64_t k_cache_head_stride, void *v_cache,
    int64_t v_page_stride, int64_t v_place_stride, int64_t v_cache_head_stride, int64_t num_pages, int page_size,
    int tokens, int heads, int kv_heads, int dim, int rotary, void *stream)
{
    using namespace lowm;
    if (tokens < 0 || heads <= 0 || kv_heads <= 0 || dim <= 0 || rotary < 0 || table_rows < 0 || num_pages < 0 ||
        page_size <= 0 || axes < 1 || axes > 3)
        return LOWM_ERR_INVALID_ARGUMENT;
    if (dim > 1024 || rotary > dim || (rotary & 1))
        return LOWM_ERR_UNSUPPORTED_SHAPE;
    if (section0 < 0 || section1 < 0 || section0 + section1 > rotary / 2 || (axes == 1 && section0 != rotary / 2) ||
        (axes == 2 && section0 + section1 != rotary / 2))
        return LOWM_ERR_INVALID_ARGUMENT;
    if (tokens == 0)
        return LOWM_OK;
    if (!q || !k || !v || !positions || !slots || !q_out || !k_cache || !v_cache || (rotary && !cos_sin))
        return LOWM_ERR_INVALID_ARGUMENT;
    const int64_t strides[] = {q_token_stride, q_head_stride, k_token_stride, k_head_stride, v_token_stride,
                               v_head_stride, q_out_token_stride, q_out_head_stride, k_page_stride, k_place_stride,
                               k_cache_head_stride, v_page_stride, v_place_stride, v_cache_head_stride};
    int64_t all = 0;
    for (int64_t s : strides) {
        if (s < 0)
            return LOWM_ERR_INVALID_ARGUMENT;
        all |= s;
    }
    const void *bf16s[] = {q, k, v, q_out, k_cache, v_cache};
    bool aligned = true;
    for (const void *x : bf16s) {
        if (!is_aligned(x, 2))
            return LOWM_ERR_MISALIGNED;
        aligned = aligned && is_aligned(x, 16);
    }
    if (!is_aligned(cos_sin, 16) || !is_aligned(positions, 8) || !is_aligned(slots, 8))
        return LOWM_ERR_MISALIGNED;
    const lowm_status_t st = host_check_device(nullptr);
    if (st != LOWM_OK)
        return st;

    RopeParams p;
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.k = static_cast<const __nv_bfloat16 *>(k);
    p.v = static_cast<const __nv_bfloat16 *>(v);
    p.q_out = static_cast<__nv_bfloat16 *>(q_out);
    p.k_cache = static_cast<__nv_bfloat16 *>(k_cache);
    p.v_cache = static_cast<__nv_bfloat16 *>(v_cache);
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
    p.cos_sin = cos_sin;
    p.positions = positions;
    p.slots = slots;
    p.table_rows = table_rows;
    p.positions_stride = positions_stride;
    p.capacity = num_pages * page_size;
    p.page_size = page_size;
    p.axes = axes;
    p.section0 = section0;
    p.section1 = section1;
    p.heads = heads;
    p.kv_heads = kv_heads;
    p.dim = dim;
    p.rotary = rotary;

    const bool vec = aligned && dim % 16 == 0 && rotary % 16 == 0 && (all & 7) == 0;
    const int units = vec ? dim / 16 : (dim + 1) / 2;
    const int rows = heads + 2 * kv_heads;
    int threads = units * rows;                        // a thread for every unit, at most 512
    if (threads > 512)
        threads = 512 / units * units;
    threads = (threads + 31) / 32 * 32;
    auto fn = vec ? (interleaved ? rope_append_kernel<8, true> : rope_append_kernel<8, false>)
                  : (interleaved ? rope_append_kernel<1, true> : rope_append_kernel<1, false>);
    return launch_pdl(fn, dim3((unsigned)tokens), dim3((unsigned)threads), 0, stream, p);
}
