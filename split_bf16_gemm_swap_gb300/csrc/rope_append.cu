// Rotary positions (one to three axes) for new queries and keys, and the
// append of keys and values to the paged cache (lowm_layer.h).
//
// Element-wise work bound by its bytes (4096 tokens of 32 / 8 heads of 128: 20 us,
// 5.1 TB/s; at few tokens by the launch and two dependent reads, position then
// table: 4 tokens 2.5 us).  One CTA owns one token; a thread owns one group of
// pairs for several heads, so a token's cosines and sines are read once per
// thread and serve every head it visits.
#include <cuda_bf16.h>

#include <math_constants.h>

#include <algorithm>
#include <climits>

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
template <int GROUP>
struct alignas(GROUP == 8 ? 16 : 2) Run {
    __nv_bfloat16 v[GROUP];
};

// Turns the pairs of one unit: runs a and b are the pairs' halves, or, with
// INTERLEAVED and GROUP 8, pair i is elements 2i, 2i + 1 of a and b in a row.
template <int GROUP, bool INTERLEAVED>
__device__ __forceinline__ void turn(Run<GROUP> &a, Run<GROUP> &b, const float (&c)[GROUP], const float (&s)[GROUP])
{
    constexpr bool kMixed = INTERLEAVED && GROUP == 8;
    const Run<GROUP> x = a, y = b;
#pragma unroll
    for (int i = 0; i < GROUP; ++i) {
        const bool lo = i < GROUP / 2;
        const float u = __bfloat162float(kMixed ? (lo ? x : y).v[(2 * i) & (GROUP - 1)] : x.v[i]);
        const float v = __bfloat162float(kMixed ? (lo ? x : y).v[(2 * i + 1) & (GROUP - 1)] : y.v[i]);
        const __nv_bfloat16 nu = __float2bfloat16_rn(u * c[i] - v * s[i]);
        const __nv_bfloat16 nv = __float2bfloat16_rn(u * s[i] + v * c[i]);
        if constexpr (kMixed) {
            (lo ? a : b).v[(2 * i) & (GROUP - 1)] = nu;
            (lo ? a : b).v[(2 * i + 1) & (GROUP - 1)] = nv;
        } else {
            a.v[i] = nu;
            b.v[i] = nv;
        }
    }
}

// At most 64 registers a thread: more threads an SM are worth more than more
// heads in flight (4096 tokens of 32 / 8 heads of 128: 20.1 us, at 70 registers
// 21.1, with four heads of q and one of k and v in flight at 128 29.8).
template <int GROUP, bool INTERLEAVED>
__global__ void __launch_bounds__(512, 2) rope_append_kernel(const RopeParams p)
{
    const int64_t t = blockIdx.x;
    const int units = (p.dim + 2 * GROUP - 1) / (2 * GROUP);
    const int u0 = threadIdx.x % units, lane0 = threadIdx.x / units, lanes = blockDim.x / units;
    const int half = p.rotary / 2;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    if (lane0 >= lanes)
        return;

    const bool turns = u0 * GROUP < half;
    // Offsets of the unit's two runs of GROUP elements (the pair halves, or 2 * GROUP neighbours).
    const int e0 = turns && !INTERLEAVED ? u0 * GROUP : (turns ? 2 * u0 * GROUP : p.rotary + 2 * (u0 * GROUP - half));
    const int e1 = turns && !INTERLEAVED ? e0 + half : e0 + GROUP;
    const bool two = e1 < p.dim;                       // false only for the last element of an odd dim
    const int64_t slot = p.slots[t];
    const int64_t pos0 = p.positions[t];
    const int64_t pos1 = p.axes > 1 ? p.positions[p.positions_stride + t] : pos0;
    const int64_t pos2 = p.axes > 2 ? p.positions[2 * p.positions_stride + t] : pos0;

    // This thread's heads of one tensor, the next one requested before this one is turned and stored.
    float c[GROUP], s[GROUP];
    auto heads = [&](const __nv_bfloat16 *src, int64_t src_step, __nv_bfloat16 *dst, int64_t dst_step, int n, bool turned) {
        if (lane0 >= n)
            return;
        src += lane0 * src_step;
        dst += lane0 * dst_step;
        src_step *= lanes;
        dst_step *= lanes;
        Run<GROUP> a = *reinterpret_cast<const Run<GROUP> *>(src + e0), b = a;
        if (two)
            b = *reinterpret_cast<const Run<GROUP> *>(src + e1);
        for (int h = lane0; h < n; h += lanes) {
            Run<GROUP> na = a, nb = b;
            if (h + lanes < n) {
                src += src_step;
                na = *reinterpret_cast<const Run<GROUP> *>(src + e0);
                if (two)
                    nb = *reinterpret_cast<const Run<GROUP> *>(src + e1);
            }
            if (turned)
                turn<GROUP, INTERLEAVED>(a, b, c, s);
            *reinterpret_cast<Run<GROUP> *>(dst + e0) = a;
            if (two)
                *reinterpret_cast<Run<GROUP> *>(dst + e1) = b;
            dst += dst_step;
            a = na;
            b = nb;
        }
    };
    const bool known = pos0 >= 0 && pos0 < p.table_rows && pos1 >= 0 && pos1 < p.table_rows && pos2 >= 0 && pos2 < p.table_rows;
    const bool append = known && slot >= 0 && slot < p.capacity;
    int64_t page = 0;
    int place = 0;
    if (append) {
        page = slot < INT_MAX ? (int)slot / p.page_size : slot / p.page_size;
        place = (int)(slot - page * p.page_size);
    }
    if (turns) {
        const int j0 = u0 * GROUP, j1 = j0 + GROUP - 1, end1 = p.section0 + p.section1;
        const float *rows[3] = {p.cos_sin + pos0 * p.rotary, p.cos_sin + pos1 * p.rotary, p.cos_sin + pos2 * p.rotary};
        const int axis0 = j0 < p.section0 ? 0 : (j0 < end1 ? 1 : 2), axis1 = j1 < p.section0 ? 0 : (j1 < end1 ? 1 : 2);
        if (GROUP == 8 && axis0 == axis1 && known) {   // one axis: 16 bytes at a time
            const float *row = axis0 == 0 ? rows[0] : (axis0 == 1 ? rows[1] : rows[2]);
#pragma unroll
            for (int i = 0; i < GROUP; i += 4) {
                *reinterpret_cast<float4 *>(c + i) = *reinterpret_cast<const float4 *>(row + j0 + i);
                *reinterpret_cast<float4 *>(s + i) = *reinterpret_cast<const float4 *>(row + half + j0 + i);
            }
        } else {
#pragma unroll
            for (int i = 0; i < GROUP; ++i) {
                const int j = j0 + i;
                const float *row = j < p.section0 ? rows[0] : (j < end1 ? rows[1] : rows[2]);
                c[i] = known ? row[j] : CUDART_NAN_F;
                s[i] = known ? row[half + j] : CUDART_NAN_F;
            }
        }
    }
    if (append) {
        heads(p.v + t * p.v_ts, p.v_hs, p.v_cache + page * p.vc_page + place * p.vc_place, p.vc_head, p.kv_heads, false);
        heads(p.k + t * p.k_ts, p.k_hs, p.k_cache + page * p.kc_page + place * p.kc_place, p.kc_head, p.kv_heads, turns);
    }
    heads(p.q + t * p.q_ts, p.q_hs, p.q_out + t * p.qo_ts, p.qo_hs, p.heads, turns);
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
    int sms = 0;
    const lowm_status_t st = host_check_device(&sms);
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
    // Few tokens: a thread for every unit, to be done soonest.  Many: fewer threads
    // with more heads each, which read a token's cosines and sines fewer times
    // (GB300, 32 / 8 heads of 128, 512 -> 128 -> 64 threads: 4 tokens 2.6, 2.8, 3.4
    // us; 1000 tokens 7.7, 5.0, 5.7; 4096 tokens 39.9, 25.3, 21.1), four heads at
    // least (4096 tokens, 64 -> 32 threads: 8 / 2 heads of 128 8.4 -> 6.5 us, 32 / 8
    // of 64 13.5 -> 11.2; but 2048 tokens of 32 / 32 of 128, eight heads, 19.5 -> 24.8).
    const int most = std::max(heads, kv_heads);
    const int lanes = tokens >= 8 * sms ? std::min(64 / units, (most + 3) / 4)
                                        : std::min((tokens >= 2 * sms ? 128 : 512) / units, most);
    const int threads = (std::max(lanes, 1) * units + 31) / 32 * 32;
    auto fn = vec ? (interleaved ? rope_append_kernel<8, true> : rope_append_kernel<8, false>)
                  : (interleaved ? rope_append_kernel<1, true> : rope_append_kernel<1, false>);
    return launch_pdl(fn, dim3((unsigned)tokens), dim3((unsigned)threads), 0, stream, p);
}
