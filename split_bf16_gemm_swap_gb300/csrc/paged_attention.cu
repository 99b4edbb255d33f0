// Attention of each sequence's newest tokens over its paged keys and values
// (lowm_layer.h).  One warp owns one (token, head): it walks the keys the
// token sees with a running maximum and sum.
#include <cuda_bf16.h>
#include <math_constants.h>

#include <algorithm>

#include "layer_host.h"
#include "ptx.cuh"

namespace lowm {
namespace {

struct AttnParams {
    const __nv_bfloat16 *q, *k, *v;
    __nv_bfloat16 *out;
    float *lse;
    int64_t q_ts, q_hs, o_ts, o_hs, k_page, k_place, k_head, v_page, v_place, v_head, num_pages, table_stride;
    const int32_t *table, *kv_lens, *cu_q;
    int page_size, table_width, batch, q_tokens, heads, kv_heads, window;
    float scale;
};

template <int DIM>
__global__ void __launch_bounds__(128) attention_kernel(const AttnParams p)
{
    constexpr int E = DIM / 32;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (unit >= (int64_t)p.q_tokens * p.heads)
        return;
    const int t = (int)(unit / p.heads), h = (int)(unit % p.heads);
    int b = 0;
    while (b < p.batch && p.cu_q[b + 1] <= t)
        ++b;
    float o[E] = {}, m = -CUDART_INF_F, l = 0.f;
    if (b < p.batch) {
        const int64_t cap = (int64_t)p.table_width * p.page_size;
        const int64_t kv = min((int64_t)max(p.kv_lens[b], 0), cap);
        const int64_t pos = kv - (p.cu_q[b + 1] - t);
        const int g = h / (p.heads / p.kv_heads);
        float q[E];
        for (int i = 0; i < E; ++i)
            q[i] = __bfloat162float(p.q[t * p.q_ts + h * p.q_hs + lane * E + i]) * p.scale;
        for (int64_t j = p.window > 0 ? max((int64_t)0, pos - p.window + 1) : 0; j <= pos; ++j) {
            const int64_t page = p.table[b * p.table_stride + j / p.page_size];
            const bool in = page >= 0 && page < p.num_pages;
            const __nv_bfloat16 *k = p.k + page * p.k_page + (j % p.page_size) * p.k_place + g * p.k_head + lane * E;
            const __nv_bfloat16 *v = p.v + page * p.v_page + (j % p.page_size) * p.v_place + g * p.v_head + lane * E;
            float s = 0.f;
            for (int i = 0; i < E; ++i)
                s += in ? q[i] * __bfloat162float(k[i]) : 0.f;
            for (int x = 16; x > 0; x >>= 1)
                s += __shfl_xor_sync(0xffffffffu, s, x);
            const float mn = fmaxf(m, s), a = expf(m - mn), e = expf(s - mn);
            l = l * a + e;
            m = mn;
            for (int i = 0; i < E; ++i)
                o[i] = o[i] * a + (in ? e * __bfloat162float(v[i]) : 0.f);
        }
    }
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    for (int i = 0; i < E; ++i)
        p.out[t * p.o_ts + h * p.o_hs + lane * E + i] = __float2bfloat16_rn(o[i] * inv);
    if (p.lse && lane == 0)
        p.lse[(int64_t)t * p.heads + h] = l == 0.f ? -CUDART_INF_F : m + logf(l);
}

bool attention_shape_ok(int batch, int q_tokens, int heads, int kv_heads, int dim)
{
    return batch >= 0 && q_tokens >= 0 && heads > 0 && kv_heads > 0 && heads % kv_heads == 0 &&
           heads / kv_heads <= 128 && (dim == 64 || dim == 128);
}

}  // namespace
}  // namespace lowm

extern "C" size_t lowm_paged_attention_workspace(int batch, int q_tokens, int heads, int kv_heads, int dim)
{
    return lowm::attention_shape_ok(batch, q_tokens, heads, kv_heads, dim) ? 16 : 0;
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
    if (batch < 0 || q_tokens < 0 || heads <= 0 || kv_heads <= 0 || dim <= 0 || num_pages < 0 || page_size <= 0 ||
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
    for (int64_t s : cache_strides) {
        if (s < 0)
            return LOWM_ERR_INVALID_ARGUMENT;
        if (s & 7)
            return LOWM_ERR_MISALIGNED;
    }
    if (q_token_stride < 0 || q_head_stride < 0 || out_token_stride < 0 || out_head_stride < 0 || page_table_stride < 0)
        return LOWM_ERR_INVALID_ARGUMENT;
    if (!is_aligned(k_cache, 16) || !is_aligned(v_cache, 16) || !is_aligned(workspace, 16) || !is_aligned(q, 2) ||
        !is_aligned(out, 2) || !is_aligned(page_table, 4) || !is_aligned(kv_lens, 4) || !is_aligned(cu_q, 4) ||
        !is_aligned(lse, 4))
        return LOWM_ERR_MISALIGNED;
    const lowm_status_t st = host_check_device(nullptr);
    if (st != LOWM_OK)
        return st;

    AttnParams p;
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.k = static_cast<const __nv_bfloat16 *>(k_cache);
    p.v = static_cast<const __nv_bfloat16 *>(v_cache);
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.lse = lse;
    p.q_ts = q_token_stride;
    p.q_hs = q_head_stride;
    p.o_ts = out_token_stride;
    p.o_hs = out_head_stride;
    p.k_page = k_page_stride;
    p.k_place = k_place_stride;
    p.k_head = k_cache_head_stride;
    p.v_page = v_page_stride;
    p.v_place = v_place_stride;
    p.v_head = v_cache_head_stride;
    p.num_pages = num_pages;
    p.table_stride = page_table_stride;
    p.table = page_table;
    p.kv_lens = kv_lens;
    p.cu_q = cu_q;
    p.page_size = page_size;
    p.table_width = table_width;
    p.batch = batch;
    p.q_tokens = q_tokens;
    p.heads = heads;
    p.kv_heads = kv_heads;
    p.window = window;
    p.scale = scale;
    const int64_t units = (int64_t)q_tokens * heads;
    return launch_pdl(dim == 64 ? attention_kernel<64> : attention_kernel<128>, dim3((unsigned)((units + 3) / 4)),
                      dim3(128), 0, stream, p);
}
