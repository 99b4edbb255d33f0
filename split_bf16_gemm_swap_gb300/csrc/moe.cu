// A mixture-of-experts layer for at most 128 tokens (lowm_layer.h): router and
// top-k, gated up-projection, down-projection with the weighted sum.
#include <cuda_bf16.h>
#include <math_constants.h>

#include <algorithm>

#include "layer_host.h"
#include "ptx.cuh"

namespace lowm {
namespace {

constexpr int kMaxTokens = 128, kMaxExperts = 1024, kMaxTopK = 16, kMaxWidth = 32768;

struct MoeParams {
    const __nv_bfloat16 *x, *router, *gate_up, *down;
    const float *bias;
    __nv_bfloat16 *out;
    int64_t x_stride, out_stride;
    int tokens, hidden, inner, experts, top_k, scoring, renormalize;
    float scale;
    int *ids;        // [tokens, top_k]
    float *weights;  // [tokens, top_k]
    float *act;      // [tokens, top_k, inner]
};

__device__ __forceinline__ float warp_dot(const __nv_bfloat16 *a, const __nv_bfloat16 *b, int n)
{
    float s = 0.f;
    for (int i = threadIdx.x & 31; i < n; i += 32)
        s = fmaf(__bfloat162float(a[i]), __bfloat162float(b[i]), s);
    for (int o = 16; o > 0; o >>= 1)
        s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// Order-preserving image of a float (NaN above +inf): the choice stays total
// and distinct whatever the scores hold.
__device__ __forceinline__ unsigned ordered_bits(float f)
{
    const unsigned u = f != f ? 0x7fffffffu : __float_as_uint(f + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(256) router_kernel(const MoeParams p)
{
    __shared__ float prob[kMaxExperts];
    __shared__ unsigned key[kMaxExperts];
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int t = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int e = warp; e < p.experts; e += 8) {
        const float s = warp_dot(p.x + t * p.x_stride, p.router + (int64_t)e * p.hidden, p.hidden);
        if (lane == 0)
            prob[e] = s;
    }
    __syncthreads();
    if (warp)
        return;
    if (p.scoring == LOWM_MOE_SOFTMAX) {
        float m = -CUDART_INF_F, l = 0.f;
        for (int e = lane; e < p.experts; e += 32)
            m = fmaxf(m, prob[e]);
        for (int o = 16; o > 0; o >>= 1)
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        for (int e = lane; e < p.experts; e += 32) {
            prob[e] = expf(prob[e] - m);
            l += prob[e];
        }
        for (int o = 16; o > 0; o >>= 1)
            l += __shfl_xor_sync(0xffffffffu, l, o);
        for (int e = lane; e < p.experts; e += 32)
            prob[e] /= l;
    } else {
        for (int e = lane; e < p.experts; e += 32)
            prob[e] = 1.f / (1.f + expf(-prob[e]));
    }
    for (int e = lane; e < p.experts; e += 32)
        key[e] = ordered_bits(prob[e] + (p.bias ? p.bias[e] : 0.f));
    __syncwarp();
    float sum = 0.f, mine = 0.f;
    for (int s = 0; s < p.top_k; ++s) {
        unsigned long long best = 0;
        for (int e = lane; e < p.experts; e += 32)
            best = max(best, ((unsigned long long)key[e] << 32) | (unsigned)(kMaxExperts - e));
        for (int o = 16; o > 0; o >>= 1)
            best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
        const int e = kMaxExperts - (int)(best & 0xffffffffu);
        const float w = prob[e];
        sum += w;
        if (lane == s)
            mine = w;
        __syncwarp();
        if (lane == 0) {
            key[e] = 0;
            p.ids[t * p.top_k + s] = e;
        }
        __syncwarp();
    }
    if (lane < p.top_k)
        p.weights[t * p.top_k + lane] = mine * p.scale / (p.renormalize ? sum : 1.f);
}

__global__ void __launch_bounds__(256) gate_up_kernel(const MoeParams p)
{
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int pair = blockIdx.x, i = blockIdx.y * 8 + (threadIdx.x >> 5);
    if (i >= p.inner)
        return;
    const __nv_bfloat16 *x = p.x + (pair / p.top_k) * p.x_stride;
    const __nv_bfloat16 *w = p.gate_up + (int64_t)p.ids[pair] * 2 * p.inner * p.hidden;
    const float g = warp_dot(x, w + (int64_t)i * p.hidden, p.hidden);
    const float u = warp_dot(x, w + (int64_t)(p.inner + i) * p.hidden, p.hidden);
    if ((threadIdx.x & 31) == 0)
        p.act[(int64_t)pair * p.inner + i] = g / (1.f + expf(-g)) * u;
}

__global__ void __launch_bounds__(256) down_kernel(const MoeParams p)
{
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int t = blockIdx.x, h = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (h >= p.hidden)
        return;
    float y = 0.f;
    for (int s = 0; s < p.top_k; ++s) {
        const int pair = t * p.top_k + s;
        const __nv_bfloat16 *w = p.down + ((int64_t)p.ids[pair] * p.hidden + h) * p.inner;
        const float *a = p.act + (int64_t)pair * p.inner;
        float d = 0.f;
        for (int i = lane; i < p.inner; i += 32)
            d = fmaf(__bfloat162float(w[i]), a[i], d);
        for (int o = 16; o > 0; o >>= 1)
            d += __shfl_xor_sync(0xffffffffu, d, o);
        y = fmaf(p.weights[pair], d, y);
    }
    if (lane == 0)
        p.out[t * p.out_stride + h] = __float2bfloat16_rn(y);
}

bool moe_shape_ok(int tokens, int hidden, int inner, int experts, int top_k)
{
    return tokens >= 0 && tokens <= kMaxTokens && hidden > 0 && hidden <= kMaxWidth && hidden % 8 == 0 && inner > 0 &&
           inner <= kMaxWidth && inner % 8 == 0 && experts > 0 && experts <= kMaxExperts && top_k > 0 &&
           top_k <= std::min(kMaxTopK, experts);
}

}  // namespace
}  // namespace lowm

extern "C" size_t lowm_moe_workspace(int tokens, int hidden, int inner, int experts, int top_k)
{
    if (!lowm::moe_shape_ok(tokens, hidden, inner, experts, top_k))
        return 0;
    return (size_t)std::max(tokens, 1) * (size_t)top_k * ((size_t)inner * 4 + 8) + 16;
}

extern "C" lowm_status_t lowm_moe(const void *x, int64_t x_stride, const void *router, const float *bias,
                                  const void *gate_up, const void *down, void *out, int64_t out_stride, int tokens,
                                  int hidden, int inner, int experts, int top_k, int scoring, int renormalize,
                                  float scale, void *workspace, size_t workspace_bytes, void *stream)
{
    using namespace lowm;
    if (tokens < 0 || hidden <= 0 || inner <= 0 || experts <= 0 || top_k <= 0 || top_k > experts ||
        (scoring != LOWM_MOE_SOFTMAX && scoring != LOWM_MOE_SIGMOID) || !(scale == scale))
        return LOWM_ERR_INVALID_ARGUMENT;
    if (!moe_shape_ok(tokens, hidden, inner, experts, top_k))
        return LOWM_ERR_UNSUPPORTED_SHAPE;
    if (tokens == 0)
        return LOWM_OK;
    if (!x || !router || !gate_up || !down || !out || !workspace ||
        workspace_bytes < lowm_moe_workspace(tokens, hidden, inner, experts, top_k) || x_stride < 0 ||
        out_stride < hidden)
        return LOWM_ERR_INVALID_ARGUMENT;
    if (!is_aligned(x, 16) || !is_aligned(router, 16) || !is_aligned(gate_up, 16) || !is_aligned(down, 16) ||
        !is_aligned(workspace, 16) || !is_aligned(bias, 4) || !is_aligned(out, 2) || (x_stride & 7))
        return LOWM_ERR_MISALIGNED;
    lowm_status_t st = host_check_device(nullptr);
    if (st != LOWM_OK)
        return st;

    MoeParams p;
    p.x = static_cast<const __nv_bfloat16 *>(x);
    p.router = static_cast<const __nv_bfloat16 *>(router);
    p.gate_up = static_cast<const __nv_bfloat16 *>(gate_up);
    p.down = static_cast<const __nv_bfloat16 *>(down);
    p.bias = bias;
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.x_stride = x_stride;
    p.out_stride = out_stride;
    p.tokens = tokens;
    p.hidden = hidden;
    p.inner = inner;
    p.experts = experts;
    p.top_k = top_k;
    p.scoring = scoring;
    p.renormalize = renormalize;
    p.scale = scale;
    const int pairs = tokens * top_k;
    p.act = static_cast<float *>(workspace);
    p.weights = p.act + (size_t)pairs * inner;
    p.ids = reinterpret_cast<int *>(p.weights + pairs);
    if ((st = launch_pdl(router_kernel, dim3((unsigned)tokens), dim3(256), 0, stream, p)) != LOWM_OK)
        return st;
    if ((st = launch_pdl(gate_up_kernel, dim3((unsigned)pairs, (unsigned)((inner + 7) / 8)), dim3(256), 0, stream,
                         p)) != LOWM_OK)
        return st;
    return launch_pdl(down_kernel, dim3((unsigned)tokens, (unsigned)((hidden + 7) / 8)), dim3(256), 0, stream, p);
}
