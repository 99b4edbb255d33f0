// The norms after and before a block, its gate and the residual scale, one
// pass: r' = s r + g RMS(y; w_post), n = RMS(r'; w_pre) (lowm_layer.h).
//
// One CTA owns one token.  Everything the row needs (y, r, gate, weights) is
// requested before the first reduction, stays in registers as it came (two
// bytes an element) and r' stays there in fp32, so each byte moves once and
// the two reductions are the only waits.  At decode sizes the time is the
// launch, one memory latency and the two reductions (4 x 4096: 2.4 us); at
// prompt sizes it is the bandwidth of r, y, r' and n (8192 x 4096 bf16: 43.7 us,
// 6.1 TB/s; with an fp32 residual and a gate per token 73.9 us, 6.4 TB/s).  Rows
// of odd widths have their weights by single loads and a warp more, or all by
// single loads, and cost up to twice as much (8000 x 4095 with a post weight
// 102 us; 8000 x 3001 64 us).
#include <cuda_bf16.h>

#include <algorithm>

#include "layer_host.h"
#include "ptx.cuh"

namespace lowm {
namespace {

struct NormParams {
    const void *residual;
    const __nv_bfloat16 *block, *post, *gate, *pre;
    void *out_residual;
    __nv_bfloat16 *out;
    int64_t residual_stride, block_stride, gate_stride, out_residual_stride, out_stride;
    int hidden, tokens;
    float scale, eps, inv_hidden;
};

// VEC elements of a row starting at i: one 16-byte access of bf16 (two of
// fp32) when VEC is 8, one element when VEC is 1.
template <int VEC>
struct alignas(2 * VEC) Pack {
    __nv_bfloat16 v[VEC];
};

template <int VEC>
__device__ __forceinline__ void load_bf16(const __nv_bfloat16 *p, Pack<VEC> &o)
{
    if constexpr (VEC == 8)
        *reinterpret_cast<uint4 *>(o.v) = *reinterpret_cast<const uint4 *>(p);
    else
        o.v[0] = *p;
}

template <int VEC>
__device__ __forceinline__ void store_bf16(__nv_bfloat16 *p, const float (&f)[VEC])
{
    if constexpr (VEC == 8) {
        uint4 u;
        __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&u);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        *reinterpret_cast<uint4 *>(p) = u;
    } else {
        *p = __float2bfloat16_rn(f[0]);
    }
}

// VEC elements of the residual stream as they lie in memory.
template <int VEC, bool F32>
struct Residual;

template <int VEC>
struct Residual<VEC, false> {
    Pack<VEC> p;
    __device__ void load(const void *base, int64_t at) { load_bf16(static_cast<const __nv_bfloat16 *>(base) + at, p); }
    __device__ void load_one(const void *base, int64_t at) { p.v[0] = static_cast<const __nv_bfloat16 *>(base)[at]; }
    __device__ float value(int j) const { return __bfloat162float(p.v[j]); }
    static __device__ void store(void *base, int64_t at, const float (&f)[VEC])
    {
        store_bf16(static_cast<__nv_bfloat16 *>(base) + at, f);
    }
    static __device__ void store_one(void *base, int64_t at, float f)
    {
        static_cast<__nv_bfloat16 *>(base)[at] = __float2bfloat16_rn(f);
    }
};

template <int VEC>
struct Residual<VEC, true> {
    float f[VEC];
    __device__ void load(const void *base, int64_t at)
    {
        const float *src = static_cast<const float *>(base) + at;
        if constexpr (VEC == 8) {
            *reinterpret_cast<float4 *>(f) = reinterpret_cast<const float4 *>(src)[0];
            *reinterpret_cast<float4 *>(f + 4) = reinterpret_cast<const float4 *>(src)[1];
        } else {
            f[0] = *src;
        }
    }
    __device__ void load_one(const void *base, int64_t at) { f[0] = static_cast<const float *>(base)[at]; }
    __device__ float value(int j) const { return f[j]; }
    static __device__ void store_one(void *base, int64_t at, float v) { static_cast<float *>(base)[at] = v; }
    static __device__ void store(void *base, int64_t at, const float (&v)[VEC])
    {
        float *dst = static_cast<float *>(base) + at;
        if constexpr (VEC == 8) {
            reinterpret_cast<float4 *>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4 *>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *dst = v[0];
        }
    }
};

// Sum over the block: lanes by shuffles, then warps in index order through
// shared memory; every thread gets the same value.
__device__ __forceinline__ float block_sum(float x, float *scratch)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        x += __shfl_xor_sync(0xffffffffu, x, o);
    const int warps = blockDim.x >> 5;
    if (warps == 1)
        return x;
    if ((threadIdx.x & 31) == 0)
        scratch[threadIdx.x >> 5] = x;
    __syncthreads();
    x = (int)(threadIdx.x & 31) < warps ? scratch[threadIdx.x & 31] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// ELEMS elements a thread in pieces of VEC, piece n at (n * threads + thread) * VEC.
// EDGES: rows of any width that lie alike in all tensors.  The pieces begin at
// the row's first 16-byte boundary; the up to 14 elements before the first and
// behind the last piece are a lane's each of one more warp, so that no warp
// runs both forms of an access.  (Rows of one CTA lie alike: a grid that walks
// is a multiple of 8.)  Not for every width: lowm_residual_norm has the rule.
// A CTA walks rows blockIdx.x, blockIdx.x + gridDim.x, ...: the weights stay in
// registers, and the next row is requested before this one's reductions.
// (LOOP false: one row a CTA, without the registers of the second.)
template <int VEC, int ELEMS, bool F32, bool LOOP, bool EDGES>
__global__ void __launch_bounds__(1024) residual_norm_kernel(const NormParams p)
{
    constexpr int NP = ELEMS / VEC;
    __shared__ float scratch[4][32];
    const bool has_gate = p.gate != nullptr, has_block = p.block != nullptr, has_post = p.post != nullptr;
    int step = (int)blockDim.x * VEC, first = (int)threadIdx.x * VEC, end = p.hidden;
    bool single = false;                     // a thread of the last warp: one element
    if constexpr (EDGES) {
        const int before = (int)(-((int64_t)blockIdx.x * p.out_stride) & 7), inner = before + (max(p.hidden - before, 0) & ~7);
        step -= 32 * VEC;
        single = threadIdx.x >= blockDim.x - 32;
        const int lane = threadIdx.x & 31;
        first = !single ? first + before : lane < before ? lane : inner + lane - before;
        if (!single)
            end = inner;
    }
    // Piece n of this thread lies in the row.
    auto has = [&](int n) { return (!EDGES || !single || n == 0) && n * step + first < end; };
    auto load_row = [&](const __nv_bfloat16 *x, Pack<VEC> &o) {
        if (EDGES && single)
            o.v[0] = *x;
        else
            load_bf16(x, o);
    };
    auto load_weight = [&](const __nv_bfloat16 *w, Pack<VEC> &o) {   // they lie apart from the rows
        if constexpr (EDGES) {
            o.v[0] = w[0];
            if (!single) {
#pragma unroll
                for (int j = 1; j < VEC; ++j)
                    o.v[j] = w[j];
            }
        } else {
            load_bf16(w, o);
        }
    };
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    struct Values {
        Pack<VEC> y[NP], g[NP];
        Residual<VEC, F32> r[NP];
    };
    auto load = [&](int64_t t, Values &v) {
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            const int i = n * step + first;
            if (!has(n))
                continue;
            if (has_block)
                load_row(p.block + t * p.block_stride + i, v.y[n]);
            if (EDGES && single)
                v.r[n].load_one(p.residual, t * p.residual_stride + i);
            else
                v.r[n].load(p.residual, t * p.residual_stride + i);
            if (has_gate && p.gate_stride)
                load_row(p.gate + t * p.gate_stride + i, v.g[n]);
        }
    };
    Values next;
#pragma unroll
    for (int n = 0; n < NP; ++n) {
        next.y[n] = {};
        next.r[n] = {};
        if (EDGES)
            next.g[n] = {};
    }
    int64_t t = blockIdx.x;
    load(t, next);
    Pack<VEC> post[NP], pre[NP];
#pragma unroll
    for (int n = 0; n < NP; ++n) {
        const int i = n * step + first;
#pragma unroll
        for (int j = 0; j < VEC; ++j)
            post[n].v[j] = pre[n].v[j] = __float2bfloat16_rn(1.f);
        if (!has(n))
            continue;
        if (has_post)
            load_weight(p.post + i, post[n]);
        if (p.pre != nullptr)
            load_weight(p.pre + i, pre[n]);
        if (has_gate && !p.gate_stride)
            load_weight(p.gate + i, next.g[n]);
    }

    for (int parity = 0;; t += gridDim.x, parity ^= 2) {
        const Values cur = next;
        if (LOOP && t + gridDim.x < p.tokens)
            load(t + gridDim.x, next);
        float inv = 1.f;
        if (has_post) {
            float sum = 0.f;
#pragma unroll
            for (int n = 0; n < NP; ++n)
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float v = __bfloat162float(cur.y[n].v[j]);
                    sum = fmaf(v, v, sum);
                }
            inv = rsqrtf(fmaf(block_sum(sum, scratch[parity]), p.inv_hidden, p.eps));
        }
        float r[NP][VEC];
        float sum = 0.f;
#pragma unroll
        for (int n = 0; n < NP; ++n)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                r[n][j] = cur.r[n].value(j);
                if (has_block) {
                    float v = __bfloat162float(cur.y[n].v[j]) * inv * __bfloat162float(post[n].v[j]);
                    if (has_gate)
                        v *= __bfloat162float(cur.g[n].v[j]);
                    r[n][j] = has(n) && (!EDGES || !single || j == 0) ? fmaf(r[n][j], p.scale, v) : 0.f;
                }
                sum = fmaf(r[n][j], r[n][j], sum);
            }
        if (has_block) {
#pragma unroll
            for (int n = 0; n < NP; ++n) {
                const int i = n * step + first;
                if (!has(n))
                    continue;
                if (EDGES && single)
                    Residual<VEC, F32>::store_one(p.out_residual, t * p.out_residual_stride + i, r[n][0]);
                else
                    Residual<VEC, F32>::store(p.out_residual, t * p.out_residual_stride + i, r[n]);
            }
        }
        inv = rsqrtf(fmaf(block_sum(sum, scratch[parity + 1]), p.inv_hidden, p.eps));
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            const int i = n * step + first;
            if (!has(n))
                continue;
            float o[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                o[j] = r[n][j] * inv * __bfloat162float(pre[n].v[j]);
            if (EDGES && single)
                p.out[t * p.out_stride + i] = __float2bfloat16_rn(o[0]);
            else
                store_bf16(p.out + t * p.out_stride + i, o);
        }
        if (!LOOP || t + gridDim.x >= p.tokens)
            return;
    }
}

template <int VEC, int ELEMS, bool LOOP, bool EDGES>
lowm_status_t launch_norm(const NormParams &p, bool f32, int grid, int threads, void *stream)
{
    return launch_pdl(f32 ? residual_norm_kernel<VEC, ELEMS, true, LOOP, EDGES>
                          : residual_norm_kernel<VEC, ELEMS, false, LOOP, EDGES>,
                      dim3((unsigned)grid), dim3((unsigned)threads), 0, stream, p);
}

// Rows a of one tensor share bytes with rows b of another.  Rows of one stride may
// lie between each other (halves of a wider matrix); other strides are told
// apart by their extents alone.
bool rows_overlap(const void *a, int64_t a_stride, int64_t a_size, const void *b, int64_t b_stride, int64_t b_size,
                  int tokens, int hidden)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    const uintptr_t nx = (uintptr_t)(((tokens - 1) * a_stride + hidden) * a_size);
    const uintptr_t ny = (uintptr_t)(((tokens - 1) * b_stride + hidden) * b_size);
    if (x >= y + ny || y >= x + nx)
        return false;
    if (a_stride * a_size != b_stride * b_size)
        return true;
    const uintptr_t stride = (uintptr_t)(a_stride * a_size), apart = y >= x ? (y - x) % stride : (stride - (x - y) % stride) % stride;
    return apart < (uintptr_t)(hidden * a_size) || stride - apart < (uintptr_t)(hidden * b_size);
}

}  // namespace
}  // namespace lowm

extern "C" lowm_status_t lowm_residual_norm(const void *residual, int residual_f32, int64_t residual_stride,
                                            const void *block, int64_t block_stride, const void *post_weight,
                                            const void *gate, int64_t gate_stride, const void *pre_weight,
                                            void *out_residual, int64_t out_residual_stride, void *out,
                                            int64_t out_stride, int tokens, int hidden, float scale, float eps,
                                            void *stream)
{
    using namespace lowm;
    constexpr int kMaxHidden = 16384;                // 1024 threads of 16 elements
    if (tokens < 0 || hidden <= 0 || !(eps >= 0.f))
        return LOWM_ERR_INVALID_ARGUMENT;
    if (hidden > kMaxHidden)
        return LOWM_ERR_UNSUPPORTED_SHAPE;
    if (block ? !out_residual : (post_weight || gate || out_residual || scale != 1.f))
        return LOWM_ERR_INVALID_ARGUMENT;
    if (tokens == 0)
        return LOWM_OK;
    if (!residual || !out)
        return LOWM_ERR_INVALID_ARGUMENT;
    if (residual_stride < 0 || block_stride < 0 || gate_stride < 0 || (out_residual && out_residual_stride < hidden) ||
        out_stride < hidden)
        return LOWM_ERR_INVALID_ARGUMENT;
    const int size = residual_f32 ? 4 : 2;
    if (!is_aligned(residual, size) || !is_aligned(out_residual, size) || !is_aligned(block, 2) ||
        !is_aligned(post_weight, 2) || !is_aligned(gate, 2) || !is_aligned(pre_weight, 2) || !is_aligned(out, 2))
        return LOWM_ERR_MISALIGNED;
    if (out_residual && rows_overlap(out_residual, out_residual_stride, size, out, out_stride, 2, tokens, hidden))
        return LOWM_ERR_INVALID_ARGUMENT;
    int sms = 0;
    const lowm_status_t st = host_check_device(&sms);
    if (st != LOWM_OK)
        return st;

    NormParams p;
    p.residual = residual;
    p.block = static_cast<const __nv_bfloat16 *>(block);
    p.post = static_cast<const __nv_bfloat16 *>(post_weight);
    p.gate = static_cast<const __nv_bfloat16 *>(gate);
    p.pre = static_cast<const __nv_bfloat16 *>(pre_weight);
    p.out_residual = out_residual;
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.residual_stride = residual_stride;
    p.block_stride = block_stride;
    p.gate_stride = gate_stride;
    p.out_residual_stride = out_residual_stride;
    p.out_stride = out_stride;
    p.hidden = hidden;
    p.tokens = tokens;
    p.scale = scale;
    p.eps = eps;
    p.inv_hidden = 1.f / (float)hidden;

    // 16-byte pieces: rows on 16-byte boundaries throughout, or (edges) rows that lie alike in all tensors.
    const bool bases = is_aligned(residual, 16) && is_aligned(block, 16) && is_aligned(out_residual, 16) &&
                       is_aligned(out, 16) && (!gate_stride || is_aligned(gate, 16));
    const int64_t rmod = residual_f32 ? 3 : 7;
    const bool vec = bases && hidden % 8 == 0 && !((residual_stride | out_residual_stride) & rmod) &&
                     !((block_stride | gate_stride | out_stride) & 7) && is_aligned(post_weight, 16) &&
                     is_aligned(gate, 16) && is_aligned(pre_weight, 16);
    auto alike = [&](bool used, int64_t stride) { return !used || ((stride - out_stride) & 7) == 0; };
    const bool lie_alike = bases && alike(true, residual_stride) && alike(block != nullptr, block_stride) &&
                           alike(out_residual != nullptr, out_residual_stride) && alike(gate_stride != 0, gate_stride) &&
                           hidden <= kMaxHidden - 512;   // 31 warps and the edges'
    const bool f32 = residual_f32 != 0;
    auto elems_of = [&](bool e) { return hidden <= (e ? kMaxHidden - 512 : kMaxHidden) / 2 ? 8 : 16; };
    auto threads_of = [&](bool e) { return ((hidden + elems_of(e) - 1) / elems_of(e) + 31) / 32 * 32 + (e ? 32 : 0); };
    // With edges or element by element?  The pieces save instructions and the edges cost a warp, which can cost an SM
    // one of its CTAs (of 1024 threads) and then loses where rows are many and bring much (GB300, element by element ->
    // edges; fp32 residual and a gate per token: 8000 x 4095 105 -> 143 us, 8000 x 601 18.0 -> 20.2, 1000 x 999 5.0 -> 5.7,
    // but 8000 x 3001, as many CTAs, 87.1 -> 81.8, and 1000 x 513, one round, 4.3 -> 3.5).  Rows that bring little gain
    // all the same down to two CTAs an SM (bf16 without a gate: 8000 x 2305 53.3 -> 44.7, 8000 x 601 15.1 -> 12.0; with a
    // post weight 17.3 -> 15.7, but 8000 x 4095, one CTA, 102 -> 114); those of one warp do not (8000 x 65 8.6 -> 9.1), and
    // below 128 elements nothing does.  Where the edges' warp makes it 16 elements a thread instead of 8, bare rows alone
    // gain (8000 x 8191 208 -> 192, with a post weight 239 -> 245, with all 255 -> 331).
    bool edges = !vec && lie_alike && hidden > 128;
    if (edges) {
        const int with = threads_of(true), ctas = 1024 / with;
        const int streams = 1 + f32 + (gate_stride != 0) + (post_weight != nullptr);
        edges = elems_of(true) != elems_of(false) ? streams == 1
                                                  : tokens <= sms * ctas || ctas == 1024 / threads_of(false) ||
                                                        (streams <= 2 && with > 64 && ctas >= 2);
    }
    const int elems = elems_of(edges), threads = threads_of(edges);
    if (elems == 16)
        return vec     ? launch_norm<8, 16, false, false>(p, f32, tokens, threads, stream)
               : edges ? launch_norm<8, 16, false, true>(p, f32, tokens, threads, stream)
                       : launch_norm<1, 16, false, false>(p, f32, tokens, threads, stream);
    if (!vec && !edges)
        return launch_norm<1, 8, false, false>(p, f32, tokens, threads, stream);
    // Walking rows pays from two rounds of 1024 threads an SM on, for rows of 256
    // threads and more (GB300, one row a CTA -> walking: 8192 x 4096 57.3 -> 43.7
    // us, 2000 x 8000 40.3 -> 29.2; 8000 x 600, 96 threads, 10.2 -> 12.5; 600 x
    // 4096, two rounds, 5.0 both), and of 192 where it saves single loads of
    // weights (6293 x 1313 35.7 -> 30.2; 2000 x 1001, 160 threads, 7.3 -> 8.4).  768
    // or 1536 threads an SM lose at 8192 x 4096 (54.9, 52.9 us).
    const int resident = sms * (1024 / threads);
    if (threads < (edges ? 192 : 256) || tokens <= 2 * resident)
        return vec ? launch_norm<8, 8, false, false>(p, f32, tokens, threads, stream)
                   : launch_norm<8, 8, false, true>(p, f32, tokens, threads, stream);
    const int rounds = (tokens + resident - 1) / resident, grid = (tokens + rounds - 1) / rounds;
    return vec ? launch_norm<8, 8, true, false>(p, f32, grid, threads, stream)
               : launch_norm<8, 8, true, true>(p, f32, std::max(8, grid / 8 * 8), threads, stream);
}
