// The 8-bit low-M GEMM with scales by block of 128 (lowm_fp8.h), and the
// quantisation that feeds it.
//
// C^T tiles: N lies on the MMA's M (128 rows of W, one block row of its scales),
// the few tokens on its N.  A CTA streams its share of K for one tile: a TMA warp
// fills a ring of K blocks (128 bytes a row, 128-byte swizzled) of W and A, one
// thread issues four tcgen05.mma (kind::f8f6f4, K = 32) a block into one of a ring
// of TMEM buffers, and the epilogue warps add the block's sums, times the block's
// two scales, to fp32 sums in registers.  So a block's products are summed by the
// tensor cores and blocks in fp32, which the scales require anyway.
//
// K is split over the CTAs of a cluster where the tiles alone would leave SMs
// idle.  They exchange their sums through distributed shared memory, the drained
// ring serving as mailbox: rank q adds those of its share of the tokens, in the
// order of the ranks, and stores them.
#include <cuda_bf16.h>

#include <algorithm>
#include <cstdlib>

#include "../../include/lowm_fp8.h"
#include "fp8_device.cuh"
#include "layer_device.cuh"
#include "layer_host.h"

namespace lowm {
namespace {

constexpr int kTileN = 128, kBlock = 128;    // rows of W a tile, K a block
constexpr int kMaxSplit = 8;

// Bits of the device status word (above those of the other operators).
enum : uint32_t {
    kErrGemm8Ring = 1u << 25,
    kErrGemm8Full = 1u << 26,
    kErrGemm8Sums = 1u << 27,
    kErrGemm8Free = 1u << 28,
    kErrGemm8Base = 1u << 29,                // dynamic shared memory not on a 1024-byte boundary
};

struct Gemm8Params {
    const float *a_scale, *w_scale;
    __nv_bfloat16 *c;
    int M, N, blocks;                        // blocks of K
    int per_stage, stages;                   // K blocks a ring stage, ring stages
    int planes;                              // the tensor maps have the K blocks as a third dimension
    unsigned flags;
    unsigned int *status;
};

template <int M_PAD>
struct Gemm8Shape {
    static constexpr int kEpilogueWarps = M_PAD > 64 ? 8 : 4;
    static constexpr int kThreads = 64 + 32 * kEpilogueWarps;
    static constexpr int kColumns = M_PAD / (kEpilogueWarps / 4);        // tokens a thread sums
    static constexpr int kBuffers = M_PAD > 64 ? 2 : 4;                  // of TMEM
    static constexpr uint32_t kTmem = kBuffers * M_PAD < 32 ? 32 : kBuffers * M_PAD;
    static constexpr uint32_t kWBytes = kTileN * kBlock, kABytes = M_PAD * kBlock;   // of a K block
    static constexpr uint32_t kScaleBytes = (M_PAD + 4) * 4;             // a K block's scales: tokens, then the tile's
    __host__ __device__ static constexpr uint32_t stage_bytes(int per_stage) { return per_stage * (kWBytes + kABytes); }
};

// Instruction descriptor, kind::f8f6f4: fp32 accumulator, e4m3 A and B, both K-major.
__host__ __device__ constexpr uint32_t make_idesc_e4m3(int m, int n)
{
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

__device__ __forceinline__ void mma_e4m3_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void copy_async_4(uint32_t dst, const float *src, uint32_t bytes)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void copies_arrive(uint32_t bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void st_cluster(uint32_t addr, float v)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

__device__ __forceinline__ uint32_t cluster_size()
{
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
    return n;
}

__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

template <int M_PAD>
__global__ void __launch_bounds__(Gemm8Shape<M_PAD>::kThreads)
    gemm_fp8_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a, const Gemm8Params p)
{
    using S = Gemm8Shape<M_PAD>;
    constexpr uint32_t kMaxStages = 16;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = ptx::smem_u32(smem);
    const uint32_t stage_bytes = S::stage_bytes(p.per_stage), a_at = p.per_stage * S::kWBytes;
    const uint32_t scales_at = p.stages * stage_bytes, scale_stage = p.per_stage * S::kScaleBytes;
    const uint32_t bars = sbase + scales_at + p.stages * scale_stage;
    const uint32_t bar_full = bars, bar_empty = bars + 8 * kMaxStages, bar_sums = bar_empty + 8 * kMaxStages,
                   bar_free = bar_sums + 8 * S::kBuffers, bar_drain = bar_free + 8 * S::kBuffers, slot = bar_drain + 8;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ranks = (int)cluster_size(), rank = (int)ptx::cluster_ctarank();
    const int n0 = (int)(blockIdx.x / ranks) * kTileN;
    // This rank's stages of K.
    const int all = (p.blocks + p.per_stage - 1) / p.per_stage;
    const int begin = (int)((int64_t)all * rank / ranks), end = (int)((int64_t)all * (rank + 1) / ranks);
    if (sbase & 1023u) {                     // (the same for every CTA)
        if (threadIdx.x == 0)
            atomicOr(p.status, kErrGemm8Base);
        return;
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            ptx::mbar_init(bar_full + 8 * s, 1 + 32);                     // codes, and each lane's scales
            ptx::mbar_init(bar_empty + 8 * s, 1 + S::kEpilogueWarps);
        }
        for (int b = 0; b < S::kBuffers; ++b) {
            ptx::mbar_init(bar_sums + 8 * b, 1);
            ptx::mbar_init(bar_free + 8 * b, S::kEpilogueWarps);
        }
        ptx::mbar_init(bar_drain, 1);
        ptx::fence_mbarrier_init_cluster();
        ptx::fence_proxy_async_shared();
    }
    if (warp == 1) {
        ptx::tmem_alloc(slot, S::kTmem);
        ptx::tmem_relinquish_alloc_permit();
        ptx::tcgen05_fence_before_thread_sync();
    }
    __syncthreads();
    ptx::tcgen05_fence_after_thread_sync();
    const uint32_t tmem = ptx::ld_volatile_shared(slot);

    float acc[S::kColumns] = {};
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t parity, uint32_t err) {
        if (!wait_short(bar, parity)) {
            ok = false;
            atomicOr(p.status, err);
        }
        ok = __all_sync(0xffffffffu, ok);
    };
    if (warp == 0) {
        // ------------------------------------------------------------ loads
        const uint64_t first = ptx::policy_evict_first(), last = ptx::policy_evict_last();
        auto load = [&](const CUtensorMap *map, uint32_t to, uint32_t block_bytes, int row, int stage, uint32_t bar, uint64_t policy) {
            if (p.planes) {
                ptx::tma_load_3d(to, map, 0, row, stage * p.per_stage, bar, policy);
            } else {
                for (int b = 0; b < p.per_stage && stage * p.per_stage + b < p.blocks; ++b)
                    ptx::tma_load_2d(to + b * block_bytes, map, (stage * p.per_stage + b) * kBlock, row, bar, policy);
            }
        };
        auto expect = [&](int stage, uint32_t bar) {
            const int n = p.planes ? p.per_stage : min(p.per_stage, p.blocks - stage * p.per_stage);
            ptx::mbar_arrive_expect_tx(bar, n * (S::kWBytes + S::kABytes));
        };
        // What does not depend on the kernel before this one: with the caller's promise W of the first ring.
        const int early = p.flags & LOWM_FLAG_W_BEFORE_PDL_WAIT ? min(p.stages, end - begin) : 0;
        if (lane == 0) {
            ptx::prefetch_tensormap(&map_w);
            ptx::prefetch_tensormap(&map_a);
            for (int i = 0; i < early; ++i) {
                expect(begin + i, bar_full + 8 * i);
                load(&map_w, sbase + i * stage_bytes, S::kWBytes, n0, begin + i, bar_full + 8 * i, first);
            }
        }
        ptx::griddep_wait();
        int i = 0;
        for (; begin + i < end; ++i) {
            const int s = i % p.stages;
            wait(bar_empty + 8 * s, ((i / p.stages) & 1) ^ 1, kErrGemm8Ring);
            if (!ok)
                break;
            if (lane == 0) {
                const uint32_t bar = bar_full + 8 * s, to = sbase + s * stage_bytes;
                if (i >= early) {
                    expect(begin + i, bar);
                    load(&map_w, to, S::kWBytes, n0, begin + i, bar, first);
                }
                load(&map_a, to + a_at, S::kABytes, 0, begin + i, bar, last);
            }
            __syncwarp();
            for (int b = 0; b < p.per_stage; ++b) {
                const int block = (begin + i) * p.per_stage + b;
                const uint32_t to = sbase + scales_at + s * scale_stage + b * S::kScaleBytes;
                if (block >= p.blocks)
                    break;
                for (int m = lane; m < M_PAD; m += 32)
                    copy_async_4(to + 4 * m, p.a_scale + (int64_t)min(m, p.M - 1) * p.blocks + block, m < p.M ? 4 : 0);
                if (lane == 0)
                    copy_async_4(to + 4 * M_PAD, p.w_scale + (int64_t)(n0 / kTileN) * p.blocks + block, 4);
            }
            copies_arrive(bar_full + 8 * s);
        }
        ptx::griddep_launch_dependents();
        // No copy may land after the ring has become the mailbox: normally all were consumed.
        for (int j = max(i - p.stages, 0); j < i; ++j)
            (void)wait_short(bar_full + 8 * (j % p.stages), (j / p.stages) & 1);
        if (!ok && i < early)                // W that was requested before a wait gave up: its barrier stays open
            (void)wait_short(bar_full + 8 * i, 0);
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMAs
        constexpr uint32_t kIdesc = make_idesc_e4m3(kTileN, M_PAD);
        const uint32_t base = uniform(tmem);
        int g = 0;                           // K blocks
        for (int i = 0; begin + i < end && ok; ++i) {
            const int s = i % p.stages;
            wait(bar_full + 8 * s, (i / p.stages) & 1, kErrGemm8Full);
            const int n = min(p.per_stage, p.blocks - (begin + i) * p.per_stage);
            for (int b = 0; b < n && ok; ++b, ++g) {
                const uint32_t buffer = g % S::kBuffers;
                wait(bar_free + 8 * buffer, ((g / S::kBuffers) & 1) ^ 1, kErrGemm8Free);
                if (!ok)
                    break;
                ptx::tcgen05_fence_after_thread_sync();
                const uint64_t w = make_sw128_kmajor_desc(sbase + s * stage_bytes + b * S::kWBytes);
                const uint64_t a = make_sw128_kmajor_desc(sbase + s * stage_bytes + a_at + b * S::kABytes);
                if (ptx::elect_one_sync()) {
#pragma unroll
                    for (uint32_t k = 0; k < 4; ++k)
                        mma_e4m3_ss(base + buffer * M_PAD, w + 2 * k, a + 2 * k, kIdesc, k > 0);
                    ptx::tcgen05_commit(bar_sums + 8 * buffer);
                    if (b + 1 == n)
                        ptx::tcgen05_commit(bar_empty + 8 * s);
                }
                __syncwarp();
            }
        }
        if (ptx::elect_one_sync())
            ptx::tcgen05_commit(bar_drain);
        __syncwarp();
        (void)wait_short(bar_drain, 0);      // nothing writes TMEM any more
    } else {
        // ------------------------------------------------------------ sums: thread = row of W = TMEM lane
        const int quarter = warp & 3, column0 = (warp - 2) / 4 * S::kColumns;
        const uint32_t from = tmem + ((uint32_t)(32 * quarter) << 16) + column0;
        int g = 0;
        for (int i = 0; begin + i < end && ok; ++i) {
            const int s = i % p.stages;
            wait(bar_full + 8 * s, (i / p.stages) & 1, kErrGemm8Full);    // the scales
            const int n = min(p.per_stage, p.blocks - (begin + i) * p.per_stage);
            for (int b = 0; b < n && ok; ++b, ++g) {
                const uint32_t buffer = g % S::kBuffers;
                wait(bar_sums + 8 * buffer, (g / S::kBuffers) & 1, kErrGemm8Sums);
                if (!ok)
                    break;
                ptx::tcgen05_fence_after_thread_sync();
                const float *scales = reinterpret_cast<const float *>(smem + scales_at + s * scale_stage + b * S::kScaleBytes);
                const float w = scales[M_PAD];
                uint32_t d[S::kColumns / 16][16];
#pragma unroll
                for (int c = 0; c < S::kColumns / 16; ++c)
                    tmem_ld_x16(from + buffer * M_PAD + 16 * c, d[c]);
                ptx::tmem_wait_ld();
                ptx::tcgen05_fence_before_thread_sync();
                __syncwarp();
                if (lane == 0)
                    ptx::mbar_arrive(bar_free + 8 * buffer);
#pragma unroll
                for (int c = 0; c < S::kColumns; c += 4) {
                    const float4 a = *reinterpret_cast<const float4 *>(scales + column0 + c);
                    acc[c] = fmaf(__uint_as_float(d[c / 16][c % 16]), a.x * w, acc[c]);
                    acc[c + 1] = fmaf(__uint_as_float(d[c / 16][c % 16 + 1]), a.y * w, acc[c + 1]);
                    acc[c + 2] = fmaf(__uint_as_float(d[c / 16][c % 16 + 2]), a.z * w, acc[c + 2]);
                    acc[c + 3] = fmaf(__uint_as_float(d[c / 16][c % 16 + 3]), a.w * w, acc[c + 3]);
                }
            }
            __syncwarp();
            if (lane == 0)
                ptx::mbar_arrive(bar_empty + 8 * s);
        }
    }
    __syncwarp();
    ptx::tcgen05_fence_before_thread_sync();
    __syncthreads();                         // every MMA has been read, every copy has landed
    if (warp == 1) {
        ptx::tcgen05_fence_after_thread_sync();
        ptx::tmem_dealloc(tmem, S::kTmem);
    }
    const int quarter = warp & 3, column0 = (warp - 2) / 4 * S::kColumns;
    const int row = 32 * quarter + lane;
    if (ranks == 1) {
        if (warp >= 2 && n0 + row < p.N) {
#pragma unroll
            for (int c = 0; c < S::kColumns; ++c)
                if (column0 + c < p.M)
                    p.c[(int64_t)(column0 + c) * p.N + n0 + row] = __float2bfloat16_rn(acc[c]);
        }
        return;
    }
    // Rank q's mailbox: [source rank][its tokens][128 rows].
    const int tokens = M_PAD / ranks;
    ptx::cluster_arrive_release();
    ptx::cluster_wait_acquire();
    if (warp >= 2) {
#pragma unroll
        for (int c = 0; c < S::kColumns; ++c) {
            const int m = column0 + c, to = m / tokens;
            if (m < p.M)
                st_cluster(ptx::mapa_shared(sbase + ((rank * tokens + m - to * tokens) * kTileN + row) * 4, to), acc[c]);
        }
    }
    ptx::cluster_arrive_release();
    ptx::cluster_wait_acquire();
    if (warp >= 2 && n0 + row < p.N) {
        for (int m = (warp - 2) / 4; m < tokens && rank * tokens + m < p.M; m += S::kEpilogueWarps / 4) {
            float sum = 0.f;
            for (int r = 0; r < ranks; ++r)
                sum += reinterpret_cast<const float *>(smem)[(r * tokens + m) * kTileN + row];
            p.c[(int64_t)(rank * tokens + m) * p.N + n0 + row] = __float2bfloat16_rn(sum);
        }
    }
}

// ------------------------------------------------------------------ quantisation
// Activations: a warp has 128 columns of a row, a lane four of them.  Bound by the launch and one memory latency at the
// few rows it is for.
template <bool VEC>
__global__ void __launch_bounds__(256)
    quantize_rows_kernel(const __nv_bfloat16 *x, int64_t stride, uint8_t *codes, float *scales, int rows, int cols, int blocks)
{
    const int lane = threadIdx.x & 31;
    const int64_t at = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int64_t row = at / blocks;
    const int block = (int)(at - row * blocks), c0 = block * 128 + 4 * lane;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    if (row >= rows)
        return;
    float v[4];
    const __nv_bfloat16 *from = x + row * stride + c0;
    if (VEC && c0 < cols) {                  // (cols a multiple of 4)
        const uint2 u = *reinterpret_cast<const uint2 *>(from);
        const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.x));
        const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.y));
        v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = !VEC && c0 + i < cols ? __bfloat162float(from[i]) : 0.f;
    }
    float amax = fmaxf(fmaxf(finite_magnitude(v[0]), finite_magnitude(v[1])), fmaxf(finite_magnitude(v[2]), finite_magnitude(v[3])));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const int e = scale_exponent(amax);
    const float inverse = power_of_two(-e);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = nan_unless_finite(v[i]) * inverse;
    const uint32_t word = to_e4m3x2(v[0], v[1]) | to_e4m3x2(v[2], v[3]) << 16;
    uint8_t *to = codes + row * cols + c0;
    if (VEC) {
        if (c0 < cols)
            *reinterpret_cast<uint32_t *>(to) = word;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c0 + i < cols)
                to[i] = (uint8_t)(word >> (8 * i));
    }
    if (lane == 0)
        scales[row * blocks + block] = power_of_two(e);
}

// Weights: a CTA has a block of 128 rows and 128 columns, read twice (the second time from the caches).
__global__ void __launch_bounds__(256)
    quantize_blocks_kernel(const __nv_bfloat16 *x, int64_t stride, uint8_t *codes, float *scales, int rows, int cols, int blocks)
{
    __shared__ float tops[8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row0 = (int64_t)(blockIdx.x / blocks) * 128;
    const int block = (int)(blockIdx.x % blocks);
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    float amax = 0.f;
    for (int r = warp; r < 128 && row0 + r < rows; r += 8)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = block * 128 + 32 * i + lane;
            if (c < cols)
                amax = fmaxf(amax, finite_magnitude(__bfloat162float(x[(row0 + r) * stride + c])));
        }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (lane == 0)
        tops[warp] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i)
        amax = fmaxf(amax, tops[i]);
    const int e = scale_exponent(amax);
    const float inverse = power_of_two(-e);
    for (int r = warp; r < 128 && row0 + r < rows; r += 8)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = block * 128 + 32 * i + lane;
            if (c < cols)
                codes[(row0 + r) * cols + c] =
                    (uint8_t)to_e4m3x2(nan_unless_finite(__bfloat162float(x[(row0 + r) * stride + c])) * inverse, 0.f);
        }
    if (threadIdx.x == 0)
        scales[blockIdx.x] = power_of_two(e);
}

// [rows, K] codes in boxes of `box_rows` rows and 128 columns, with the blocks of K as a third dimension (`per_stage` of
// them a box) where K is a whole number of them; zeros outside.
lowm_status_t encode_matrix(const void *base, int rows, int K, int box_rows, int per_stage, bool planes, CUtensorMap *map)
{
    EncodeTiledFn enc = host_encode_fn();
    if (!enc)
        return LOWM_ERR_CUDA;
    const cuuint64_t dims3[3] = {kBlock, (cuuint64_t)rows, (cuuint64_t)(K / kBlock)}, strides3[2] = {(cuuint64_t)K, kBlock};
    const cuuint64_t dims2[2] = {(cuuint64_t)K, (cuuint64_t)rows}, strides2[1] = {(cuuint64_t)K};
    const cuuint32_t box[3] = {kBlock, (cuuint32_t)box_rows, (cuuint32_t)per_stage}, step[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, planes ? 3 : 2, const_cast<void *>(base), planes ? dims3 : dims2,
               planes ? strides3 : strides2, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? LOWM_OK
               : LOWM_ERR_CUDA;
}

constexpr int kSmem = 227 * 1024;

template <int M_PAD>
lowm_status_t launch_gemm_fp8(const void *A, const void *W, Gemm8Params &p, int K, int sms, void *stream)
{
    using S = Gemm8Shape<M_PAD>;
    const int tiles = (p.N + kTileN - 1) / kTileN;
    int split = 1;
    while (split < kMaxSplit && tiles * split * 2 <= 2 * sms && p.blocks >= 4 * split)
        split *= 2;
    if (const char *e = getenv("LOWM8_SPLIT"))
        split = atoi(e);
    const bool two = tiles * split > sms;                                // CTAs an SM
    const int share = (p.blocks + split - 1) / split;
    p.per_stage = 1;
    if (const char *e = getenv("LOWM8_KB"))
        p.per_stage = atoi(e);
    const int overhead = 1024;                                           // barriers
    const int budget = two ? kSmem / 2 - 1024 : kSmem;
    auto bytes_of = [](int blocks) { return (int)S::stage_bytes(blocks) + blocks * (int)S::kScaleBytes; };
    while (p.per_stage > 1 && 2 * bytes_of(p.per_stage) > budget - overhead)
        p.per_stage /= 2;
    const int stage = bytes_of(p.per_stage);
    p.stages = std::min({(budget - overhead) / stage, (share + p.per_stage - 1) / p.per_stage, 16});
    p.planes = K % kBlock == 0;
    // The ring is the mailbox, too.
    const int ring = std::max(p.stages * stage, split > 1 ? M_PAD * kTileN * 4 : 0);
    const int bytes = std::max(ring, p.stages * stage) + overhead;
    CUtensorMap map_w, map_a;
    lowm_status_t st = encode_matrix(W, p.N, K, kTileN, p.per_stage, p.planes, &map_w);
    if (st == LOWM_OK)
        st = encode_matrix(A, p.M, K, M_PAD, p.per_stage, p.planes, &map_a);
    if (st != LOWM_OK)
        return st;
    static SmemOptIn opt_in;
    if (!opt_in.set(reinterpret_cast<const void *>(gemm_fp8_kernel<M_PAD>), kSmem))
        return LOWM_ERR_CUDA;
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3((unsigned)(tiles * split));
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = split;
    attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
    cfg.attrs = attrs;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, gemm_fp8_kernel<M_PAD>, map_w, map_a, p) == cudaSuccess ? LOWM_OK : LOWM_ERR_CUDA;
}

}  // namespace
}  // namespace lowm

extern "C" lowm_status_t lowm_quantize_fp8(const void *x, int64_t x_stride, void *codes, float *scales, int rows, int cols,
                                           int block_rows, void *stream)
{
    using namespace lowm;
    if (rows < 0 || cols <= 0 || x_stride < 0 || (block_rows != 1 && block_rows != 128))
        return LOWM_ERR_INVALID_ARGUMENT;
    const int blocks = (cols - 1) / 128 + 1;
    const int64_t ctas = block_rows == 1 ? ((int64_t)rows * blocks + 7) / 8 : ((int64_t)rows + 127) / 128 * blocks;
    if (ctas > 0x7fffffff)
        return LOWM_ERR_UNSUPPORTED_SHAPE;
    if (rows == 0)
        return LOWM_OK;
    if (!x || !codes || !scales)
        return LOWM_ERR_INVALID_ARGUMENT;
    if (!is_aligned(x, 2) || !is_aligned(scales, 4))
        return LOWM_ERR_MISALIGNED;
    int sms = 0;
    const lowm_status_t st = host_check_device(&sms);
    if (st != LOWM_OK)
        return st;
    const bool vec = is_aligned(x, 8) && is_aligned(codes, 4) && !((x_stride | cols) & 3);
    auto fn = block_rows == 128 ? quantize_blocks_kernel : (vec ? quantize_rows_kernel<true> : quantize_rows_kernel<false>);
    return launch_pdl(fn, dim3((unsigned)ctas), dim3(256), 0, stream, static_cast<const __nv_bfloat16 *>(x), x_stride,
                      static_cast<uint8_t *>(codes), scales, rows, cols, blocks);
}

extern "C" lowm_status_t lowm_gemm_fp8(const void *A, const float *a_scale, const void *W, const float *w_scale, void *C, int M,
                                       int N, int K, unsigned flags, void *stream)
{
    using namespace lowm;
    if (M <= 0 || N <= 0 || K <= 0 || (flags & ~(unsigned)LOWM_FLAG_W_BEFORE_PDL_WAIT))
        return LOWM_ERR_INVALID_ARGUMENT;
    if (M > 128 || K % 16 || N > (1 << 30))
        return LOWM_ERR_UNSUPPORTED_SHAPE;
    if (!A || !a_scale || !W || !w_scale || !C)
        return LOWM_ERR_INVALID_ARGUMENT;
    if (!is_aligned(A, 16) || !is_aligned(W, 16) || !is_aligned(C, 2) || !is_aligned(a_scale, 4) || !is_aligned(w_scale, 4))
        return LOWM_ERR_MISALIGNED;
    int sms = 0;
    const lowm_status_t st = host_check_device(&sms);
    if (st != LOWM_OK)
        return st;
    Gemm8Params p;
    std::memset(&p, 0, sizeof p);
    p.a_scale = a_scale;
    p.w_scale = w_scale;
    p.c = static_cast<__nv_bfloat16 *>(C);
    p.M = M;
    p.N = N;
    p.blocks = (K + kBlock - 1) / kBlock;
    p.flags = flags;
    p.status = host_status_word();
    if (!p.status)
        return LOWM_ERR_CUDA;
    return M <= 16   ? launch_gemm_fp8<16>(A, W, p, K, sms, stream)
           : M <= 32 ? launch_gemm_fp8<32>(A, W, p, K, sms, stream)
           : M <= 64 ? launch_gemm_fp8<64>(A, W, p, K, sms, stream)
                     : launch_gemm_fp8<128>(A, W, p, K, sms, stream);
}
