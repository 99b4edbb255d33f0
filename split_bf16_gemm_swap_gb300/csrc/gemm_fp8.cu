// The 8-bit low-M GEMM with scales by block of 128 (lowm_fp8.h), and the
// quantisation that feeds it.
//
// C^T tiles: N lies on the MMA's M (128 rows of W, one block row of its scales),
// the few tokens on its N.  A CTA streams its share of K for a tile: a TMA warp
// fills a ring of W, another (or four that quantise bf16 rows on the way) of A and
// of the scales, each token's times the tile's; one thread issues four tcgen05.mma
// (kind::f8f6f4, K = 32) a block of 128 into one of a ring of TMEM buffers, and the
// epilogue warps multiply the block's sums by its scales and add them to fp32 sums
// in registers.  So a block's products are summed by the tensor cores and blocks in
// fp32, which scales of any size require anyway.
//
// Where the tiles alone would leave SMs idle K is split over the CTAs of a cluster.
// They exchange their sums by asynchronous stores into distributed shared memory (at
// 64 tokens and more into the drained ring): rank q adds those of its share of the
// tokens, in the order of the ranks, and stores them.  Else a CTA keeps its SM and
// has every so manieth tile.
//
// What bounds it.  Few tokens: the bandwidth of W (4 tokens, N 49152, K 4096: 34 us,
// 88 % of the copy rate) and, with few tiles, the chain from the launch to the first
// block and from the last to the exchange (N 6144: 6.7 us, floor 3.7).  128 tokens: the
// epilogue, 128 x 128 sums a block (N 49152: 46.6 us, floor 31.8).  What a step was
// worth: no divisions for the ring's places (a stage 1000 -> 800 cycles), two blocks a
// copy, scales on a ring of their own, so that W's stages come back with the MMAs (64
// tokens 73 -> 45 us), 32 sums a tcgen05.ld and the stage's two waits at once (128
// tokens 59 -> 47 us).  Sixteen epilogue warps instead of eight lost (69 us for 62).
#include <cuda_bf16.h>

#include <algorithm>

#include "../../include/lowm_fp8.h"
#include "fp8_device.cuh"
#include "layer_device.cuh"
#include "layer_host.h"

namespace lowm {
namespace {

constexpr int kTileN = 128, kBlock = 128;    // rows of W a tile, K a block
constexpr int kMaxSplit = 8;
constexpr int kBuffers = 4;                  // of a K block's sums in TMEM: two stages of two blocks, or four of one
// A stage's scales stay until they have been used: behind the ring's stages, those of the sums in TMEM and one more, since a
// load of stage i means that stage i - stages has been multiplied, so that the sums of the kBuffers before it have been
// read and all but the last of those used.
constexpr uint32_t kMaxStages = 16, kMaxScales = kMaxStages + kBuffers + 1;
constexpr uint32_t kRingAt = 1024;           // (the barriers take 520 bytes)

// Bits of the device status word (above those of the other operators).
enum : uint32_t {
    kErrGemm8Ring = 1u << 25,
    kErrGemm8Full = 1u << 26,
    kErrGemm8Sums = 1u << 27,
    kErrGemm8Free = 1u << 28,
    kErrGemm8Base = 1u << 29,                // dynamic shared memory not on a 1024-byte boundary
    kErrGemm8Mail = 1u << 30,
};

struct Gemm8Params {
    const float *a_scale, *w_scale;          // a_scale: codes
    const __nv_bfloat16 *x;                  // or the activations themselves (QUANT)
    int64_t x_stride;
    bool x_vec;                              // 8-byte loads
    __nv_bfloat16 *c;
    int M, N, K, blocks;                     // blocks of K
    int per_stage, stages;                   // K blocks a ring stage, ring stages
    int planes;                              // the tensor maps have the K blocks as a third dimension
    int mailbox, apart;                      // offset of the ranks' mailbox; not the drained ring
    unsigned flags;
    unsigned int *status;
};

// Warps: 0 requests W, 1 issues MMAs, then the epilogue's, then those that bring A and the scales.
template <int M_PAD, bool QUANT>
struct Gemm8Shape {
    static constexpr int kColumns = M_PAD < 32 ? M_PAD : (M_PAD < 128 ? 32 : 64);    // tokens a thread sums
    static constexpr int kEpilogueWarps = 4 * (M_PAD / kColumns);
    static constexpr int kLoadWarp = 2 + kEpilogueWarps, kLoadWarps = QUANT ? 4 : 1;
    static constexpr int kThreads = 32 * (kLoadWarp + kLoadWarps);
    static constexpr uint32_t kTmem = kBuffers * M_PAD;
    static constexpr uint32_t kWBytes = kTileN * kBlock, kABytes = M_PAD * kBlock;   // of a K block
    static constexpr uint32_t kScaleBytes = M_PAD * 4;                   // a K block's: each token's scale times the tile's
    static_assert(!QUANT || M_PAD == 16, "four rows a warp");
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

__device__ __forceinline__ uint32_t cluster_size()
{
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
    return n;
}

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[N])
{
    if constexpr (N == 16)
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
              "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
            : "r"(taddr)
            : "memory");
    else
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

// A place in a ring and the parity of its phase, without a division a step (two of them took 200 of a stage's 1000 cycles).
struct RingPlace {
    uint32_t at = 0, phase = 0;
    __device__ __forceinline__ void step(uint32_t places)
    {
        if (++at == places) {
            at = 0;
            phase ^= 1;
        }
    }
};

// Four rows of activations, 128 columns each, as one warp quantises them: a lane has four columns.
struct FourRows {
    uint2 v[4];

    __device__ __forceinline__ void load(const Gemm8Params &p, int row0, int column)
    {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            v[r] = make_uint2(0, 0);
            if (row0 + r >= p.M || column >= p.K)            // (K is a multiple of 16)
                continue;
            const __nv_bfloat16 *x = p.x + (row0 + r) * p.x_stride + column;
            if (p.x_vec) {
                v[r] = *reinterpret_cast<const uint2 *>(x);
            } else {
                const uint16_t *e = reinterpret_cast<const uint16_t *>(x);
                v[r] = make_uint2(e[0] | (uint32_t)e[1] << 16, e[2] | (uint32_t)e[3] << 16);
            }
        }
    }

    // Codes into rows row0.. of a swizzled block, and their scales times w.
    __device__ __forceinline__ void store(uint8_t *block, float *scales, int row0, float w) const
    {
        const int lane = threadIdx.x & 31;
        uint32_t top[4];                     // bits of the largest magnitudes (which order as these do)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            top[r] = __vmaxu2(v[r].x & 0x7fff7fffu, v[r].y & 0x7fff7fffu);
#pragma unroll
        for (int r = 0; r < 4; ++r)
            top[r] = __reduce_max_sync(0xffffffffu, max(top[r] << 16, top[r] & 0xffff0000u));
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&v[r].x));
            float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&v[r].y));
            if (top[r] >= 0x7f800000u) {     // not all are finite
                const float m = fmaxf(fmaxf(finite_magnitude(a.x), finite_magnitude(a.y)),
                                      fmaxf(finite_magnitude(b.x), finite_magnitude(b.y)));
                top[r] = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
                a = make_float2(nan_unless_finite(a.x), nan_unless_finite(a.y));
                b = make_float2(nan_unless_finite(b.x), nan_unless_finite(b.y));
            }
            const int e = scale_exponent(__uint_as_float(top[r])), row = row0 + r;
            const float inverse = power_of_two(-e);
            *reinterpret_cast<uint32_t *>(block + row * kBlock + (((lane >> 2) ^ (row & 7)) << 4) + (lane & 3) * 4) =
                to_e4m3x2(a.x * inverse, a.y * inverse) | to_e4m3x2(b.x * inverse, b.y * inverse) << 16;
            if (lane == 0)
                scales[row] = power_of_two(e) * w;
        }
    }
};

template <int M_PAD, bool QUANT>
__global__ void __launch_bounds__(Gemm8Shape<M_PAD, QUANT>::kThreads, M_PAD > 32 ? 1 : 2)
    gemm_fp8_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a, const Gemm8Params p)
{
    using S = Gemm8Shape<M_PAD, QUANT>;
    extern __shared__ __align__(1024) uint8_t smem[];
    // [barriers, 1 KiB][ring of W and A][ring of scales][mailbox, if apart].
    const uint32_t sbase = ptx::smem_u32(smem), ring = sbase + kRingAt;
    const uint32_t a_at = p.per_stage * S::kWBytes, stage_bytes = a_at + p.per_stage * S::kABytes;
    const uint32_t scales_at = kRingAt + p.stages * stage_bytes, scale_stage = p.per_stage * S::kScaleBytes;
    const uint32_t bar_full = sbase, bar_empty = sbase + 8 * kMaxStages, bar_sums = bar_empty + 8 * kMaxStages,
                   bar_free = bar_sums + 8 * kBuffers, bar_drain = bar_free + 8 * kBuffers, bar_mail = bar_drain + 8,
                   bar_scales = bar_mail + 8, slot = bar_scales + 8 * kMaxScales;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ranks = (int)cluster_size(), rank = (int)ptx::cluster_ctarank();
    // A cluster has a tile; CTAs on their own have every gridDim-th one.  This rank's stages of K, and its share of the tokens.
    const int first_tile = (int)(blockIdx.x / ranks), tile_step = (int)(gridDim.x / ranks), tiles = (p.N + kTileN - 1) / kTileN;
    const int all = (p.blocks + p.per_stage - 1) / p.per_stage;
    const int begin = (int)((int64_t)all * rank / ranks), end = (int)((int64_t)all * (rank + 1) / ranks);
    const int buffers = kBuffers / p.per_stage;              // stages' sums in TMEM
    const uint32_t scale_slots = p.stages + buffers + 1;
    const int tokens = M_PAD / ranks, mine = min(max(p.M - rank * tokens, 0), tokens);
    if (sbase & 1023u) {                     // (the same for every CTA)
        if (threadIdx.x == 0)
            atomicOr(p.status, kErrGemm8Base);
        return;
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            ptx::mbar_init(bar_full + 8 * s, 1 + S::kLoadWarps);         // W, A
            ptx::mbar_init(bar_empty + 8 * s, 1);
        }
        for (uint32_t s = 0; s < scale_slots; ++s)
            ptx::mbar_init(bar_scales + 8 * s, S::kLoadWarps);
        for (int b = 0; b < kBuffers; ++b) {
            ptx::mbar_init(bar_sums + 8 * b, 1);
            ptx::mbar_init(bar_free + 8 * b, S::kEpilogueWarps);
        }
        ptx::mbar_init(bar_drain, 1);
        ptx::mbar_init(bar_mail, 1);
        ptx::fence_mbarrier_init_cluster();
        ptx::fence_proxy_async_shared();
        if (ranks > 1 && mine > 0)           // four tokens of 128 rows a store, from every rank
            ptx::mbar_arrive_expect_tx(bar_mail, ranks * ((mine + 3) / 4) * kTileN * 16);
    }
    if (warp == 1) {
        ptx::tmem_alloc(slot, S::kTmem);
        ptx::tmem_relinquish_alloc_permit();
        ptx::tcgen05_fence_before_thread_sync();
    }
    __syncthreads();
    ptx::tcgen05_fence_after_thread_sync();
    const uint32_t tmem = ptx::ld_volatile_shared(slot);
    if (ranks > 1 && p.apart)                // the others wait for this before they send
        ptx::cluster_arrive_release();

    uint64_t acc[S::kColumns / 2] = {};      // pairs of tokens
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t parity, uint32_t err) {
        if (!wait_short(bar, parity)) {
            ok = false;
            atomicOr(p.status, err);
        }
        ok = __all_sync(0xffffffffu, ok);
    };
    // One of the two operands' blocks of a stage.
    auto load = [&](const CUtensorMap *map, uint32_t to, uint32_t block_bytes, int row, int stage, uint32_t bar, uint64_t policy) {
        const int n = p.planes ? p.per_stage : min(p.per_stage, p.blocks - stage * p.per_stage);
        ptx::mbar_arrive_expect_tx(bar, n * block_bytes);
        if (p.planes) {
            ptx::tma_load_3d(to, map, 0, row, stage * p.per_stage, bar, policy);
        } else {
            for (int b = 0; b < n; ++b)
                ptx::tma_load_2d(to + b * block_bytes, map, (stage * p.per_stage + b) * kBlock, row, bar, policy);
        }
    };
    if (warp == 0) {
        // ------------------------------------------------------------ W
        const uint64_t policy = ptx::policy_evict_first();
        // With the caller's promise the first ring does not wait for the kernel before this one.
        const int early = p.flags & LOWM_FLAG_W_BEFORE_PDL_WAIT ? min(p.stages, end - begin) : 0;
        if (lane == 0) {
            ptx::prefetch_tensormap(&map_w);
            for (int i = 0; i < early; ++i)
                load(&map_w, ring + i * stage_bytes, S::kWBytes, first_tile * kTileN, begin + i, bar_full + 8 * i, policy);
            // Without it the ring's W is requested into L2, where a later write would find it.
            for (int i = early; i < min(p.stages, end - begin) && p.planes; ++i)
                ptx::tma_prefetch_3d(&map_w, 0, first_tile * kTileN, (begin + i) * p.per_stage);
        }
        ptx::griddep_wait();
        RingPlace r;
        for (int tile = first_tile; tile < tiles && ok; tile += tile_step)
            for (int i = begin; i < end; ++i, r.step(p.stages)) {
                if (tile == first_tile && i - begin < early)
                    continue;
                wait(bar_empty + 8 * r.at, r.phase ^ 1, kErrGemm8Ring);
                if (!ok)
                    break;
                if (lane == 0)
                    load(&map_w, ring + r.at * stage_bytes, S::kWBytes, tile * kTileN, i, bar_full + 8 * r.at, policy);
                __syncwarp();
            }
        ptx::griddep_launch_dependents();
    } else if (warp >= S::kLoadWarp) {
        // ------------------------------------------------------------ A and the scales
        RingPlace r, q;                      // of the ring, of the scales
        ptx::griddep_wait();
        for (int tile = first_tile; tile < tiles && ok; tile += tile_step) {
            const float *w_scale = p.w_scale + (int64_t)tile * p.blocks + begin * p.per_stage;
            int left = min(p.blocks - begin * p.per_stage, (end - begin) * p.per_stage);            // K blocks
            if constexpr (QUANT) {
                // A stage's rows (two blocks at most) are requested while those of the stage before are quantised.
                const int row0 = 4 * (warp - S::kLoadWarp);
                FourRows x[2];
                float w[2] = {};
                int column = begin * p.per_stage * kBlock + 4 * lane;
                auto fetch = [&]() {
#pragma unroll
                    for (int b = 0; b < 2; ++b)
                        if (b < p.per_stage && left > 0) {
                            x[b].load(p, row0, column);
                            w[b] = *w_scale++;
                            column += kBlock;
                            --left;
                        }
                };
                fetch();
                for (int i = begin; i < end; ++i, r.step(p.stages), q.step(scale_slots)) {
                    wait(bar_empty + 8 * r.at, r.phase ^ 1, kErrGemm8Ring);
                    if (!ok)
                        break;
                    const FourRows now[2] = {x[0], x[1]};
                    const float scale[2] = {w[0], w[1]};
                    const int n = min(p.per_stage, p.blocks - i * p.per_stage);
                    fetch();
                    uint8_t *block = smem + kRingAt + r.at * stage_bytes + a_at;
                    float *scales = reinterpret_cast<float *>(smem + scales_at + q.at * scale_stage);
#pragma unroll
                    for (int b = 0; b < 2; ++b)
                        if (b < n)
                            now[b].store(block + b * S::kABytes, scales + b * M_PAD, row0, scale[b]);
                    ptx::fence_proxy_async_shared();
                    __syncwarp();
                    if (lane == 0) {
                        ptx::mbar_arrive(bar_full + 8 * r.at);
                        ptx::mbar_arrive(bar_scales + 8 * q.at);
                    }
                }
            } else {
                const uint64_t policy = ptx::policy_evict_last();
                // This lane's tokens' scales (a token past the last counts 0).
                constexpr int kEach = (M_PAD + 31) / 32;
                const float *a_scale[kEach];
                float next[kEach], w = 0.f;  // the next block's
                auto fetch = [&]() {
#pragma unroll
                    for (int k = 0; k < kEach; ++k)
                        next[k] = lane + 32 * k < p.M ? *a_scale[k]++ : 0.f;
                    w = *w_scale++;
                };
#pragma unroll
                for (int k = 0; k < kEach; ++k)
                    a_scale[k] = p.a_scale + (int64_t)min(lane + 32 * k, p.M - 1) * p.blocks + begin * p.per_stage;
                if (left > 0)
                    fetch();
                for (int i = begin; i < end; ++i, r.step(p.stages), q.step(scale_slots)) {
                    wait(bar_empty + 8 * r.at, r.phase ^ 1, kErrGemm8Ring);
                    if (!ok)
                        break;
                    if (lane == 0)
                        load(&map_a, ring + r.at * stage_bytes + a_at, S::kABytes, 0, i, bar_full + 8 * r.at, policy);
                    __syncwarp();
                    float *scales = reinterpret_cast<float *>(smem + scales_at + q.at * scale_stage);
                    for (int b = 0; b < p.per_stage && left > 0; ++b, scales += M_PAD) {
#pragma unroll
                        for (int k = 0; k < kEach; ++k)
                            if (lane + 32 * k < M_PAD)
                                scales[lane + 32 * k] = next[k] * w;
                        if (--left > 0)
                            fetch();
                    }
                    __syncwarp();
                    if (lane == 0)
                        ptx::mbar_arrive(bar_scales + 8 * q.at);
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMAs
        constexpr uint32_t kIdesc = make_idesc_e4m3(kTileN, M_PAD);
        const uint32_t base = uniform(tmem);
        RingPlace r, d;                      // of the ring, of the buffers
        for (int tile = first_tile; tile < tiles && ok; tile += tile_step)
        for (int i = begin; i < end && ok; ++i, r.step(p.stages), d.step(buffers)) {
            wait(bar_full + 8 * r.at, r.phase, kErrGemm8Full);
            const int n = min(p.per_stage, p.blocks - i * p.per_stage);
            wait(bar_free + 8 * d.at, d.phase ^ 1, kErrGemm8Free);
            if (!ok)
                break;
            ptx::tcgen05_fence_after_thread_sync();
            uint64_t w = make_sw128_kmajor_desc(ring + r.at * stage_bytes);
            uint64_t a = make_sw128_kmajor_desc(ring + r.at * stage_bytes + a_at);
            uint32_t to = base + d.at * p.per_stage * M_PAD;
            if (ptx::elect_one_sync()) {
                for (int b = 0; b < n; ++b, w += S::kWBytes / 16, a += S::kABytes / 16, to += M_PAD) {
#pragma unroll
                    for (uint32_t k = 0; k < 4; ++k)
                        mma_e4m3_ss(to, w + 2 * k, a + 2 * k, kIdesc, k > 0);
                }
                ptx::tcgen05_commit(bar_sums + 8 * d.at);
                ptx::tcgen05_commit(bar_empty + 8 * r.at);
            }
            __syncwarp();
        }
        if (ptx::elect_one_sync())
            ptx::tcgen05_commit(bar_drain);
        __syncwarp();
        (void)wait_short(bar_drain, 0);      // nothing writes TMEM any more
    } else {
        // ------------------------------------------------------------ sums: thread = row of W = TMEM lane
        const int column0 = (warp - 2) / 4 * S::kColumns;
        const uint32_t from = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + column0;
        // kAtOnce tokens at a time, the next ones on their way while these are multiplied (the last ones of a stage: the next
        // stage's first).
        constexpr int kAtOnce = M_PAD < 64 ? 16 : 32, kPieces = S::kColumns / kAtOnce;
        RingPlace q, d;                      // of the scales, of the buffers
        uint32_t v[2][kAtOnce];
        auto multiply = [&](const uint32_t (&x)[kAtOnce], const float *scales, int c0) {
#pragma unroll
            for (int c = 0; c < kAtOnce; c += 4) {
                const float4 a = *reinterpret_cast<const float4 *>(scales + column0 + c0 + c);
                uint64_t *to = acc + (c0 + c) / 2;
                to[0] = fma2(pack2(x[c], x[c + 1]), pack2(a.x, a.y), to[0]);
                to[1] = fma2(pack2(x[c + 2], x[c + 3]), pack2(a.z, a.w), to[1]);
            }
        };
        for (int tile = first_tile; tile < tiles && ok; tile += tile_step) {
            const float *last = nullptr;     // scales of the tokens in v[1], the last ones of their block
            for (int i = begin; i < end && ok; ++i, q.step(scale_slots), d.step(buffers)) {
                // Both at once: each takes 200 cycles, passed or not.
                const bool sums = mbar_try_wait_for(bar_sums + 8 * d.at, d.phase, 1000000u);
                const bool known = mbar_try_wait_for(bar_scales + 8 * q.at, q.phase, 1000000u);
                if (!__all_sync(0xffffffffu, sums && known)) {
                    wait(bar_sums + 8 * d.at, d.phase, kErrGemm8Sums);
                    if (ok)
                        wait(bar_scales + 8 * q.at, q.phase, kErrGemm8Full);
                    if (!ok)
                        break;
                }
                ptx::tcgen05_fence_after_thread_sync();
                const int n = min(p.per_stage, p.blocks - i * p.per_stage);
                const float *scales = reinterpret_cast<const float *>(smem + scales_at + q.at * scale_stage);
                const uint32_t at = from + d.at * p.per_stage * M_PAD;
#pragma unroll
                for (int k = 0; k < 2 * kPieces; ++k) {              // (two blocks a stage at most)
                    constexpr int kLast = (kPieces - 1) * kAtOnce;
                    const int b = k / kPieces, c0 = k % kPieces * kAtOnce;
                    if (b >= n)
                        break;
                    tmem_ld<kAtOnce>(at + b * M_PAD + c0, v[k & 1]);
                    if (k > 0)
                        multiply(v[~k & 1], scales + (k - 1) / kPieces * M_PAD, (k - 1) % kPieces * kAtOnce);
                    else if (last)
                        multiply(v[1], last, kLast);
                    ptx::tmem_wait_ld();
                }
                ptx::tcgen05_fence_before_thread_sync();
                __syncwarp();
                if (lane == 0)
                    ptx::mbar_arrive(bar_free + 8 * d.at);
                if ((n * kPieces) & 1) {     // they are in v[0], where the next ones come
                    multiply(v[0], scales + (n - 1) * M_PAD, (kPieces - 1) * kAtOnce);
                    last = nullptr;
                } else {
                    last = scales + (n - 1) * M_PAD;
                }
            }
            if (last && ok)
                multiply(v[1], last, (kPieces - 1) * kAtOnce);
            const int n0 = tile * kTileN, row = 32 * (warp & 3) + lane;
            if (ranks > 1 || !ok)
                break;
#pragma unroll
            for (int c = 0; c < S::kColumns; ++c) {
                if (column0 + c < p.M && n0 + row < p.N) {
                    const float2 x = unpack2(acc[c / 2]);
                    p.c[(int64_t)(column0 + c) * p.N + n0 + row] = __float2bfloat16_rn(c & 1 ? x.y : x.x);
                }
            }
#pragma unroll
            for (int c = 0; c < S::kColumns / 2; ++c)
                acc[c] = 0;
        }
    }
    __syncwarp();
    ptx::tcgen05_fence_before_thread_sync();
    if (!__syncthreads_and(ok)) {
        // A wait gave up (reported): no copy may land after the CTA has ended, nor in the mailbox.  Whatever is still
        // under way has landed long before this gives up, too.
        (void)wait_short(bar_drain, 1);
    }
    // Every sum has been read, every copy has landed.
    if (warp == 1) {
        ptx::tcgen05_fence_after_thread_sync();
        ptx::tmem_dealloc(tmem, S::kTmem);
    }
    const int column0 = (warp - 2) / 4 * S::kColumns;
    const int row = 32 * (warp & 3) + lane;
    const bool sums = warp >= 2 && warp < S::kLoadWarp;
    if (ranks == 1)
        return;
    const int n0 = first_tile * kTileN;
    // Rank q's mailbox: [source rank][128 rows][its tokens], four tokens at a place that depends on the row, so that
    // neighbouring rows' are on different banks.  Each rank's barrier counts the bytes that it waits for.
    if (!p.apart)
        ptx::cluster_arrive_release();
    ptx::cluster_wait_acquire();
    const int groups = tokens / 4;
    auto place = [&](int source, int group) { return ((source * kTileN + row) * groups + (group ^ (row & (groups - 1)))) * 16; };
    if (sums) {
#pragma unroll
        for (int c = 0; c < S::kColumns; c += 4) {
            const int m = column0 + c, to = m / tokens, group = (m - to * tokens) / 4;
            if (m >= p.M)
                continue;
            const float2 x = unpack2(acc[c / 2]), y = unpack2(acc[c / 2 + 1]);
            ptx::st_async_v4(ptx::mapa_shared(sbase + p.mailbox + place(rank, group), to), ptx::mapa_shared(bar_mail, to), x.x, x.y, y.x,
                             y.y);
        }
        if (mine == 0)
            return;
        const uint64_t t0 = ptx::globaltimer();
        while (!ptx::mbar_try_wait_relaxed_cluster(bar_mail, 0))
            if (ptx::globaltimer() - t0 > kDefaultTimeoutNs) {
                atomicOr(p.status, kErrGemm8Mail);
                return;
            }
        ptx::fence_acquire_shared_cluster();
        if (n0 + row < p.N)
            for (int group = (warp - 2) / 4; 4 * group < mine; group += S::kEpilogueWarps / 4) {
                float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int r = 0; r < ranks; ++r) {
                    const float4 x = *reinterpret_cast<const float4 *>(smem + p.mailbox + place(r, group));
                    sum.x += x.x, sum.y += x.y, sum.z += x.z, sum.w += x.w;
                }
                __nv_bfloat16 *c = p.c + (int64_t)(rank * tokens + 4 * group) * p.N + n0 + row;
                c[0] = __float2bfloat16_rn(sum.x);
                if (4 * group + 1 < mine)
                    c[p.N] = __float2bfloat16_rn(sum.y);
                if (4 * group + 2 < mine)
                    c[2 * (int64_t)p.N] = __float2bfloat16_rn(sum.z);
                if (4 * group + 3 < mine)
                    c[3 * (int64_t)p.N] = __float2bfloat16_rn(sum.w);
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

// CTAs that find an SM each in clusters of `split`: a cluster lies in one GPC (of 152 SMs 144 in fours and 120 in eights, by
// cudaOccupancyMaxActiveClusters).
int room_of(int split, int sms) { return split >= 8 ? sms * 15 / 19 : (split >= 4 ? sms * 18 / 19 : sms); }

// Ranks along K as long as the CTAs find an SM, or, with up to 16 tokens, half of one (us at N 6144, K 4096, split 1, 2, 4: 4
// tokens 10.1, 7.4, 6.6; 32 tokens 11.9, 9.3, 9.7; 64 tokens 13.4, 11.4, 18.7; 128 tokens 18.5, 15.6, 26.5), and with 32 half
// of one where clusters leave SMs out.  The exchange grows with the tokens (N 1024, K 4096, split 4, 8: 64 tokens 10.6, 9.9; 128
// tokens 13.7, 14.5), and clusters that have to wait cost most (N 2304, K 4096, split 4, 8: 32 tokens, two CTAs an SM, 9.1, 8.3;
// 64 tokens 10.8, 17.8; 128 tokens 14.0, 25.7).
int split_of(int m_pad, int tiles, int blocks, int sms)
{
    const int most = m_pad <= 64 ? std::min(m_pad / 4, kMaxSplit) : 4;
    auto room = [&](int split) { return m_pad <= 16 ? 2 * room_of(split, sms) : (m_pad <= 32 ? sms : room_of(split, sms)); };
    int split = 1;
    while (split < most && tiles * split * 2 <= room(split * 2) && blocks >= 4 * split)
        split *= 2;
    return split;
}

template <int M_PAD, bool QUANT>
lowm_status_t launch_gemm_fp8(const void *A, const void *W, Gemm8Params &p, int sms, void *stream)
{
    using S = Gemm8Shape<M_PAD, QUANT>;
    const int tiles = (p.N + kTileN - 1) / kTileN;
    const int split = split_of(M_PAD, tiles, p.blocks, sms);
    // Two CTAs an SM hide each other's ends (4 tokens, N 49152: 37.7 -> 36.2 us); more tokens take an SM's registers.
    const bool two = M_PAD <= 32 && tiles * split > room_of(split, sms);
    // A copy costs much the same whatever its size (K blocks a copy 1, 2: 4 tokens, N 49152 48.1, 37.7 us).
    p.per_stage = 2;
    const int mailbox = split > 1 ? M_PAD * kTileN * 4 : 0;
    p.apart = M_PAD <= 32;                                               // else the mailbox is the drained ring
    const int budget = (two ? kSmem / 2 - 1024 : kSmem) - (int)kRingAt - (p.apart ? mailbox : 0) - 64 - (kBuffers + 4) * (int)S::kScaleBytes;
    // (the scales' extra slots: those of kBuffers + 1 blocks at most)
    const int extra = (kBuffers + p.per_stage) * (int)S::kScaleBytes;
    auto bytes_of = [](int blocks) { return blocks * (int)(S::kWBytes + S::kABytes + S::kScaleBytes); };
    while (p.per_stage > 1 && (2 * bytes_of(p.per_stage) > budget || p.blocks < p.per_stage * split))
        p.per_stage /= 2;
    const int stage = bytes_of(p.per_stage), share = ((p.blocks + p.per_stage - 1) / p.per_stage + split - 1) / split;
    p.stages = std::min({budget / stage, share, (int)kMaxStages});
    if (p.stages < 1)
        return LOWM_ERR_UNSUPPORTED_SHAPE;
    p.planes = p.K % kBlock == 0;
    const int used = (int)kRingAt + p.stages * stage + extra;            // (a multiple of 16)
    p.mailbox = p.apart ? used : (int)kRingAt;
    const int bytes = std::max(used, p.mailbox + mailbox);
    CUtensorMap map_w, map_a;
    lowm_status_t st = encode_matrix(W, p.N, p.K, kTileN, p.per_stage, p.planes, &map_w);
    if (st != LOWM_OK)
        return st;
    map_a = map_w;                                                       // (not read)
    if (!QUANT && (st = encode_matrix(A, p.M, p.K, M_PAD, p.per_stage, p.planes, &map_a)) != LOWM_OK)
        return st;
    static SmemOptIn opt_in;
    if (!opt_in.set(reinterpret_cast<const void *>(gemm_fp8_kernel<M_PAD, QUANT>), kSmem))
        return LOWM_ERR_CUDA;
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    // CTAs on their own keep their SM, so that the next tile's loads do not wait for this one's end.
    cfg.gridDim = dim3((unsigned)(split > 1 ? tiles * split : std::min(tiles, (two ? 2 : 1) * sms)));
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
    return cudaLaunchKernelEx(&cfg, gemm_fp8_kernel<M_PAD, QUANT>, map_w, map_a, p) == cudaSuccess ? LOWM_OK : LOWM_ERR_CUDA;
}

// The checks that both forms share, and what they fill in.
lowm_status_t prepare_gemm(const void *A, const void *W, const float *w_scale, void *C, int M, int N, int K, unsigned flags,
                           Gemm8Params &p, int &sms)
{
    if (M <= 0 || N <= 0 || K <= 0 || (flags & ~(unsigned)LOWM_FLAG_W_BEFORE_PDL_WAIT))
        return LOWM_ERR_INVALID_ARGUMENT;
    if (M > 128 || K % 16 || N > (1 << 30))
        return LOWM_ERR_UNSUPPORTED_SHAPE;
    if (!A || !W || !w_scale || !C)
        return LOWM_ERR_INVALID_ARGUMENT;
    if (!is_aligned(W, 16) || !is_aligned(C, 2) || !is_aligned(w_scale, 4))
        return LOWM_ERR_MISALIGNED;
    std::memset(&p, 0, sizeof p);
    p.w_scale = w_scale;
    p.c = static_cast<__nv_bfloat16 *>(C);
    p.M = M;
    p.N = N;
    p.K = K;
    p.blocks = (K + kBlock - 1) / kBlock;
    p.flags = flags;
    return LOWM_OK;
}

lowm_status_t launch_codes(const void *A, const void *W, Gemm8Params &p, int sms, void *stream)
{
    return p.M <= 16   ? launch_gemm_fp8<16, false>(A, W, p, sms, stream)
           : p.M <= 32 ? launch_gemm_fp8<32, false>(A, W, p, sms, stream)
           : p.M <= 64 ? launch_gemm_fp8<64, false>(A, W, p, sms, stream)
                       : launch_gemm_fp8<128, false>(A, W, p, sms, stream);
}

// Up to 16 tokens are quantised by the GEMM itself, every CTA its share of K for each of its tiles: 0.2 us a K block that
// way, against a launch of its own (us inside, apart: N 6144, K 4096, 8 blocks a CTA 8.3, 10.1; N 2304, K 12288, 24 blocks
// 14.4, 11.6; N 49152, K 4096, 64 and 32 blocks 40.0, 35.4).  More tokens are too much for it.
constexpr int kQuantTokens = 16, kQuantBlocks = 12;

bool quantises_inside(const Gemm8Params &p, int sms)
{
    const int tiles = (p.N + kTileN - 1) / kTileN, split = split_of(16, tiles, p.blocks, sms);
    const int64_t turns = ((int64_t)tiles * split + 2 * sms - 1) / (2 * sms);
    return p.M <= kQuantTokens && turns * ((p.blocks + split - 1) / split) <= kQuantBlocks;
}

size_t code_bytes(int M, int K) { return ((size_t)M * K + 15) / 16 * 16; }

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
    Gemm8Params p;
    int sms = 0;
    lowm_status_t st = prepare_gemm(A, W, w_scale, C, M, N, K, flags, p, sms);
    if (st != LOWM_OK)
        return st;
    if (!a_scale)
        return LOWM_ERR_INVALID_ARGUMENT;
    if (!is_aligned(A, 16) || !is_aligned(a_scale, 4))
        return LOWM_ERR_MISALIGNED;
    if ((st = host_check_device(&sms)) != LOWM_OK)
        return st;
    p.a_scale = a_scale;
    p.status = host_status_word();
    return p.status ? launch_codes(A, W, p, sms, stream) : LOWM_ERR_CUDA;
}

extern "C" size_t lowm_gemm_fp8_bf16_workspace(int M, int K)
{
    using namespace lowm;
    if (M <= 0 || M > 128 || K <= 0 || K % 16)
        return 0;
    return code_bytes(M, K) + (size_t)M * ((K + kBlock - 1) / kBlock) * sizeof(float);
}

extern "C" lowm_status_t lowm_gemm_fp8_bf16(const void *x, int64_t x_stride, const void *W, const float *w_scale, void *C, int M,
                                            int N, int K, unsigned flags, void *workspace, size_t workspace_bytes, void *stream)
{
    using namespace lowm;
    Gemm8Params p;
    int sms = 0;
    lowm_status_t st = prepare_gemm(x, W, w_scale, C, M, N, K, flags, p, sms);
    if (st != LOWM_OK)
        return st;
    if (x_stride < 0 || !workspace || workspace_bytes < lowm_gemm_fp8_bf16_workspace(M, K))
        return LOWM_ERR_INVALID_ARGUMENT;
    if (!is_aligned(x, 2) || !is_aligned(workspace, 16))
        return LOWM_ERR_MISALIGNED;
    if ((st = host_check_device(&sms)) != LOWM_OK)
        return st;
    p.status = host_status_word();
    if (!p.status)
        return LOWM_ERR_CUDA;
    if (quantises_inside(p, sms)) {
        p.x = static_cast<const __nv_bfloat16 *>(x);
        p.x_stride = x_stride;
        p.x_vec = is_aligned(x, 8) && x_stride % 4 == 0;
        return launch_gemm_fp8<16, true>(nullptr, W, p, sms, stream);
    }
    float *scales = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + code_bytes(M, K));
    st = lowm_quantize_fp8(x, x_stride, workspace, scales, M, K, 1, stream);
    if (st != LOWM_OK)
        return st;
    // The quantisation does not write W, and it begins only after what came before it has ended.
    p.a_scale = scales;
    p.flags |= LOWM_FLAG_W_BEFORE_PDL_WAIT;
    return launch_codes(workspace, W, p, sms, stream);
}
