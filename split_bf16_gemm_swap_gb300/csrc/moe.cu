// A mixture-of-experts layer for at most 128 tokens (lowm_layer.h), in two
// kernels.
//
// router_kernel.  A cluster of 8 CTAs owns 8 tokens, the N of an
// mma.m16n8k16: each CTA takes every 8th tile of 16 experts (or a part of the K
// steps of one), its 8 warps the 32-wide K steps in turns with eight steps'
// loads in flight (the kernel is a few memory latencies long), the logits go to the shared memory of the CTA that
// scores the token, and after the cluster barrier it picks the top k.
//
// experts_kernel.  The layer reads every reached expert's 3 * inner * hidden
// weights once, at most 128 times as many operations: HBM bandwidth bounds it.
// It is one persistent CTA per SM, as the GEMM swapped: 64 weight rows are the
// MMA's M and an expert's tokens (up to 64 at a time) its N.  A TMA warp keeps
// a ring of weight tiles full across all of the CTA's work items, a loader warp
// gathers the tokens' rows beside them (cp.async), two MMA warps issue the even
// and the odd K16 steps (one for all: 174 us for 172 with 128 tokens), and
// four warps empty one pair of accumulators while the other fills.
//   up:    an item is 32 inner elements of one expert, the 32 gate rows and 32
//          up rows interleaved by 8, so that gate and up of an element sit 8
//          lanes apart in TMEM and meet by a shuffle; silu(gate) * up goes to
//          the workspace in bf16 (the next MMA's operand type), by expert.
//   down:  an item is 64 hidden elements of one expert; fp32 products per
//          (token, choice) go to the workspace.
//   sum:   the choices of a token, weighted, in order.
// Up and down items form one list that the CTAs take in turns, so that a CTA
// short of an up item has a down item more.  A down item needs its expert's
// activations only: a counter per expert says when its up items are done, and
// the loader waits for it (a cooperative launch: the CTAs run together); the
// weight stream runs on.  One grid barrier separates the sum.  (A barrier
// between up and down left HBM idle for 15 us of 203 with 128 tokens; requests
// of the next weights into L2 ahead of the ring cost more than they hid, 144 to
// 154 us with 24 tokens.)
#include <cuda_bf16.h>
#include <math_constants.h>

#include <algorithm>

#include "layer_host.h"
#include "layer_device.cuh"

namespace lowm {
namespace {

constexpr int kMaxTokens = 128, kMaxExperts = 1024, kMaxTopK = 16, kMaxWidth = 32768;
constexpr int kRouterCluster = 8;            // CTAs (and tokens) of a router cluster
constexpr int kMoeThreads = 256;             // TMA warp 0, MMA warps 1 and 6, epilogue warps 2-5, loader warp 7
constexpr int kMoeRows = 64;                 // weight rows of an item = the MMA's M
constexpr int kMaxColumns = 64;              // tokens of an item; an expert with more gets several items
constexpr int kLoaderLag = 1;                // stages whose rows the loader has in flight behind the newest; below
                                             // the ring's stages, or it waits for one that it has not handed on
constexpr uint32_t kWBlockBytes = kMoeRows * 128u;

// Bits of the device status word (above those of paged_attention.cu).
enum : uint32_t {
    kErrMoeRing = 1u << 18,
    kErrMoeFull = 1u << 19,
    kErrMoeAccumulator = 1u << 20,
    kErrMoeGrid = 1u << 21,
};

struct MoeParams {
    const __nv_bfloat16 *x, *router;
    const float *bias;
    __nv_bfloat16 *out;
    int64_t x_stride, out_stride;
    int tokens, hidden, inner, experts, top_k, scoring, renormalize;
    float scale;
    bool out_vec;        // 8-byte stores of out
    // workspace
    __nv_bfloat16 *act;  // [tokens * top_k, inner], by expert
    float *product;      // [tokens * top_k, hidden]
    float *weights;      // [tokens * top_k]
    int *ids;            // [tokens * top_k]
    unsigned *arrived;   // the grid barrier, then [groups] epilogue warps done with an up item; zeroed by the router
    int counters;        // words of it
    // experts_kernel
    int columns, stages; // most tokens of an item (a multiple of 8), ring depth
    unsigned int *status;
};

// Order-preserving image of a float (NaN above +inf): the choice stays total
// and distinct whatever the scores hold.
__device__ __forceinline__ unsigned ordered_bits(float f)
{
    const unsigned u = f != f ? 0x7fffffffu : __float_as_uint(f + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// D[16 experts][8 tokens] += A[16][16] . B[16][8], bf16 operands, fp32 sums.
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A float into the shared memory of another CTA of the cluster (address from mapa_shared).
__device__ __forceinline__ void st_cluster(uint32_t addr, float v)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// One warp scores a token from its logits (the sum of `parts` rows) and picks
// its top k; a lane holds experts lane, lane + 32, ... (128 experts: 4 a lane).
template <int PER>
__device__ __forceinline__ void score_token(const MoeParams &p, int t, const float *logits, int parts)
{
    const int lane = threadIdx.x & 31;
    float prob[PER];
    unsigned key[PER];
    float m = -CUDART_INF_F, l = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 32 * i;
        prob[i] = e < p.experts ? logits[e] : -CUDART_INF_F;
        for (int j = 1; j < parts && e < p.experts; ++j)
            prob[i] += logits[j * p.experts + e];
        m = fmaxf(m, prob[i]);
    }
    if (p.scoring == LOWM_MOE_SOFTMAX) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            prob[i] = lane + 32 * i < p.experts ? expf(prob[i] - m) : 0.f;
            l += prob[i];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            l += __shfl_xor_sync(0xffffffffu, l, o);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 32 * i;
        prob[i] = p.scoring == LOWM_MOE_SOFTMAX ? prob[i] / l : 1.f / (1.f + expf(-prob[i]));
        key[i] = e < p.experts ? ordered_bits(prob[i] + (p.bias ? p.bias[e] : 0.f)) : 0u;
    }
    float sum = 0.f, mine = 0.f;
    int chosen = 0;
    for (int s = 0; s < p.top_k; ++s) {
        unsigned best = 0, at = kMaxExperts;
        float w = 0.f;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (key[i] > best) {
                best = key[i];
                at = lane + 32 * i;
                w = prob[i];
            }
        const unsigned top = __reduce_max_sync(0xffffffffu, best);
        const unsigned e = __reduce_min_sync(0xffffffffu, best == top ? at : (unsigned)kMaxExperts);
        w = __shfl_sync(0xffffffffu, w, e & 31);
        sum += w;
        if (lane == s) {
            mine = w;
            chosen = (int)e;
        }
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (e == lane + 32 * i)
                key[i] = 0;
    }
    if (lane < p.top_k) {
        p.ids[t * p.top_k + lane] = chosen;
        p.weights[t * p.top_k + lane] = mine * p.scale / (p.renormalize ? sum : 1.f);
    }
}

constexpr int kRouterWarps = 8;

__global__ void __cluster_dims__(kRouterCluster, 1, 1) __launch_bounds__(32 * kRouterWarps, 2) router_kernel(const MoeParams p)
{
    __shared__ float prob[kMaxExperts];
    __shared__ float part[kRouterWarps][16][8];
    // Every CTA of the cluster runs before one writes into another's shared memory.
    ptx::cluster_arrive_release();
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    ptx::cluster_wait_acquire();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)ptx::cluster_ctarank(), t0 = blockIdx.x / kRouterCluster * kRouterCluster;
    const int nt = min(kRouterCluster, p.tokens - t0);
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < p.counters; i += 32 * kRouterWarps)
            p.arrived[i] = 0u;

    // A thread's 8 consecutive k of a 32-wide step serve both K16 products:
    // the same permutation of k on both operands leaves the sum alone.
    const int row = lane >> 2, k0 = warp * 32 + (lane & 3) * 8;
    const __nv_bfloat16 *x = p.x + (t0 + min(row, nt - 1)) * p.x_stride;
    // Fewer than 8 tiles of experts: the spare CTAs take a part of the K steps each.
    const int tiles = (p.experts + 15) / 16, parts = max(1, kRouterCluster / tiles);
    const int share = rank / tiles, first = parts > 1 ? rank % tiles : rank;
    for (int tile = parts > 1 && share >= parts ? tiles : first; tile < tiles; tile += kRouterCluster) {
        const int e0 = tile * 16 + row, e1 = e0 + 8;
        const __nv_bfloat16 *w0 = p.router + (int64_t)min(e0, p.experts - 1) * p.hidden;
        const __nv_bfloat16 *w1 = p.router + (int64_t)min(e1, p.experts - 1) * p.hidden;
        float d[4] = {};
        constexpr int kSteps = 8;
        const int stride = 32 * kRouterWarps * parts;
        for (int base = parts > 1 ? share * 32 * kRouterWarps : 0; base < p.hidden; base += kSteps * stride) {
            uint4 a[kSteps], b[kSteps], c[kSteps];
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                const int k = base + k0 + i * stride;
                a[i] = b[i] = c[i] = make_uint4(0, 0, 0, 0);
                if (k < p.hidden) {
                    a[i] = *reinterpret_cast<const uint4 *>(w0 + k);
                    b[i] = *reinterpret_cast<const uint4 *>(w1 + k);
                    c[i] = *reinterpret_cast<const uint4 *>(x + k);
                }
            }
            asm volatile("" ::: "memory");   // all loads before the first product
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                mma_16x8x16(d, a[i].x, b[i].x, a[i].y, b[i].y, c[i].x, c[i].y);
                mma_16x8x16(d, a[i].z, b[i].z, a[i].w, b[i].w, c[i].z, c[i].w);
            }
        }
        const int col = (lane & 3) * 2;
        part[warp][row][col] = d[0];
        part[warp][row][col + 1] = d[1];
        part[warp][row + 8][col] = d[2];
        part[warp][row + 8][col + 1] = d[3];
        __syncthreads();
        if (threadIdx.x < 128) {
            const int r = threadIdx.x & 15, t = threadIdx.x >> 4;
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kRouterWarps; ++w)
                s += part[w][r][t];
            if (t < nt && tile * 16 + r < p.experts)   // to the CTA that scores the token
                st_cluster(ptx::mapa_shared(ptx::smem_u32(&prob[(parts > 1 ? share : 0) * p.experts + tile * 16 + r]), (uint32_t)t), s);
        }
        __syncthreads();
    }
    ptx::cluster_arrive_release();
    ptx::cluster_wait_acquire();
    if (warp || rank >= nt)
        return;
    if (p.experts <= 128)
        score_token<4>(p, t0 + rank, prob, parts);
    else
        score_token<kMaxExperts / 32>(p, t0 + rank, prob, 1);
}

// ------------------------------------------------------------------ experts_kernel
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const void *tmap, int x, int y, int z, int v, int w,
                                            uint32_t bar, uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(v), "r"(w), "r"(bar), "l"(policy)
        : "memory");
}

// 16 bytes to shared memory past L1; zeros when `bytes` is 0.
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void *src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void cp_async_commit()
{
    asm volatile("cp.async.commit_group;" ::: "memory");
}

template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Shared memory: the ring first (1024-byte tiles), then lists and barriers.
struct MoeSmem {
    uint32_t w, b, stage_b, mask, first, sorted, group, source, bars, slot, bytes;
};

__host__ __device__ inline int moe_max_groups(int experts, int pairs, int columns)
{
    return (pairs < experts ? pairs : experts) + pairs / columns;
}

// `blocks` 64-wide K blocks a stage.
__host__ __device__ inline MoeSmem moe_smem(int experts, int pairs, int columns, int blocks, int stages)
{
    MoeSmem L;
    L.w = 0;                                                   // [stages][blocks][64 rows][64]
    L.stage_b = blocks * columns * 128u;
    L.b = stages * blocks * kWBlockBytes;                  // [stages][blocks][columns][64]
    L.bars = L.b + stages * L.stage_b;                         // full, empty [stages]; accumulator full, free [2]; drain
    L.slot = L.bars + (2 * stages + 5) * 8;
    L.slot = (L.slot + 15) / 16 * 16;
    L.source = L.slot + 16;                                    // the loader's rows: a pointer each
    L.mask = L.source + kMaxColumns * 8;                                  // u32 [experts][4]: the expert's tokens
    L.group = L.mask + experts * 16;                           // (expert, first place, tokens) as 3 x u16, 8 bytes
    L.first = L.group + moe_max_groups(experts, pairs, columns) * 8;    // u16 [experts]: the expert's first place
    L.sorted = L.first + experts * 2;                          // u16 [pairs]: pair at each place
    L.bytes = L.sorted + pairs * 2 + 1024;                     // slack to align the base
    return L;
}

__device__ __forceinline__ unsigned ld_acquire(const unsigned *p)
{
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ void add_release(unsigned *p)
{
    asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(p) : "memory");
}

__device__ __forceinline__ bool wait_grid(const unsigned *p, unsigned want)
{
    const uint64_t t0 = ptx::globaltimer();
    for (;;) {
        for (int i = 0; i < 256; ++i)
            if (ld_acquire(p) >= want)
                return true;
        if (ptx::globaltimer() - t0 > kDefaultTimeoutNs)
            return false;
    }
}

template <int BLOCKS>
__global__ void __launch_bounds__(kMoeThreads, 1)
    experts_kernel(const __grid_constant__ CUtensorMap map_up, const __grid_constant__ CUtensorMap map_down,
                   const __grid_constant__ CUtensorMap map_up_tail, const __grid_constant__ CUtensorMap map_down_tail,
                   const MoeParams p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = ptx::smem_u32(smem);
    const int pairs = p.tokens * p.top_k, stages = p.stages;
    const MoeSmem L = moe_smem(p.experts, pairs, p.columns, BLOCKS, stages);
    const uint32_t bar_full = sbase + L.bars, bar_empty = bar_full + 8 * stages, bar_acc = bar_empty + 8 * stages,
                   bar_free = bar_acc + 16, bar_drain = bar_free + 16;
    uint32_t *mask = reinterpret_cast<uint32_t *>(smem + L.mask);
    ushort4 *group = reinterpret_cast<ushort4 *>(smem + L.group);
    uint16_t *first = reinterpret_cast<uint16_t *>(smem + L.first), *sorted = reinterpret_cast<uint16_t *>(smem + L.sorted);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr uint32_t kColumnsTmem = 4 * kMaxColumns;        // two accumulators (one an issuer), twice

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            ptx::mbar_init(bar_full + 8 * s, 2);      // weights, token rows
            ptx::mbar_init(bar_empty + 8 * s, 2);     // both MMA issuers
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(bar_acc + 8 * i, 2);
            ptx::mbar_init(bar_free + 8 * i, 4);      // epilogue warps
        }
        ptx::mbar_init(bar_drain, 2);
        ptx::fence_mbarrier_init_cluster();
        ptx::fence_proxy_async_shared();
    }
    if (warp == 1) {
        ptx::tmem_alloc(sbase + L.slot, kColumnsTmem);
        ptx::tmem_relinquish_alloc_permit();
        ptx::tcgen05_fence_before_thread_sync();
    }
    for (int e = threadIdx.x; e < 4 * p.experts; e += kMoeThreads)
        mask[e] = 0;
    ptx::griddep_wait();
    __syncthreads();
    ptx::tcgen05_fence_after_thread_sync();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + L.slot);

    // The pairs (token, choice) by expert, tokens in order, the same in every
    // CTA: an expert's tokens as a bit mask, a token's place the bits below its own.
    for (int i = threadIdx.x; i < pairs; i += kMoeThreads) {
        const int t = i / p.top_k;
        atomicOr(&mask[4 * p.ids[i] + (t >> 5)], 1u << (t & 31));
    }
    __syncthreads();
    int *num_groups = reinterpret_cast<int *>(smem + L.slot + 8);
    if (warp == 0) {
        int place = 0, groups = 0;
        for (int e0 = 0; e0 < p.experts; e0 += 32) {
            const int e = e0 + lane;
            int n = 0;
            for (int j = 0; e < p.experts && j < 4; ++j)
                n += __popc(mask[4 * e + j]);
            const int g = (n + p.columns - 1) / p.columns;
            int sn = n, sg = g;
            for (int o = 1; o < 32; o <<= 1) {
                const int a = __shfl_up_sync(0xffffffffu, sn, o), b = __shfl_up_sync(0xffffffffu, sg, o);
                if (lane >= o) {
                    sn += a;
                    sg += b;
                }
            }
            const int at = place + sn - n;
            if (e < p.experts)
                first[e] = (uint16_t)at;
            for (int j = 0; j < g; ++j)
                group[groups + sg - g + j] = make_ushort4((unsigned short)e, (unsigned short)(at + j * p.columns),
                                                          (unsigned short)min(p.columns, n - j * p.columns), 0);
            place += __shfl_sync(0xffffffffu, sn, 31);
            groups += __shfl_sync(0xffffffffu, sg, 31);
        }
        if (lane == 0)
            *num_groups = groups;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < pairs; i += kMoeThreads) {
        const int t = i / p.top_k, e = p.ids[i];
        int place = first[e] + __popc(mask[4 * e + (t >> 5)] & ((1u << (t & 31)) - 1));
        for (int j = 0; j < (t >> 5); ++j)
            place += __popc(mask[4 * e + j]);
        sorted[place] = (uint16_t)i;
    }
    __syncthreads();

    const int up_tiles = (p.inner + 31) / 32, down_tiles = (p.hidden + 63) / 64;
    const int up_items = *num_groups * up_tiles, items = up_items + *num_groups * down_tiles;
    const int up_blocks = (p.hidden + 63) / 64, down_blocks = (p.inner + 63) / 64;
    const int up_stages = (up_blocks + BLOCKS - 1) / BLOCKS, down_stages = (down_blocks + BLOCKS - 1) / BLOCKS;

    if (warp == 0) {
        // ------------------------------------------------------------ TMA
        // By an elected thread of a converged warp, as the MMAs below (128 tokens over
        // 32 experts 172.2 -> 170.9 us, one over 64 20.5 -> 20.3).
        const uint64_t once = ptx::policy_evict_first();
        uint32_t i = 0;
        bool ok = true;
        auto weights = [&](bool up, int item, int k) {
            const int s = i % stages;
            if (!wait_short(bar_empty + 8 * s, ((i / stages) & 1) ^ 1)) {
                ok = false;
                atomicOr(p.status, kErrMoeRing);
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok)
                return;
            const int tiles = up ? up_tiles : down_tiles, blocks = up ? up_blocks : down_blocks;
            const int e = uniform((int)group[item / tiles].x), width = up ? p.hidden : p.inner;
            // One copy brings a stage's blocks (those past a K of whole blocks as zeros); the last stage
            // of a K that ends inside a block comes block by block, so that the rest reads as zeros.
            const bool whole = width % 64 == 0 || (k + 1) * BLOCKS * 64 <= width;
            const int used = whole ? 1 : blocks - k * BLOCKS;
            const int row = up ? e * (p.inner / 4) + item % tiles * 4 : e * p.hidden + item % tiles * kMoeRows;
            if (ptx::elect_one_sync()) {
                ptx::mbar_arrive_expect_tx(bar_full + 8 * s, (whole ? BLOCKS : used) * kWBlockBytes);
                for (int j = 0; j < used; ++j) {
                    const uint32_t dst = sbase + L.w + (s * BLOCKS + j) * kWBlockBytes;
                    const int kb = k * BLOCKS + j, x = whole ? 0 : 64 * kb, z = whole ? kb : 0;
                    if (up)      // (k, 8 rows, gate / up, groups of 8 rows, k block)
                        tma_load_5d(dst, whole ? &map_up : &map_up_tail, x, 0, 0, row, z, bar_full + 8 * s, once);
                    else         // (k, row, k block)
                        ptx::tma_load_3d(dst, whole ? &map_down : &map_down_tail, x, row, z, bar_full + 8 * s, once);
                }
            }
            __syncwarp();
            ++i;
        };
        for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
            const bool up = item < up_items;
            for (int k = 0; k < (up ? up_stages : down_stages) && ok; ++k)
                weights(up, up ? item : item - up_items, k);
        }
        if (!ok)        // no copy may land after the CTA has ended (normally the MMAs have consumed all)
            for (uint32_t j = i > (uint32_t)stages ? i - stages : 0; j < i; ++j)
                (void)wait_short(bar_full + 8 * (j % stages), (j / stages) & 1);
        __syncwarp();
    } else if (warp == 7) {
        // ------------------------------------------------------------ token rows
        // Eight lanes copy the 128 bytes a row has in a block, each its 16-byte
        // chunk to the chunk's swizzled place.  The rows' addresses are looked
        // up once an item (looked up and divided out at every stage they cost
        // more than the stream: 128 tokens over 32 experts took 367 us).  The
        // copies of a stage are seen complete kLoaderLag stages later and then
        // handed to the tensor core (async proxy).
        uint32_t i = 0, handed = 0;
        bool ok = true;
        const int sub = lane >> 3, chunk = lane & 7;
        const __nv_bfloat16 **source = reinterpret_cast<const __nv_bfloat16 **>(smem + L.source);
        auto sources = [&](bool up, const ushort4 g) {
            __syncwarp();
            for (int r = lane; r < g.z; r += 32)
                source[r] = up ? p.x + (sorted[g.y + r] / p.top_k) * p.x_stride : p.act + (int64_t)(g.y + r) * p.inner;
            __syncwarp();
        };
        auto hand = [&](uint32_t upto) {
            for (; handed < upto; ++handed) {
                if (handed + kLoaderLag < i)
                    cp_async_wait<kLoaderLag>();
                else
                    cp_async_wait<0>();
                ptx::fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0)
                    ptx::mbar_arrive(bar_full + 8 * (handed % stages));
            }
        };
        auto rows = [&](bool up, const ushort4 g, int k) {
            const int s = i % stages;
            if (!wait_short(bar_empty + 8 * s, ((i / stages) & 1) ^ 1)) {
                ok = false;
                atomicOr(p.status, kErrMoeRing);
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok)
                return;
            const int width = up ? p.hidden : p.inner, at = k * (BLOCKS * 64) + chunk * 8;
            for (int r = sub; r < g.z; r += 4) {
                const __nv_bfloat16 *src = source[r];
                const uint32_t dst = sbase + L.b + s * L.stage_b + r * 128 + ((chunk ^ (r & 7)) << 4);
#pragma unroll
                for (int j = 0; j < BLOCKS; ++j) {
                    const bool in = at + 64 * j < width;
                    cp_async_16(dst + j * p.columns * 128, src + (in ? at + 64 * j : 0), in ? 16 : 0);
                }
            }
            __syncwarp();
            cp_async_commit();
            ++i;
            if (i > kLoaderLag)
                hand(i - kLoaderLag);
        };
        int ready = -1;                                          // the last group known to be complete
        for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
            const bool up = item < up_items;
            const int n = up ? item / up_tiles : (item - up_items) / down_tiles;
            const ushort4 g = group[n];
            if (!up && n != ready) {
                hand(i);                                         // no one waits for a stage while this warp does
                if (!wait_grid(&p.arrived[1 + n], 4 * up_tiles)) {
                    ok = false;
                    atomicOr(p.status, kErrMoeGrid);
                }
                ok = __all_sync(0xffffffffu, ok);
                ready = n;
            }
            sources(up, g);
            for (int k = 0; k < (up ? up_stages : down_stages) && ok; ++k)
                rows(up, g, k);
        }
        hand(i);
    } else if (warp == 1 || warp == 6) {
        // ------------------------------------------------------------ MMA: even or odd K16 steps
        // Converged warps that elect the issuing thread, with operands that the
        // compiler knows to be the same in all lanes: from a branch for lane 0
        // they issue more slowly (128 tokens over 32 experts 185 us, this way 172 to
        // 175; 24 over 128 138 -> 131; one over 64 22.3 -> 20.7).
        const uint32_t odd = uniform(warp) == 6;
        uint32_t i = 0, n = 0;
        bool ok = true;
        auto wait = [&](uint32_t bar, uint32_t parity, uint32_t err) {
            if (ok && !wait_short(bar, parity)) {
                ok = false;
                if (lane == 0)
                    atomicOr(p.status, err);
            }
            ok = __all_sync(0xffffffffu, ok);
            ptx::tcgen05_fence_after_thread_sync();
        };
        auto item_products = [&](const ushort4 g, int blocks, int num_stages) {
            const uint32_t d = uniform(tmem) + ((n & 1) * 2 + odd) * kMaxColumns;
            const uint32_t idesc = uniform(make_idesc_bf16(kMoeRows, (g.z + 7) / 8 * 8));
            wait(bar_free + 8 * (n & 1), ((n >> 1) & 1) ^ 1, kErrMoeAccumulator);
            for (int k = 0; k < num_stages && ok; ++k, ++i) {
                const int s = i % stages;
                wait(bar_full + 8 * s, (i / stages) & 1, kErrMoeFull);
                if (ok && ptx::elect_one_sync()) {
                    const int used = min(BLOCKS, blocks - k * BLOCKS);
                    for (int j = 0; j < used; ++j) {
                        const uint64_t a = make_sw128_kmajor_desc(sbase + L.w + (s * BLOCKS + j) * kWBlockBytes);
                        const uint64_t b = make_sw128_kmajor_desc(sbase + L.b + s * L.stage_b + j * p.columns * 128);
#pragma unroll
                        for (uint32_t q = 0; q < 2; ++q)
                            ptx::mma_bf16_ss(d, a + 2 * (2 * q + odd), b + 2 * (2 * q + odd), idesc, k + j + (int)q > 0);
                    }
                    ptx::tcgen05_commit(bar_empty + 8 * s);
                    if (k == num_stages - 1)
                        ptx::tcgen05_commit(bar_acc + 8 * (n & 1));
                }
                __syncwarp();
            }
            ++n;
        };
        for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
            const bool up = item < up_items;
            item_products(group[up ? item / up_tiles : (item - up_items) / down_tiles], up ? up_blocks : down_blocks,
                          up ? up_stages : down_stages);
        }
        if (ptx::elect_one_sync())        // the thread that issued the MMAs
            ptx::tcgen05_commit(bar_drain);
        __syncwarp();
        (void)wait_short(bar_drain, 0);   // nothing writes TMEM any more
    } else {
        // ------------------------------------------------------------ epilogue
        const int quarter = warp & 3;
        const uint32_t lanes = tmem + ((uint32_t)(32 * quarter) << 16);
        uint32_t n = 0;
        bool ok = true;
        auto wait_acc = [&]() {
            if (ok && !wait_short(bar_acc + 8 * (n & 1), (n >> 1) & 1)) {
                ok = false;
                atomicOr(p.status, kErrMoeAccumulator);
            }
            ok = __all_sync(0xffffffffu, ok);
            ptx::tcgen05_fence_after_thread_sync();
        };
        auto release = [&]() {
            ptx::tcgen05_fence_before_thread_sync();
            __syncwarp();
            if (lane == 0)
                ptx::mbar_arrive(bar_free + 8 * (n & 1));
            ++n;
        };
        for (int item = blockIdx.x; item < items; item += gridDim.x) {
            const bool up = item < up_items;
            const int at = up ? item : item - up_items, tiles = up ? up_tiles : down_tiles;
            const ushort4 g = group[at / tiles];
            wait_acc();
            if (!ok)
                break;
            // up: lane l of quarter q holds gate (l < 8) or up (8 <= l < 16) of element 32 tile + 8 q + l % 8.
            const int row = up ? at % tiles * 32 + quarter * 8 + lane : at % tiles * kMoeRows + quarter * 16 + lane;
            for (int c = 0; c < g.z; c += 8) {
                float v[8], u[8];
                load_accumulator_pair<8>(lanes + (n & 1) * 2 * kMaxColumns + c, lanes + ((n & 1) * 2 + 1) * kMaxColumns + c, v, u);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float y = v[j] + u[j], z = __shfl_down_sync(0xffffffffu, y, 8);
                    if (c + j >= g.z)
                        continue;
                    if (up) {
                        if (lane < 8 && row < p.inner)
                            p.act[(int64_t)(g.y + c + j) * p.inner + row] = __float2bfloat16_rn(y / (1.f + expf(-y)) * z);
                    } else if (lane < 16 && row < p.hidden) {
                        p.product[(int64_t)sorted[g.y + c + j] * p.hidden + row] = y;
                    }
                }
            }
            release();
            if (up) {                                            // after the release this warp's quarter of the item is in memory
                __syncwarp();
                if (lane == 0)
                    add_release(&p.arrived[1 + at / tiles]);
            }
        }
    }
    // Every product of this CTA is in memory; all threads add once every CTA's are.
    ptx::tcgen05_fence_before_thread_sync();
    __syncthreads();
    if (threadIdx.x == 0) {
        add_release(&p.arrived[0]);
        if (!wait_grid(&p.arrived[0], gridDim.x))
            atomicOr(p.status, kErrMoeGrid);
    }
    if (warp == 1) {
        ptx::tcgen05_fence_after_thread_sync();
        ptx::tmem_dealloc(tmem, kColumnsTmem);
    }
    __syncthreads();
    ptx::griddep_launch_dependents();
    const int quads = p.hidden / 4, total = p.tokens * quads;
    for (int c = blockIdx.x * kMoeThreads + threadIdx.x; c < total; c += gridDim.x * kMoeThreads) {
        const int t = c / quads, h = c % quads * 4;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int s = 0; s < p.top_k; ++s) {
            const float w = p.weights[t * p.top_k + s];
            const float4 d = __ldcg(reinterpret_cast<const float4 *>(p.product + (int64_t)(t * p.top_k + s) * p.hidden + h));
            y.x = fmaf(w, d.x, y.x);
            y.y = fmaf(w, d.y, y.y);
            y.z = fmaf(w, d.z, y.z);
            y.w = fmaf(w, d.w, y.w);
        }
        __nv_bfloat16 *o = p.out + t * p.out_stride + h;
        const __nv_bfloat162 a = __floats2bfloat162_rn(y.x, y.y), b = __floats2bfloat162_rn(y.z, y.w);
        if (p.out_vec) {
            uint2 u;
            u.x = *reinterpret_cast<const uint32_t *>(&a);
            u.y = *reinterpret_cast<const uint32_t *>(&b);
            *reinterpret_cast<uint2 *>(o) = u;
        } else {
            o[0] = a.x, o[1] = a.y, o[2] = b.x, o[3] = b.y;
        }
    }
}

bool moe_shape_ok(int tokens, int hidden, int inner, int experts, int top_k)
{
    return tokens >= 0 && tokens <= kMaxTokens && hidden > 0 && hidden <= kMaxWidth && hidden % 8 == 0 && inner > 0 &&
           inner <= kMaxWidth && inner % 8 == 0 && experts > 0 && experts <= kMaxExperts && top_k > 0 &&
           top_k <= std::min(kMaxTopK, experts);
}

// Tokens of an item.  The ring holds that many rows beside the 64 weight rows
// of every block, so room for 64 leaves half of the weights in flight that room
// for 16 does; an expert with more tokens reads its weights again (from L2:
// its items run side by side).  Twice the average and 8 more covers nearly all
// experts of a balanced router.
int moe_columns(int tokens, int experts, int top_k)
{
    const int usual = 2 * ((tokens * top_k + experts - 1) / experts) + 8;
    return std::min({kMaxColumns, (tokens + 7) / 8 * 8, (usual + 7) / 8 * 8});
}

constexpr int kMaxSmem = 232448;             // 227 KiB

// K blocks a stage.  A copy has a fixed cost, so eight blocks (64 KiB of
// weights) beat four where two such stages fit and K fills its last stage:
// GB300, 4 -> 8 blocks: 128 tokens over 32 experts of 4096 x 1400 191 -> 175 us,
// 8 tokens over 64 of 2048 x 768 47.6 -> 43.8; but 37 over 64 of 1544 x 920, whose
// 25 and 15 blocks would leave a fifth of the stages empty, 90.9 -> 95.8.
int moe_blocks(int hidden, int inner, int experts, int pairs, int columns)
{
    auto rounded = [](int n, int to) { return (n + to - 1) / to * to; };
    const int up = rounded(hidden, 64) / 64, down = rounded(inner, 64) / 64;
    const bool filled = 10 * (2 * rounded(up, 8) + rounded(down, 8)) <= 11 * (2 * up + down);
    return filled && (int)moe_smem(experts, pairs, columns, 8, 2).bytes <= kMaxSmem ? 8 : 4;
}

size_t round16(size_t n) { return (n + 15) / 16 * 16; }

struct MoeWorkspace {
    size_t act, product, weights, ids, arrived, bytes;
    int counters;
};

MoeWorkspace moe_workspace(int tokens, int hidden, int inner, int experts, int top_k)
{
    const size_t pairs = (size_t)std::max(tokens, 1) * top_k;
    MoeWorkspace w;
    w.act = 0;
    w.product = w.act + round16(pairs * inner * 2);
    w.weights = w.product + round16(pairs * hidden * 4);
    w.ids = w.weights + round16(pairs * 4);
    w.arrived = w.ids + round16(pairs * 4);
    w.counters = 1 + moe_max_groups(experts, (int)pairs, std::max(8, moe_columns(tokens, experts, top_k)));
    w.bytes = w.arrived + round16((size_t)w.counters * 4);
    return w;
}

lowm_status_t encode_bf16(CUtensorMap *map, const void *base, int rank, const cuuint64_t *dims, const cuuint64_t *strides,
                          const cuuint32_t *box)
{
    EncodeTiledFn enc = host_encode_fn();
    const cuuint32_t step[5] = {1, 1, 1, 1, 1};
    return enc && enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void *>(base), dims, strides, box,
                      step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? LOWM_OK
               : LOWM_ERR_CUDA;
}

}  // namespace
}  // namespace lowm

extern "C" size_t lowm_moe_workspace(int tokens, int hidden, int inner, int experts, int top_k)
{
    if (!lowm::moe_shape_ok(tokens, hidden, inner, experts, top_k))
        return 0;
    return lowm::moe_workspace(tokens, hidden, inner, experts, top_k).bytes;
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
        workspace_bytes < lowm_moe_workspace(tokens, hidden, inner, experts, top_k) || x_stride < hidden ||
        out_stride < hidden)
        return LOWM_ERR_INVALID_ARGUMENT;
    if (!is_aligned(x, 16) || !is_aligned(router, 16) || !is_aligned(gate_up, 16) || !is_aligned(down, 16) ||
        !is_aligned(workspace, 16) || !is_aligned(bias, 4) || !is_aligned(out, 2) || (x_stride & 7))
        return LOWM_ERR_MISALIGNED;
    int sms = 0;
    lowm_status_t st = host_check_device(&sms);
    if (st != LOWM_OK)
        return st;

    const int pairs = tokens * top_k;
    const MoeWorkspace w = moe_workspace(tokens, hidden, inner, experts, top_k);
    uint8_t *base = static_cast<uint8_t *>(workspace);
    MoeParams p;
    p.x = static_cast<const __nv_bfloat16 *>(x);
    p.router = static_cast<const __nv_bfloat16 *>(router);
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
    p.out_vec = is_aligned(out, 8) && (out_stride & 3) == 0;
    p.act = reinterpret_cast<__nv_bfloat16 *>(base + w.act);
    p.product = reinterpret_cast<float *>(base + w.product);
    p.weights = reinterpret_cast<float *>(base + w.weights);
    p.ids = reinterpret_cast<int *>(base + w.ids);
    p.arrived = reinterpret_cast<unsigned *>(base + w.arrived);
    p.counters = w.counters;
    p.columns = moe_columns(tokens, experts, top_k);
    const int blocks = moe_blocks(hidden, inner, experts, pairs, p.columns);
    for (p.stages = 8; p.stages > 2 && (int)moe_smem(experts, pairs, p.columns, blocks, p.stages).bytes > kMaxSmem; --p.stages) {
    }
    const int smem = (int)moe_smem(experts, pairs, p.columns, blocks, p.stages).bytes;
    if (smem > kMaxSmem)
        return LOWM_ERR_UNSUPPORTED_SHAPE;
    p.status = host_status_word();
    if (!p.status)
        return LOWM_ERR_CUDA;

    // gate_up as (k, 8 rows, gate / up, groups of 8 rows, k block): a box is 4 groups of 8 gate and 8 up rows.
    // An expert is inner / 4 groups further; the extent ends with the last expert's up rows, so every
    // element of a box lies inside the tensor or reads as zero.  The tail maps see K as one dimension.
    CUtensorMap maps[4];
    const cuuint64_t h2 = (cuuint64_t)hidden * 2, i2 = (cuuint64_t)inner * 2;
    const cuuint64_t groups = (cuuint64_t)experts * (inner / 4) - inner / 8, rows = (cuuint64_t)experts * hidden;
    for (int tail = 0; tail < 2; ++tail) {
        const cuuint64_t up_dims[5] = {tail ? (cuuint64_t)hidden : 64u, 8, 2, groups,
                                       tail ? 1u : (cuuint64_t)std::max(1, hidden / 64)};
        const cuuint64_t up_strides[4] = {h2, h2 * inner, h2 * 8, 128};
        const cuuint32_t deep = tail ? 1u : (cuuint32_t)blocks, up_box[5] = {64, 8, 2, 4, deep};
        const cuuint64_t down_dims[3] = {tail ? (cuuint64_t)inner : 64u, rows, tail ? 1u : (cuuint64_t)std::max(1, inner / 64)};
        const cuuint64_t down_strides[2] = {i2, 128};
        const cuuint32_t down_box[3] = {64, (cuuint32_t)kMoeRows, deep};
        // A K of whole blocks has no tail, a K below one block nothing else.
        const bool up_used = tail ? hidden % 64 != 0 : hidden >= 64, down_used = tail ? inner % 64 != 0 : inner >= 64;
        if (up_used && (st = encode_bf16(&maps[2 * tail], gate_up, 5, up_dims, up_strides, up_box)) != LOWM_OK)
            return st;
        if (down_used && (st = encode_bf16(&maps[2 * tail + 1], down, 3, down_dims, down_strides, down_box)) != LOWM_OK)
            return st;
        if (!up_used)
            std::memset(&maps[2 * tail], 0, sizeof maps[0]);
        if (!down_used)
            std::memset(&maps[2 * tail + 1], 0, sizeof maps[0]);
    }

    const int clusters = (tokens + kRouterCluster - 1) / kRouterCluster;
    if ((st = launch_pdl(router_kernel, dim3((unsigned)(clusters * kRouterCluster)), dim3(32 * kRouterWarps), 0, stream, p)) !=
        LOWM_OK)
        return st;
    static SmemOptIn opt_in[2];
    auto *kernel = blocks == 8 ? experts_kernel<8> : experts_kernel<4>;
    if (!opt_in[blocks == 8].set(reinterpret_cast<const void *>(kernel), kMaxSmem))
        return LOWM_ERR_CUDA;
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3((unsigned)sms);
    cfg.blockDim = dim3(kMoeThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeCooperative;  // its CTAs wait for one another
    attrs[0].val.cooperative = 1;
    attrs[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attrs;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, maps[0], maps[1], maps[2], maps[3], p) == cudaSuccess ? LOWM_OK
                                                                                                        : LOWM_ERR_CUDA;
}
