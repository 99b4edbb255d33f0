// Attention of each sequence's newest tokens over a paged cache of e4m3 codes
// with a scale for each block of tokens and head (lowm_fp8.h).
//
//     s_j = scale (q . k_j) a_j,  out = sum_j softmax_j(s) b_j v_j
//
// with codes k, v and the scales a_j, b_j of the blocks that key j lies in.
//
// Products.  Both run on the 8-bit tensor cores from registers (m16n8k32), the
// codes as they lie in the cache: nothing is widened.  The other operand is the
// sum of two e4m3 numbers, one product each into the same sums.  q, times a power
// of two for its row, is such a sum exactly but for elements below 2^-17 of the
// row's largest (a bf16 number has 8 significant bits, an e4m3 number 4).  A
// weight w_j = 2^(t_j - max + 8) with t_j = s_j log2(e) + log2(b_j), the maximum
// over the 32 keys at hand, is one to 2^-9 of itself (or 2^-18 of the maximum).
// The 32 keys' product is then added in fp32, times 2^(max - row maximum), so that
// small weights keep their digits whatever other keys weigh.  The softmax's sum is
// that of w_j / b_j.  (One thread's row of a tcgen05 product would have to be
// scaled alike for all keys: its sums stay in the tensor memory.)
//
// Work.  Items, shares and parts are those of attention_line.cuh.  Eight warps
// have R rows each (8: decoding; 16: chunks).  Where an item has fewer rows, warps
// share them and each takes every KS-th 32 keys; their sums are joined through
// shared memory in a fixed order.  A ninth warp feeds a ring of 64-key tiles: codes
// by TMA, page by page (swizzled, so that the fragments' 16-byte reads meet no bank
// twice), scales by 4-byte asynchronous copies.
//
// V is the product's B operand with its keys in a row: four keys' words are
// transposed in registers by byte permutes.  The orders of the head's elements
// (for q.k) and of the 32 keys (for w.v) within a product are free; they are
// chosen so that a thread's fragments are neighbouring bytes of the cache and the
// scores it holds are the weights that it needs.
#include <cuda_bf16.h>
#include <math_constants.h>

#include <algorithm>
#include <climits>

#include "../../include/lowm_fp8.h"
#include "attention_line.cuh"
#include "fp8_device.cuh"
#include "layer_device.cuh"
#include "layer_host.h"

namespace lowm {
namespace {

constexpr int kWarps = 8;                    // that compute
constexpr int kThreads8 = 32 * (kWarps + 1);
constexpr int kUnitKeys = 32;                // of one product
constexpr int kMaxCtas = 320;
constexpr int kItemCost8 = 4, kMinShare8 = 4;
constexpr float kWeightLog2 = 8.f;           // the largest weight is 2^8 (e4m3 ends at 448)
constexpr float kMaxScale = 1.125899906842624e15f;   // 2^50: scales are taken as 2^-50 .. 2^50

// Bits of the device status word (above those of the other operators).
enum : uint32_t {
    kErrAttn8Ring = 1u << 22,
    kErrAttn8Full = 1u << 23,
    kErrAttn8Base = 1u << 24,                // dynamic shared memory not on a 1024-byte boundary
};

struct CutItem8 {
    int parts;                               // shares the item lies in; 0: there is none
    int q0, q_len, head, q_tile;
};

template <int ROWS>
struct Attn8Params : LineParams<ROWS, kItemCost8, kMinShare8> {
    const __nv_bfloat16 *q;
    const float *k_scale, *v_scale;
    __nv_bfloat16 *out;
    float *lse;
    int64_t q_ts, q_hs, o_ts, o_hs, table_stride, num_pages;
    int64_t ks_page, ks_block, ks_head, vs_page, vs_block, vs_head;
    const int32_t *table;
    int page_size, page_shift, block_shift, heads, slot_rows;
    float scale_log2;                        // scale * log2(e)
    bool q_vec, out_vec;                     // 16-byte rows
    float *parts;                            // [2 * ctas][slot_rows][dim] sums, then [2 * ctas][slot_rows] (max, sum) pairs
    CutItem8 *cuts;                          // [ctas]
    unsigned int *status;
};

// ------------------------------------------------------------------ PTX of this kernel
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// c += A . B, e4m3, A [16 x 32] row-major, B [32 x 8] column-major.
__device__ __forceinline__ void mma_e4m3(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void *tmap, int x, int y, int z, int w, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}

// Copies 4 bytes when `bytes` is 4 and writes zeros when it is 0.
__device__ __forceinline__ void copy_async_4(uint32_t dst, const float *src, uint32_t bytes)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// Arrives on `bar`, whose count includes this, once this thread's copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint32_t bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

template <int BYTES>
__device__ __forceinline__ void load_shared(uint32_t at, uint32_t (&w)[BYTES / 4])
{
    if constexpr (BYTES == 16)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at));
    else
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at));
}

// ------------------------------------------------------------------ shared memory
template <int DIM, int R>
struct Attn8Smem {
    static constexpr uint32_t kTileBytes = kTileKeys * DIM;             // of K or V; 1024-byte multiples
    static constexpr uint32_t kStages = (R == 8 ? 5 : 10) * (128 / DIM);
    static constexpr uint32_t kOut = R * DIM / 32;                      // sums a thread holds
    static constexpr uint32_t kScales = kStages * 2 * kTileBytes;       // [stages][K, V][64]
    static constexpr uint32_t kMerge = kScales + kStages * 2 * kTileKeys * 4;   // [4 warps][kOut + 4][32]
    static constexpr uint32_t kKeys = kMerge + 4 * (kOut + 4) * 32 * 4;         // [warps][3][32] of the 32 keys at hand
    static constexpr uint32_t kBars = kKeys + kWarps * 3 * kUnitKeys * 4;       // full, empty [stages]
    static constexpr uint32_t kBytes = kBars + 2 * kStages * 8;
};

// 0xff in the bytes of NaN codes.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w)
{
    return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu);
}

// Transposes 4 x 4 bytes: out word d holds byte d of w[0], w[1], w[2], w[3].
__device__ __forceinline__ void transpose_bytes(uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3, uint32_t (&out)[4])
{
    const uint32_t a = __byte_perm(w0, w1, 0x5140), b = __byte_perm(w0, w1, 0x7362);
    const uint32_t c = __byte_perm(w2, w3, 0x5140), d = __byte_perm(w2, w3, 0x7362);
    out[0] = __byte_perm(a, c, 0x5410);
    out[1] = __byte_perm(a, c, 0x7632);
    out[2] = __byte_perm(b, d, 0x5410);
    out[3] = __byte_perm(b, d, 0x7632);
}

// One warp's R rows of an item: q, running maximum, sum and weighted values.  Thread 4 g + t holds row g (and g + 8):
// of q elements [DIM / 4 t, DIM / 4 (t + 1)), of the sums the same ones, sums[e] being element e, then, from DIM / 8 on,
// DIM / 8 + e of them.
template <int DIM, int R>
struct Rows8 {
    static constexpr int kSets = R / 8;      // rows a thread holds
    uint32_t q[2][DIM / 32][4];              // two terms
    float unit[kSets];                       // power of two that q was divided by
    float top[kSets], sum[kSets];            // (sum: this thread's keys)
    float out[DIM / 8][2 * kSets];
};

template <int DIM, int R, class P>
__device__ __forceinline__ void load_rows(const P &p, const Row (&rows)[R / 8], Rows8<DIM, R> &x)
{
    constexpr int N = DIM / 4;               // elements a thread holds of a row
    const int t = threadIdx.x & 3;
#pragma unroll
    for (int i = 0; i < DIM / 32; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            x.q[0][i][j] = x.q[1][i][j] = 0;
#pragma unroll
    for (int set = 0; set < R / 8; ++set) {
        alignas(16) __nv_bfloat16 v[N];
        const __nv_bfloat16 *from = p.q + rows[set].token * p.q_ts + rows[set].q_head * p.q_hs + N * t;
#pragma unroll
        for (int i = 0; i < N; i += 8) {
            if (!rows[set].valid) {
                *reinterpret_cast<uint4 *>(v + i) = make_uint4(0, 0, 0, 0);
            } else if (p.q_vec) {
                *reinterpret_cast<uint4 *>(v + i) = *reinterpret_cast<const uint4 *>(from + i);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[i + j] = from[i + j];
            }
        }
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i)
            amax = fmaxf(amax, finite_magnitude(__bfloat162float(v[i])));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const int e = scale_exponent(amax);
        x.unit[set] = power_of_two(e);
        const float inverse = power_of_two(-e);
#pragma unroll
        for (int i = 0; i < N; i += 4) {     // four elements: one word of each term
            uint32_t w0 = 0, w1 = 0;
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                const float a = nan_unless_finite(__bfloat162float(v[i + j])) * inverse;
                const float b = nan_unless_finite(__bfloat162float(v[i + j + 1])) * inverse;
                const uint32_t first = to_e4m3x2(a, b);
                const float2 back = __half22float2(e4m3x2_to_half2(first));
                w0 |= first << (8 * j);
                w1 |= to_e4m3x2(a - back.x, b - back.y) << (8 * j);
            }
            x.q[0][i / 8][(i & 4) / 2 + set] = w0;
            x.q[1][i / 8][(i & 4) / 2 + set] = w1;
        }
        x.top[set] = -CUDART_INF_F;
        x.sum[set] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < DIM / 8; ++i)
#pragma unroll
        for (int j = 0; j < 2 * (R / 8); ++j)
            x.out[i][j] = 0.f;
}

// The 32 keys from key0 on (rows `first` to `first` + 31 of the tile) for one warp's rows.
template <int DIM, int R>
__device__ __forceinline__ void attend(Rows8<DIM, R> &x, const Row (&rows)[R / 8], const Seen &seen, int key0, int first,
                                       uint32_t k_tile, uint32_t v_tile, const float *scales, float *mine, float scale_log2)
{
    constexpr int kSets = R / 8;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    // Scales of the 32 keys, a key a lane; those that no row sees count nothing.
    {
        const int key = key0 + lane;
        const bool known = key >= seen.lo && key < seen.end;
        const float a = known ? scales[first + lane] * scale_log2 : 0.f;
        const float b = known ? fminf(fmaxf(scales[kTileKeys + first + lane], 1.f / kMaxScale), kMaxScale) : 1.f;
        mine[lane] = a;
        mine[32 + lane] = __log2f(b);
        mine[64 + lane] = __fdividef(1.f, b);
        __syncwarp();
    }
    // Scores: thread 4 g + t has keys 8 j + 2 t, 8 j + 2 t + 1 of rows g and g + 8.
    float s[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
        const int row = first + 8 * j + g;
#pragma unroll
        for (int i = 0; i < DIM / 64; ++i) {
            uint32_t w[4];
            const uint32_t chunk = DIM == 128 ? (uint32_t)((2 * t + i) ^ (row & 7)) : (uint32_t)(t ^ ((row >> 1) & 3));
            load_shared<16>(k_tile + row * DIM + chunk * 16, w);
#pragma unroll
            for (int term = 0; term < 2; ++term) {
                mma_e4m3(s[j], x.q[term][2 * i], w[0], w[1]);
                mma_e4m3(s[j], x.q[term][2 * i + 1], w[2], w[3]);
            }
        }
    }
    float2 inverse[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 a = *reinterpret_cast<const float2 *>(mine + 8 * j + 2 * t);
        const float2 b = *reinterpret_cast<const float2 *>(mine + 32 + 8 * j + 2 * t);
        inverse[j] = *reinterpret_cast<const float2 *>(mine + 64 + 8 * j + 2 * t);
#pragma unroll
        for (int set = 0; set < kSets; ++set) {
            s[j][2 * set] = fmaf(s[j][2 * set] * a.x, x.unit[set], b.x);
            s[j][2 * set + 1] = fmaf(s[j][2 * set + 1] * a.y, x.unit[set], b.y);
        }
    }
    const bool edge = key0 < seen.all_lo || key0 + kUnitKeys - 1 > seen.all_hi;
    if (edge) {
#pragma unroll
        for (int set = 0; set < kSets; ++set) {
            const int hi = rows[set].valid ? rows[set].hi - key0 : -1, lo = rows[set].lo - key0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int k = 8 * j + 2 * t + c;
                    if (k > hi || k < lo)
                        s[j][2 * set + c] = -CUDART_INF_F;
                }
        }
    }
    // Weights, as two terms.
    uint32_t w0[4] = {}, w1[4] = {};
    float factor[kSets];
#pragma unroll
    for (int set = 0; set < kSets; ++set) {
        float top = -CUDART_INF_F;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            top = fmaxf(top, fmaxf(s[j][2 * set], s[j][2 * set + 1]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float shift = top == -CUDART_INF_F ? 0.f : top - kWeightLog2;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float a = ex2(s[j][2 * set] - shift), b = ex2(s[j][2 * set + 1] - shift);
            sum = fmaf(a, inverse[j].x, fmaf(b, inverse[j].y, sum));
            const __half2 h = __floats2half2_rn(a, b);
            const uint32_t one = half2_to_e4m3x2(h);
            const uint32_t two = half2_to_e4m3x2(__hsub2(h, e4m3x2_to_half2(one)));
            w0[(j & 2) + set] |= one << (16 * (j & 1));
            w1[(j & 2) + set] |= two << (16 * (j & 1));
        }
        // Into the row's sums, at the scale of its largest weight so far.
        const float now = fmaxf(x.top[set], top);
        const float before = now == x.top[set] ? 1.f : ex2(x.top[set] - now);
        factor[set] = top == -CUDART_INF_F ? 0.f : ex2(top - now);
        x.top[set] = now;
        x.sum[set] = fmaf(sum, factor[set], x.sum[set] * before);
        if (__any_sync(0xffffffffu, before != 1.f)) {
#pragma unroll
            for (int e = 0; e < DIM / 8; ++e) {
                x.out[e][2 * set] *= before;
                x.out[e][2 * set + 1] *= before;
            }
        }
        if (sum != sum)                      // a score that is not a number
            factor[set] = CUDART_NAN_F;
    }
    // Values.  Keys 4 t .. 4 t + 3 of the product's 32 are 2 t, 2 t + 1, 8 + 2 t, 9 + 2 t, and 16 + those for the second half.
    constexpr int kWords = DIM / 32;         // words of a key that a thread holds: elements DIM / 8 g ..
    uint32_t v[8][kWords];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = first + 16 * (i >> 2) + 8 * ((i >> 1) & 1) + 2 * t + (i & 1);
        if constexpr (DIM == 128)
            load_shared<16>(v_tile + row * DIM + ((g ^ (row & 7)) << 4), v[i]);
        else
            load_shared<8>(v_tile + row * DIM + (((g >> 1) ^ ((row >> 1) & 3)) << 4) + (g & 1) * 8, v[i]);
    }
    // A weight of 0 does not silence a NaN: keys that no row sees may hold anything and are cleared; NaN codes of keys
    // that some rows see and others do not are found apart, by counting for each row those that it sees.
    bool apart = false;
    uint32_t sees[4] = {};
    if (edge) {
        uint32_t bad = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int key = key0 + 16 * (i >> 2) + 8 * ((i >> 1) & 1) + 2 * t + (i & 1);
            const bool known = key >= seen.lo && key < seen.end;
#pragma unroll
            for (int w = 0; w < kWords; ++w) {
                v[i][w] = known ? v[i][w] : 0u;
                bad |= nan_codes(v[i][w]);
            }
        }
        apart = __any_sync(0xffffffffu, bad != 0);
        if (apart) {
#pragma unroll
            for (int set = 0; set < kSets; ++set)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int key = key0 + 16 * (i >> 2) + 8 * ((i >> 1) & 1) + 2 * t + (i & 1);
                    if (rows[set].valid && key <= rows[set].hi && key >= rows[set].lo)
                        sees[2 * (i >> 2) + set] |= 0x38u << (8 * (i & 3));      // 1.0
                }
        }
    }
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
        uint32_t b0[4], b1[4];
        transpose_bytes(v[0][w], v[1][w], v[2][w], v[3][w], b0);
        transpose_bytes(v[4][w], v[5][w], v[6][w], v[7][w], b1);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float o[4] = {0.f, 0.f, 0.f, 0.f};
            if (apart) {
                const uint32_t n0 = nan_codes(b0[e]), n1 = nan_codes(b1[e]);
                mma_e4m3(o, sees, n0 & 0x38383838u, n1 & 0x38383838u);
                b0[e] &= ~n0;
                b1[e] &= ~n1;
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    o[c] = o[c] > 0.f ? CUDART_NAN_F : 0.f;
            }
            mma_e4m3(o, w0, b0[e], b1[e]);
            mma_e4m3(o, w1, b0[e], b1[e]);
#pragma unroll
            for (int set = 0; set < kSets; ++set) {
                x.out[4 * w + e][2 * set] = fmaf(o[2 * set], factor[set], x.out[4 * w + e][2 * set]);
                x.out[4 * w + e][2 * set + 1] = fmaf(o[2 * set + 1], factor[set], x.out[4 * w + e][2 * set + 1]);
            }
        }
    }
    __syncwarp();                            // before `mine` is written again
}

// Joins the sums of the warps that share rows: in each step the upper half of them hand theirs over.  The warps'
// number is the same for the whole CTA; all of its kWarps warps come here.
template <int DIM, int R>
__device__ __forceinline__ void join_warps(Rows8<DIM, R> &x, float *merge, int warps, int row_tiles, int warp)
{
    constexpr int kSets = R / 8, kOut = R * DIM / 32;
    const int lane = threadIdx.x & 31;
    const int rt = warp % row_tiles, part = warp / row_tiles;
    for (int half = warps / 2; half > 0; half /= 2) {
        float *at = merge + ((part & (half - 1)) * row_tiles + rt) * (kOut + 4) * 32 + lane;
        if (part >= half && part < 2 * half) {
#pragma unroll
            for (int e = 0; e < DIM / 8; ++e)
#pragma unroll
                for (int c = 0; c < 2 * kSets; ++c)
                    at[(e * 2 * kSets + c) * 32] = x.out[e][c];
#pragma unroll
            for (int set = 0; set < kSets; ++set) {
                at[(kOut + 2 * set) * 32] = x.top[set];
                at[(kOut + 2 * set + 1) * 32] = x.sum[set];
            }
        }
        ptx::named_barrier_sync(1, 32 * kWarps);
        if (part < half) {
#pragma unroll
            for (int set = 0; set < kSets; ++set) {
                const float top = at[(kOut + 2 * set) * 32];
                const float now = fmaxf(x.top[set], top);
                const float base = now == -CUDART_INF_F ? 0.f : now;
                const float a = ex2(x.top[set] - base), b = ex2(top - base);
                x.top[set] = now;
                x.sum[set] = fmaf(x.sum[set], a, at[(kOut + 2 * set + 1) * 32] * b);
#pragma unroll
                for (int e = 0; e < DIM / 8; ++e)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        x.out[e][2 * set + c] = fmaf(x.out[e][2 * set + c], a, at[(e * 2 * kSets + 2 * set + c) * 32] * b);
            }
        }
        ptx::named_barrier_sync(1, 32 * kWarps);
    }
}

template <int DIM, int R>
__global__ void __launch_bounds__(kThreads8, R == 8 ? 2 : 1)
    paged_attention_fp8_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                               const Attn8Params<kWarps * R> p)
{
    using L = Attn8Smem<DIM, R>;
    constexpr int kSets = R / 8;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = ptx::smem_u32(smem);
    const uint32_t bar_full = sbase + L::kBars, bar_empty = bar_full + 8 * L::kStages;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (sbase & 1023u) {                     // (the swizzle's pattern follows the address)
        if (threadIdx.x == 0)
            atomicOr(p.status, kErrAttn8Base);
        return;
    }
    if (threadIdx.x == 0) {
        for (uint32_t s = 0; s < L::kStages; ++s) {
            ptx::mbar_init(bar_full + 8 * s, 1 + 32);        // the codes, and each lane's scales
            ptx::mbar_init(bar_empty + 8 * s, kWarps);
        }
        ptx::fence_mbarrier_init_cluster();
        ptx::fence_proxy_async_shared();
    }
    __syncthreads();
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    const Line line = make_line(p);
    const int share = share_of(p, line.total, gridDim.x);
    const int begin = (int)min((int64_t)share * blockIdx.x, (int64_t)line.total), end = min(share, line.total - begin) + begin;
    if (threadIdx.x == 0)
        p.cuts[blockIdx.x].parts = 0;        // until this thread finds one
    Piece c;
    if (!(begin < end && first_piece(p, c, line, begin, end)))
        return;
    const Item &it = c.it;
    uint32_t i = 0;                          // tiles passed
    bool ok = true;
    if (warp == kWarps) {
        // ------------------------------------------------------------ loads
        const int box_keys = min(p.page_size, kTileKeys), boxes = kTileKeys / box_keys;
        const int mine = lane & 7;           // lanes 0-7: this lane's box of K, 8-15: of V
        const CUtensorMap *map = lane < 8 ? &map_k : &map_v;
        const uint32_t at = (lane < 8 ? 0 : L::kTileBytes) + mine * box_keys * DIM;
        do {
            const int from = c.from, n = c.to - c.from;
            const int32_t *pages = p.table + it.b * p.table_stride;
            // The page of a key: -1 past the sequence's end.
            auto entry = [&](int key) { return key < it.kv ? pages[key >> p.page_shift] : -1; };
            auto box_key = [&](int j) { return (it.first_tile + j) * kTileKeys + mine * box_keys; };
            auto key_at = [&](int j, int h) { return (it.first_tile + j) * kTileKeys + 32 * h + lane; };
            int box = mine < boxes ? entry(box_key(from)) : -1;
            int page[2] = {entry(key_at(from, 0)), entry(key_at(from, 1))};
            for (int j = from; j < from + n; ++j, ++i) {
                int next_box = -1, next[2] = {-1, -1};
                if (j + 1 < from + n) {
                    next_box = mine < boxes ? entry(box_key(j + 1)) : -1;
                    next[0] = entry(key_at(j + 1, 0));
                    next[1] = entry(key_at(j + 1, 1));
                }
                const uint32_t s = i % L::kStages;
                if (!wait_short(bar_empty + 8 * s, ((i / L::kStages) & 1) ^ 1)) {
                    ok = false;
                    atomicOr(p.status, kErrAttn8Ring);
                }
                ok = __all_sync(0xffffffffu, ok);
                if (!ok)
                    break;
                const int key0 = (it.first_tile + j) * kTileKeys;
                const int used = min(boxes, max(1, (it.kv - key0 + box_keys - 1) / box_keys));   // pages past the end are not requested
                if (lane == 0)
                    ptx::mbar_arrive_expect_tx(bar_full + 8 * s, 2u * used * box_keys * DIM);
                __syncwarp();
                if (lane < 16 && mine < used)
                    tma_load_4d(sbase + s * 2 * L::kTileBytes + at, map, 0, key0 & (p.page_size - 1), it.head, box, bar_full + 8 * s);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const bool known = page[h] >= 0 && page[h] < p.num_pages;
                    const int64_t pg = known ? page[h] : 0;
                    const int64_t block = (key_at(j, h) & (p.page_size - 1)) >> p.block_shift;
                    const uint32_t to = sbase + L::kScales + (s * 2 * kTileKeys + 32 * h + lane) * 4;
                    copy_async_4(to, p.k_scale + pg * p.ks_page + block * p.ks_block + it.head * p.ks_head, known ? 4 : 0);
                    copy_async_4(to + kTileKeys * 4, p.v_scale + pg * p.vs_page + block * p.vs_block + it.head * p.vs_head, known ? 4 : 0);
                    page[h] = next[h];
                }
                copies_arrive(bar_full + 8 * s);
                box = next_box;
            }
        } while (ok && next_piece(p, c, end));
        // No copy may land after the CTA has ended: normally all were consumed long ago.
        for (uint32_t j = i > L::kStages ? i - L::kStages : 0; j < i; ++j)
            (void)wait_short(bar_full + 8 * (j % L::kStages), (j / L::kStages) & 1);
        return;
    }
    // ---------------------------------------------------------------- rows
    float *keys = reinterpret_cast<float *>(smem + L::kKeys) + warp * 3 * kUnitKeys;
    float *merge = reinterpret_cast<float *>(smem + L::kMerge);
    const int g = lane >> 2, t = lane & 3;
    do {
        const int from = c.from, n = c.to - c.from;
        const int in_item = min(p.kRows, it.q_len * p.group - it.q_tile * p.kRows);
        int row_tiles = 1;
        while (row_tiles * R < in_item)
            row_tiles *= 2;
        const int sharing = kWarps / row_tiles, rt = warp % row_tiles, part = warp / row_tiles;
        Row rows[kSets];
#pragma unroll
        for (int set = 0; set < kSets; ++set)
            rows[set] = row_of(p, it, rt * R + 8 * set + g);
        const bool has_rows = __any_sync(0xffffffffu, rows[0].valid);
        const Seen seen = seen_by(p, it);
        Rows8<DIM, R> x;
        load_rows<DIM, R>(p, rows, x);
        for (int j = 0; j < n; ++j, ++i) {
            const uint32_t s = i % L::kStages;
            if (ok && !wait_short(bar_full + 8 * s, (i / L::kStages) & 1)) {
                ok = false;
                atomicOr(p.status, kErrAttn8Full);
            }
            ok = __all_sync(0xffffffffu, ok);
            const uint32_t k_tile = sbase + s * 2 * L::kTileBytes;
            const float *scales = reinterpret_cast<const float *>(smem + L::kScales) + s * 2 * kTileKeys;
#pragma unroll 1
            for (int h = 0; h < kTileKeys / kUnitKeys; ++h)
                if (ok && has_rows && ((2 * j + h) & (sharing - 1)) == part)
                    attend<DIM, R>(x, rows, seen, (it.first_tile + from + j) * kTileKeys + kUnitKeys * h, kUnitKeys * h, k_tile,
                                   k_tile + L::kTileBytes, scales, keys, p.scale_log2);
            __syncwarp();
            if (lane == 0)
                ptx::mbar_arrive(bar_empty + 8 * s);
        }
        if (sharing > 1)
            join_warps<DIM, R>(x, merge, sharing, row_tiles, warp);
        // The item's rows: finished here, or a part for the join.
        const bool whole = n == it.tiles;
        const int64_t slot = 2 * (int64_t)blockIdx.x + (from == 0 ? 1 : 0);
        if (threadIdx.x == 0 && from == 0 && !whole)
            p.cuts[blockIdx.x] = {(it.start + p.kCost + it.tiles - 1) / share - (int)blockIdx.x + 1, it.q0, it.q_len, it.head,
                                  it.q_tile};
        if (part == 0) {
#pragma unroll
            for (int set = 0; set < kSets; ++set) {
                float sum = x.sum[set];
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                if (!rows[set].valid)
                    continue;
                constexpr int N = DIM / 8;
                if (whole) {
                    const float inv = sum == 0.f ? 0.f : 1.f / sum;
                    __nv_bfloat16 *o = p.out + rows[set].token * p.o_ts + rows[set].q_head * p.o_hs + 2 * N * t;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        alignas(16) __nv_bfloat162 v[N / 2];
#pragma unroll
                        for (int e = 0; e < N; e += 2)
                            v[e / 2] = __floats2bfloat162_rn(x.out[e][2 * set + half] * inv, x.out[e + 1][2 * set + half] * inv);
                        if (p.out_vec) {
#pragma unroll
                            for (int e = 0; e < N; e += 8)
                                *reinterpret_cast<uint4 *>(o + N * half + e) = *reinterpret_cast<const uint4 *>(v + e / 2);
                        } else {
#pragma unroll
                            for (int e = 0; e < N; e += 2) {
                                o[N * half + e] = v[e / 2].x;
                                o[N * half + e + 1] = v[e / 2].y;
                            }
                        }
                    }
                    if (p.lse && t == 0)
                        p.lse[(int64_t)rows[set].token * p.heads + rows[set].q_head] =
                            sum == 0.f ? -CUDART_INF_F : (x.top[set] - kWeightLog2 + log2f(sum)) * CUDART_LN2_F;
                } else {
                    const int64_t row = slot * p.slot_rows + rt * R + 8 * set + g;
                    float *o = p.parts + row * DIM + 2 * N * t;
#pragma unroll
                    for (int half = 0; half < 2; ++half)
#pragma unroll
                        for (int e = 0; e < N; e += 4)
                            *reinterpret_cast<float4 *>(o + N * half + e) =
                                make_float4(x.out[e][2 * set + half], x.out[e + 1][2 * set + half], x.out[e + 2][2 * set + half],
                                            x.out[e + 3][2 * set + half]);
                    if (t == 0)
                        reinterpret_cast<float2 *>(p.parts + 2 * (int64_t)gridDim.x * p.slot_rows * DIM)[row] =
                            make_float2(x.top[set], sum);
                }
            }
        }
    } while (next_piece(p, c, end));
}

// Joins the parts of the items that shares cut: CTA c owns the one that begins in share c and ends in a later one.  A
// thread owns four elements of a row.  Part i counts 2^(its maximum - the largest one), and the parts add in the order
// of the keys.
constexpr int kJoinThreads8 = 256, kJoinSplit8 = 4;

template <int DIM, int ROWS>
__global__ void __launch_bounds__(kJoinThreads8) join_parts_fp8_kernel(const Attn8Params<ROWS> p, int ctas)
{
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    if (blockIdx.x == 0 && blockIdx.y == 0) {   // rows of no sequence
        const int first = p.batch > 0 ? min(max(p.cu_q[0], 0), p.q_tokens) : p.q_tokens;
        const int last = p.batch > 0 ? min(max(p.cu_q[p.batch], 0), p.q_tokens) : p.q_tokens;
        for (int t = threadIdx.x >> 5; t < p.q_tokens; t += kJoinThreads8 / 32)
            if (t < first || t >= last)
                for (int h = 0; h < p.heads; ++h) {
                    for (int d = threadIdx.x & 31; d < DIM; d += 32)
                        p.out[t * p.o_ts + h * p.o_hs + d] = __float2bfloat16_rn(0.f);
                    if ((threadIdx.x & 31) == 0 && p.lse)
                        p.lse[(int64_t)t * p.heads + h] = -CUDART_INF_F;
                }
    }
    if (p.batch == 0)
        return;
    const CutItem8 cut = p.cuts[blockIdx.x];
    if (cut.parts == 0)
        return;
    const float2 *ml = reinterpret_cast<const float2 *>(p.parts + 2 * (int64_t)ctas * p.slot_rows * DIM);
    const int rows = min(ROWS, cut.q_len * p.group - cut.q_tile * ROWS);
    auto slot = [&](int i) { return 2 * (int64_t)(blockIdx.x + i) + (i == 0 ? 1 : 0); };
    for (int c = threadIdx.x + blockIdx.y * kJoinThreads8; c < rows * (DIM / 4); c += kJoinSplit8 * kJoinThreads8) {
        const int r = c / (DIM / 4), d = c % (DIM / 4) * 4;
        const int row = cut.q_tile * ROWS + r, t = cut.q0 + row / p.group, h = cut.head * p.group + row % p.group;
        float top = -CUDART_INF_F;
#pragma unroll 4
        for (int i = 0; i < cut.parts; ++i)
            top = fmaxf(top, ml[slot(i) * p.slot_rows + r].x);
        const float base = top == -CUDART_INF_F ? 0.f : top;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.f;
#pragma unroll 4
        for (int i = 0; i < cut.parts; ++i) {
            const float2 x = ml[slot(i) * p.slot_rows + r];
            const float4 o = *reinterpret_cast<const float4 *>(p.parts + (slot(i) * p.slot_rows + r) * DIM + d);
            const float a = ex2(x.x - base);
            sum = fmaf(x.y, a, sum);
            acc.x = fmaf(o.x, a, acc.x);
            acc.y = fmaf(o.y, a, acc.y);
            acc.z = fmaf(o.z, a, acc.z);
            acc.w = fmaf(o.w, a, acc.w);
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        alignas(8) __nv_bfloat162 v[2] = {__floats2bfloat162_rn(acc.x * inv, acc.y * inv), __floats2bfloat162_rn(acc.z * inv, acc.w * inv)};
        __nv_bfloat16 *o = p.out + t * p.o_ts + h * p.o_hs + d;
        if (p.out_vec) {
            *reinterpret_cast<uint2 *>(o) = *reinterpret_cast<const uint2 *>(v);
        } else {
            o[0] = v[0].x;
            o[1] = v[0].y;
            o[2] = v[1].x;
            o[3] = v[1].y;
        }
        if (p.lse && d == 0)
            p.lse[(int64_t)t * p.heads + h] = sum == 0.f ? -CUDART_INF_F : (base - kWeightLog2 + log2f(sum)) * CUDART_LN2_F;
    }
}

constexpr int kMaxGroup = 128;

bool attention_fp8_shape_ok(int batch, int q_tokens, int heads, int kv_heads, int dim)
{
    return batch >= 0 && q_tokens >= 0 && heads > 0 && kv_heads > 0 && heads % kv_heads == 0 && heads / kv_heads <= kMaxGroup &&
           (dim == 64 || dim == 128) && (int64_t)q_tokens * heads < INT_MAX / 2;
}

// Rows a part can have: a tile's, or all there are.
int slot_rows_fp8(int q_tokens, int heads, int kv_heads)
{
    return (int)std::min<int64_t>(16 * kWarps, std::max<int64_t>(1, (int64_t)q_tokens * (heads / kv_heads)));
}

// (dim, place, head, page) view of a cache of codes; a box is one head's row of up to 64 places of a page, zeros outside.
lowm_status_t encode_codes(const void *base, int64_t page_stride, int64_t place_stride, int64_t head_stride, int64_t num_pages,
                           int page_size, int kv_heads, int dim, CUtensorMap *map)
{
    EncodeTiledFn enc = host_encode_fn();
    if (!enc)
        return LOWM_ERR_CUDA;
    // A dimension of one never uses its stride, but the encoder checks it.
    const cuuint64_t unit = 16;
    const cuuint64_t dims[4] = {(cuuint64_t)dim, (cuuint64_t)page_size, (cuuint64_t)kv_heads, (cuuint64_t)num_pages};
    const cuuint64_t strides[3] = {page_size > 1 ? (cuuint64_t)place_stride : unit, kv_heads > 1 ? (cuuint64_t)head_stride : unit,
                                   num_pages > 1 ? (cuuint64_t)page_stride : unit};
    const cuuint32_t box[4] = {(cuuint32_t)dim, (cuuint32_t)std::min(page_size, kTileKeys), 1, 1};
    const cuuint32_t step[4] = {1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(base), dims, strides, box, step,
               CU_TENSOR_MAP_INTERLEAVE_NONE, dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? LOWM_OK
               : LOWM_ERR_CUDA;
}

template <int DIM, int R>
lowm_status_t launch_fp8(const CUtensorMap &map_k, const CUtensorMap &map_v, const Attn8Params<kWarps * R> &p, int sms, void *stream)
{
    static SmemOptIn opt_in;
    if (!opt_in.set(reinterpret_cast<const void *>(paged_attention_fp8_kernel<DIM, R>), Attn8Smem<DIM, R>::kBytes))
        return LOWM_ERR_CUDA;
    const int ctas = std::min((R == 8 ? 2 : 1) * sms, kMaxCtas);
    if (p.batch > 0) {
        const lowm_status_t st = launch_pdl(paged_attention_fp8_kernel<DIM, R>, dim3((unsigned)ctas), dim3(kThreads8),
                                            Attn8Smem<DIM, R>::kBytes, stream, map_k, map_v, p);
        if (st != LOWM_OK)
            return st;
    }
    return launch_pdl(join_parts_fp8_kernel<DIM, kWarps * R>, dim3((unsigned)ctas, kJoinSplit8), dim3(kJoinThreads8), 0, stream, p,
                      ctas);
}

}  // namespace
}  // namespace lowm

extern "C" size_t lowm_paged_attention_fp8_workspace(int batch, int q_tokens, int heads, int kv_heads, int dim)
{
    using namespace lowm;
    if (!attention_fp8_shape_ok(batch, q_tokens, heads, kv_heads, dim))
        return 0;
    return (size_t)2 * kMaxCtas * slot_rows_fp8(q_tokens, heads, kv_heads) * (dim + 2) * sizeof(float) + kMaxCtas * sizeof(CutItem8);
}

extern "C" lowm_status_t lowm_paged_attention_fp8(
    const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *k_cache, int64_t k_page_stride,
    int64_t k_place_stride, int64_t k_cache_head_stride, const void *v_cache, int64_t v_page_stride, int64_t v_place_stride,
    int64_t v_cache_head_stride, const float *k_scale, int64_t ks_page_stride, int64_t ks_block_stride, int64_t ks_head_stride,
    const float *v_scale, int64_t vs_page_stride, int64_t vs_block_stride, int64_t vs_head_stride, int64_t num_pages,
    int page_size, int block, const int32_t *page_table, int64_t page_table_stride, int table_width, const int32_t *kv_lens,
    const int32_t *cu_q, void *out, int64_t out_token_stride, int64_t out_head_stride, float *lse, int batch, int q_tokens,
    int heads, int kv_heads, int dim, float scale, int window, void *workspace, size_t workspace_bytes, void *stream)
{
    using namespace lowm;
    if (batch < 0 || q_tokens < 0 || heads <= 0 || kv_heads <= 0 || dim <= 0 || num_pages <= 0 || num_pages > INT_MAX ||
        page_size <= 0 || block <= 0 || table_width < 0 || window < 0 || !(scale == scale))
        return LOWM_ERR_INVALID_ARGUMENT;
    if (!attention_fp8_shape_ok(batch, q_tokens, heads, kv_heads, dim) || page_size < 8 || page_size > 1024 ||
        (page_size & (page_size - 1)) || block > page_size || (block & (block - 1)))
        return LOWM_ERR_UNSUPPORTED_SHAPE;
    if (q_tokens == 0)
        return LOWM_OK;
    if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !cu_q || !out || !workspace || (batch && !kv_lens) ||
        (batch && table_width && !page_table))
        return LOWM_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < lowm_paged_attention_fp8_workspace(batch, q_tokens, heads, kv_heads, dim))
        return LOWM_ERR_INVALID_ARGUMENT;
    const int64_t cache_strides[] = {k_page_stride, k_place_stride, k_cache_head_stride,
                                     v_page_stride, v_place_stride, v_cache_head_stride};
    const int64_t extents[] = {num_pages, page_size, kv_heads, num_pages, page_size, kv_heads};
    for (int i = 0; i < 6; ++i) {
        if (extents[i] == 1)                     // the stride of a single one is not used
            continue;
        if (cache_strides[i] < 0)
            return LOWM_ERR_INVALID_ARGUMENT;
        if (cache_strides[i] & 15)
            return LOWM_ERR_MISALIGNED;
    }
    const int64_t more[] = {q_token_stride, q_head_stride, out_token_stride, out_head_stride, page_table_stride, ks_page_stride,
                            ks_block_stride, ks_head_stride, vs_page_stride, vs_block_stride, vs_head_stride};
    for (int64_t s : more)
        if (s < 0)
            return LOWM_ERR_INVALID_ARGUMENT;
    if (!is_aligned(k_cache, 16) || !is_aligned(v_cache, 16) || !is_aligned(workspace, 16) || !is_aligned(q, 2) ||
        !is_aligned(out, 2) || !is_aligned(page_table, 4) || !is_aligned(kv_lens, 4) || !is_aligned(cu_q, 4) ||
        !is_aligned(lse, 4) || !is_aligned(k_scale, 4) || !is_aligned(v_scale, 4))
        return LOWM_ERR_MISALIGNED;
    // The tensor maps take strides below 2^40 bytes, and no stride of 0 where it is used.
    for (int i = 0; i < 6; ++i)
        if (extents[i] > 1 && (cache_strides[i] == 0 || cache_strides[i] >= ((int64_t)1 << 40)))
            return LOWM_ERR_INVALID_ARGUMENT;
    // Tile counts are 32-bit in the kernels, rounding up to equal shares included.
    const int group = heads / kv_heads;
    const int64_t capacity = std::min<int64_t>((int64_t)table_width * page_size, kMaxKeys);
    const int64_t q_tiles = (int64_t)q_tokens * group / (8 * kWarps) + batch;
    if ((double)q_tiles * kv_heads * (double)(capacity / kTileKeys + 2 + kItemCost8) > (double)(INT_MAX - kMinShare8 * kMaxCtas))
        return LOWM_ERR_UNSUPPORTED_SHAPE;
    int sms = 0;
    lowm_status_t st = host_check_device(&sms);
    if (st != LOWM_OK)
        return st;
    unsigned int *status = host_status_word();
    if (!status)
        return LOWM_ERR_CUDA;
    CUtensorMap map_k, map_v;
    if ((st = encode_codes(k_cache, k_page_stride, k_place_stride, k_cache_head_stride, num_pages, page_size, kv_heads, dim,
                           &map_k)) != LOWM_OK ||
        (st = encode_codes(v_cache, v_page_stride, v_place_stride, v_cache_head_stride, num_pages, page_size, kv_heads, dim,
                           &map_v)) != LOWM_OK)
        return st;

    auto fill = [&](auto &p) {
        p.q = static_cast<const __nv_bfloat16 *>(q);
        p.out = static_cast<__nv_bfloat16 *>(out);
        p.lse = lse;
        p.q_ts = q_token_stride;
        p.q_hs = q_head_stride;
        p.o_ts = out_token_stride;
        p.o_hs = out_head_stride;
        p.k_scale = k_scale;
        p.ks_page = ks_page_stride;
        p.ks_block = ks_block_stride;
        p.ks_head = ks_head_stride;
        p.v_scale = v_scale;
        p.vs_page = vs_page_stride;
        p.vs_block = vs_block_stride;
        p.vs_head = vs_head_stride;
        p.table = page_table;
        p.table_stride = page_table_stride;
        p.num_pages = num_pages;
        p.kv_lens = kv_lens;
        p.cu_q = cu_q;
        p.page_size = page_size;
        p.page_shift = p.block_shift = 0;
        while ((1 << p.page_shift) < page_size)
            ++p.page_shift;
        while ((1 << p.block_shift) < block)
            ++p.block_shift;
        p.batch = batch;
        p.q_tokens = q_tokens;
        p.heads = heads;
        p.kv_heads = kv_heads;
        p.group = group;
        p.window = window < kMaxKeys ? window : 0;
        p.capacity = (int)capacity;
        p.slot_rows = slot_rows_fp8(q_tokens, heads, kv_heads);
        p.scale_log2 = scale * 1.44269504088896340736f;
        p.q_vec = is_aligned(q, 16) && !((q_token_stride | q_head_stride) & 7);
        p.out_vec = is_aligned(out, 16) && !((out_token_stride | out_head_stride) & 7);
        p.parts = static_cast<float *>(workspace);
        p.cuts = reinterpret_cast<CutItem8 *>(static_cast<uint8_t *>(workspace) +
                                              (size_t)2 * kMaxCtas * p.slot_rows * (dim + 2) * sizeof(float));
        p.status = status;
    };
    // Rows that a sequence brings on average: few go to warps of 8 rows, two CTAs an SM.
    if ((int64_t)q_tokens * group <= 32 * (int64_t)std::max(batch, 1)) {
        Attn8Params<8 * kWarps> p;
        fill(p);
        return dim == 64 ? launch_fp8<64, 8>(map_k, map_v, p, sms, stream) : launch_fp8<128, 8>(map_k, map_v, p, sms, stream);
    }
    Attn8Params<16 * kWarps> p;
    fill(p);
    return dim == 64 ? launch_fp8<64, 16>(map_k, map_v, p, sms, stream) : launch_fp8<128, 16>(map_k, map_v, p, sms, stream);
}
