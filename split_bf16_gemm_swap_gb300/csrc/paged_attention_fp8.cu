// Attention of each sequence's newest tokens over a paged cache of e4m3 codes
// with a scale for each block of tokens and head (lowm_fp8.h).
//
//     s_j = scale (q . k_j) a_j,  out = sum_j softmax_j(s) b_j v_j
//
// with codes k, v and the scales a_j, b_j of the blocks that key j lies in.
//
// Products.  An e4m3 number is an fp16 number, so the codes are widened in registers (cvt, two at a time) and both products
// run on the tensor cores from registers (m16n8k16, fp32 sums) with the keys, then the head's elements, on their 16 rows and
// eight rows of q on their columns: a decoding step's few rows waste nothing.  q is divided by a power of two for its row,
// which fp16 holds exactly but for elements below 2^-24 of the row's largest.  A weight is 2^(t_j - m + 8) with
// t_j = s_j log2(e) + log2(b_j) and m the row's largest t at the last rescaling, which follows when it has grown by 2^7:
// at most 2^15, rounded to fp16 (2^-11 of itself, or 2^-32 of the largest), whatever the scales are.  The softmax's sum is
// that of weight / b_j in fp32.  (mma.sync takes e4m3 operands, too, but widens them itself, and adds in separate
// instructions: 1280 a 32 keys and 16 rows against 300 a 32 keys and 8 rows here.)
//
// Work.  Items, shares and parts are those of attention_line.cuh, with items of 32 rows.  Four warps have eight rows each;
// where an item has fewer, warps share them and each takes every second or fourth 32 keys, and their sums are joined through
// shared memory in a fixed order.  A fifth warp feeds a ring of 64-key tiles: codes by TMA, page by page (swizzled, so that the
// fragments' 16-byte reads meet no bank twice), scales by 4-byte asynchronous copies.  Two CTAs an SM with rings of five
// tiles: 24 sequences of up to 16384 keys 90.5 us (floor 74.4), with three CTAs and three tiles, whose registers do not
// suffice, 96, with four and two 123.  Sixteen rows a warp (a key widened once for two products) were slower for any number
// of rows: 8 sequences of 8 tokens over 4000 keys 39.5 us for 29.7.  Heads of 64 leave registers for three CTAs of seven tiles
// (24 such sequences: 83 us, with two 103, with four of five 82, but 8 sequences of 7 tokens 26.5 for 24.6).  L2 fetches what a
// row has: from 64-byte rows with 128 bytes half of what came was not used (83 us for 63); 256 at 128: 123 us for 96.
//
// The orders of the head's elements (for q.k) and of the elements' rows (for w.v) within a product are free; they are chosen
// so that a thread's fragments are neighbouring bytes of the cache.  V's keys are paired by byte permutes before they are
// widened, the weights transposed by movmatrix.
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

constexpr int kWarps = 4;                    // that compute
constexpr int kWarpRows = 8;                 // rows of a warp, the columns of its products
constexpr int kThreads8 = 32 * (kWarps + 1);
constexpr int kUnitKeys = 32;                // of one product
constexpr int kMaxCtas = 480;                // three per SM, and a bound for the workspace
constexpr int kItemCost8 = 4, kMinShare8 = 4;
constexpr float kWeightLog2 = 8.f, kRescaleLog2 = 7.f;   // the largest weight is 2^15 (fp16 ends at 65504)
constexpr float kMaxScale = 1.125899906842624e15f;   // 2^50: V's scales are taken as 2^-50 .. 2^50

// Bits of the device status word (above those of the other operators).
enum : uint32_t {
    kErrAttn8Ring = 1u << 22,
    kErrAttn8Full = 1u << 23,
    kErrAttn8Base = 1u << 24,                // dynamic shared memory not on a 1024-byte boundary
};

struct Attn8Params : LineParams<kWarps * kWarpRows, kItemCost8, kMinShare8> {
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
    CutItem *cuts;                          // [ctas]
    unsigned int *status;
};

// ------------------------------------------------------------------ PTX of this kernel
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// c += A . B, fp16, A [16 x 16] row-major, B [16 x 8] column-major.
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transposes the 8 x 8 matrix of which thread 4 g + t holds elements 2 t, 2 t + 1 of row g.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Two codes as two fp16 numbers: the low or the high half of a word.
__device__ __forceinline__ uint32_t widen_lo(uint32_t w)
{
    const __half2 h = e4m3x2_to_half2(w & 0xffffu);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ uint32_t widen_hi(uint32_t w)
{
    const __half2 h = e4m3x2_to_half2(w >> 16);
    return *reinterpret_cast<const uint32_t *>(&h);
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

template <int WORDS>
__device__ __forceinline__ void load_shared(const uint8_t *at, uint32_t (&w)[WORDS])
{
    if constexpr (WORDS == 4) {
        const uint4 u = *reinterpret_cast<const uint4 *>(at);
        w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
    } else {
        const uint2 u = *reinterpret_cast<const uint2 *>(at);
        w[0] = u.x, w[1] = u.y;
    }
}

// ------------------------------------------------------------------ shared memory
template <int DIM>
struct Attn8Smem {
    static constexpr int kCtas = DIM == 128 ? 2 : 3;                    // an SM
    static constexpr uint32_t kTileBytes = kTileKeys * DIM;             // of K or V; 1024-byte multiples
    static constexpr uint32_t kStages = DIM == 128 ? 5 : 7;
    static constexpr uint32_t kOut = DIM / 4;                           // sums a thread holds
    static constexpr uint32_t kSums = 4;                                // and maxima and sums of weights
    static constexpr uint32_t kScales = kStages * 2 * kTileBytes;       // [stages][K, V][64]
    static constexpr uint32_t kMerge = kScales + kStages * 2 * kTileKeys * 4;       // [warps / 2][kOut + kSums][32]
    static constexpr uint32_t kKeys = kMerge + kWarps / 2 * (kOut + kSums) * 32 * 4;    // [warps][32 keys at hand][4]
    static constexpr uint32_t kBars = kKeys + kWarps * kUnitKeys * 16;  // full, empty [stages]
    static constexpr uint32_t kBytes = kBars + 2 * kStages * 8;
};

// 0xff in the bytes of NaN codes.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w)
{
    return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu);
}

// Whether b is a scale of V; less than 2^-50 counts as that.
__device__ __forceinline__ bool is_value_scale(float b) { return b >= 0.f && b <= kMaxScale; }

// One warp's rows of an item.  Thread 4 g + t has of row g elements [DIM / 4 t, DIM / 4 (t + 1)) of
// q, and of rows 2 t and 2 t + 1 the maximum, the sum of its keys' weights and elements [DIM / 8 g, DIM / 8 (g + 1)) of the
// weighted values: out[e] holds elements 2 e and 2 e + 1 of those, of row 2 t, row 2 t + 1, row 2 t, row 2 t + 1.
template <int DIM>
struct Rows8 {
    uint32_t q[DIM / 16][2];
    float unit[2];                    // power of two that q was divided by
    int hi[2], lo[2];          // keys that a row sees (none: hi < lo)
    float top[2], sum[2];
    float out[DIM / 16][4];
};

template <int DIM, class P>
__device__ __forceinline__ void load_rows(const P &p, const Item &it, int row0, Rows8<DIM> &x)
{
    constexpr int N = DIM / 4;               // elements a thread holds of a row of q
    const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
    const Row row = row_of(p, it, row0 + g);
    alignas(16) __nv_bfloat16 v[N];
    const __nv_bfloat16 *from = p.q + row.token * p.q_ts + row.q_head * p.q_hs + N * t;
#pragma unroll
    for (int i = 0; i < N; i += 8) {
        if (!row.valid) {
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
    const float inverse = power_of_two(-e);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const __half2 h = __floats2half2_rn(__bfloat162float(v[i]) * inverse, __bfloat162float(v[i + 1]) * inverse);
        x.q[i / 4][i / 2 & 1] = *reinterpret_cast<const uint32_t *>(&h);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const int from_lane = 4 * (2 * t + c);
        x.unit[c] = power_of_two(__shfl_sync(0xffffffffu, e, from_lane));
        x.hi[c] = __shfl_sync(0xffffffffu, row.valid ? row.hi : -1, from_lane);
        x.lo[c] = __shfl_sync(0xffffffffu, row.valid ? row.lo : 0, from_lane);
        x.top[c] = -CUDART_INF_F;
        x.sum[c] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < DIM / 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            x.out[i][j] = 0.f;
}

// Key i of this thread's four among 16 of V.
__device__ __forceinline__ int value_key(int i, int t) { return 8 * (i >> 1) + 2 * t + (i & 1); }

// out += V^T . w for the rows of all sets: 16 keys, elements 4 w .. 4 w + 3 of the thread's from its keys' words; b0, b1:
// the weights of keys 2 t, 2 t + 1 and 8 + those of row g.
template <int TILES>
__device__ __forceinline__ void weigh(float (&out)[TILES][4], const uint32_t (&v)[4], int w, const uint32_t (&b0),
                                      const uint32_t (&b1))
{
    const uint32_t lo0 = __byte_perm(v[0], v[1], 0x5140), hi0 = __byte_perm(v[0], v[1], 0x7362);   // elements 0, 1 and 2, 3
    const uint32_t lo1 = __byte_perm(v[2], v[3], 0x5140), hi1 = __byte_perm(v[2], v[3], 0x7362);
    mma_f16(out[2 * w], widen_lo(lo0), widen_hi(lo0), widen_lo(lo1), widen_hi(lo1), b0, b1);
    mma_f16(out[2 * w + 1], widen_lo(hi0), widen_hi(hi0), widen_lo(hi1), widen_hi(hi1), b0, b1);
}

// The 32 keys from key0 on (rows `first` to `first` + 31 of the tile) for one warp's rows.
template <int DIM>
__device__ __forceinline__ void attend(Rows8<DIM> &x, const Seen &seen, int key0, int first, const uint8_t *k_tile,
                                       const uint8_t *v_tile, const float *scales, float4 *mine, float scale_log2)
{
    constexpr int kWords = DIM / 32;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    // Scales of the 32 keys, a key a lane; those that no row sees count nothing.  (One of V that is none makes the key's scores
    // NaN, which the mask still takes out of the rows that do not see it.)
    {
        const int key = key0 + lane;
        const bool known = key >= seen.lo && key < seen.end;
        const float of_v = known ? scales[kTileKeys + first + lane] : 1.f, b = fminf(fmaxf(of_v, 1.f / kMaxScale), kMaxScale);
        const float of_k = known ? scales[first + lane] * scale_log2 : 0.f;
        mine[lane] = make_float4(is_value_scale(of_v) ? of_k : CUDART_NAN_F, __log2f(b), __fdividef(1.f, b), 0.f);
        __syncwarp();
    }
    // Scores: thread 4 g + t has keys g + 8 j of rows 2 t and 2 t + 1.
    float s[2][4] = {};
#pragma unroll
    for (int i = 0; i < DIM / 64; ++i) {
        uint32_t w[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = first + 8 * j + g;
            const uint32_t chunk = DIM == 128 ? (uint32_t)((2 * t + i) ^ (row & 7)) : (uint32_t)(t ^ ((row >> 1) & 3));
            load_shared<4>(k_tile + row * DIM + chunk * 16, w[j]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const uint32_t a0 = widen_lo(w[2 * m][k]), a1 = widen_lo(w[2 * m + 1][k]), a2 = widen_hi(w[2 * m][k]),
                               a3 = widen_hi(w[2 * m + 1][k]);
                mma_f16(s[m], a0, a1, a2, a3, x.q[4 * i + k][0], x.q[4 * i + k][1]);
            }
    }
    const bool edge = key0 < seen.all_lo || key0 + kUnitKeys - 1 > seen.all_hi;
    float inverse[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {            // key g + 8 j
        const float4 a = mine[g + 8 * j];
        inverse[j] = a.z;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float &y = s[j >> 1][2 * (j & 1) + c];
            y = fmaf(y * a.x, x.unit[c], a.y);
            if (edge && (key0 + g + 8 * j > x.hi[c] || key0 + g + 8 * j < x.lo[c]))
                y = -CUDART_INF_F;
        }
    }
    __syncwarp();                            // `mine` may be written again
    // Weights.
    uint32_t weights[4];              // of keys 8 i + 2 t, 8 i + 2 t + 1 and row g
    float top[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        top[c] = fmaxf(fmaxf(s[0][c], s[0][2 + c]), fmaxf(s[1][c], s[1][2 + c]));
#pragma unroll
        for (int o = 4; o < 32; o *= 2)
            top[c] = fmaxf(top[c], __shfl_xor_sync(0xffffffffu, top[c], o));
    }
    if (__any_sync(0xffffffffu, top[0] > x.top[0] + kRescaleLog2 || top[1] > x.top[1] + kRescaleLog2)) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const float now = fmaxf(x.top[c], top[c]);
            const float before = now == x.top[c] ? 1.f : ex2(x.top[c] - now);
            x.top[c] = now;
            x.sum[c] *= before;
#pragma unroll
            for (int e = 0; e < DIM / 16; ++e) {
                x.out[e][c] *= before;
                x.out[e][2 + c] *= before;
            }
        }
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const float shift = x.top[c] == -CUDART_INF_F ? 0.f : x.top[c] - kWeightLog2;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float &y = s[j >> 1][2 * (j & 1) + c];
            y = ex2(y - shift);
            x.sum[c] = fmaf(y, inverse[j], x.sum[c]);
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __half2 h = __floats2half2_rn(s[j >> 1][2 * (j & 1)], s[j >> 1][2 * (j & 1) + 1]);
        weights[j] = transpose_8x8(*reinterpret_cast<const uint32_t *>(&h));
    }
    // Values, 16 keys at a time.
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        uint32_t v[4][kWords], b0, b1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = first + 16 * half + value_key(i, t);
            if constexpr (DIM == 128)
                load_shared<4>(v_tile + row * DIM + ((g ^ (row & 7)) << 4), v[i]);
            else
                load_shared<2>(v_tile + row * DIM + (((g >> 1) ^ ((row >> 1) & 3)) << 4) + (g & 1) * 8, v[i]);
        }
        // A weight of 0 does not silence a NaN: keys that no row sees may hold anything and are cleared.  NaN codes of keys
        // that some rows see and others do not are taken out; how many of them a row sees is a product of its own, of ones.
        if (edge) {
            const int k0 = key0 + 16 * half;
            uint32_t bad = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int key = k0 + value_key(i, t);
                const bool known = key >= seen.lo && key < seen.end;
#pragma unroll
                for (int w = 0; w < kWords; ++w) {
                    v[i][w] = known ? v[i][w] : 0u;
                    bad |= nan_codes(v[i][w]);
                }
            }
            if (__any_sync(0xffffffffu, bad != 0)) {
                uint32_t ones[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int key = k0 + g + 8 * j;
                    ones[j] = key <= x.hi[0] && key >= x.lo[0] ? 0x3c00u : 0u;
                    ones[j] |= key <= x.hi[1] && key >= x.lo[1] ? 0x3c000000u : 0u;
                }
                b0 = transpose_8x8(ones[0]);
                b1 = transpose_8x8(ones[1]);
#pragma unroll
                for (int w = 0; w < kWords; ++w) {
                    uint32_t flags[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t nan = nan_codes(v[i][w]);
                        flags[i] = nan & 0x38383838u;         // 1.0
                        v[i][w] &= ~nan;
                    }
                    float count[2][4] = {};
                    weigh(count, flags, 0, b0, b1);
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            if (count[e][c] > 0.f)
                                x.out[2 * w + e][c] = CUDART_NAN_F;
                }
            }
        }
        b0 = weights[2 * half];
        b1 = weights[2 * half + 1];
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
            const uint32_t word[4] = {v[0][w], v[1][w], v[2][w], v[3][w]};
            weigh(x.out, word, w, b0, b1);
        }
    }
}

// Joins the sums of the warps that share rows: in each step the upper half of them hand theirs over.  Their number is the
// same for the whole CTA; all of its kWarps warps come here.
template <int DIM>
__device__ __forceinline__ void join_warps(Rows8<DIM> &x, float *merge, int sharing, int row_tiles, int warp)
{
    constexpr int kOut = DIM / 4, kAll = kOut + 4;
    const int lane = threadIdx.x & 31;
    const int rt = warp % row_tiles, part = warp / row_tiles;
    for (int half = sharing / 2; half > 0; half /= 2) {
        float *at = merge + ((part & (half - 1)) * row_tiles + rt) * kAll * 32 + lane;
        if (part >= half && part < 2 * half) {
#pragma unroll
            for (int e = 0; e < DIM / 16; ++e)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    at[(e * 4 + c) * 32] = x.out[e][c];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                at[(kOut + c) * 32] = x.top[c];
                at[(kOut + 2 + c) * 32] = x.sum[c];
            }
        }
        ptx::named_barrier_sync(1, 32 * kWarps);
        if (part < half) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float top = at[(kOut + c) * 32];
                const float now = fmaxf(x.top[c], top);
                const float base = now == -CUDART_INF_F ? 0.f : now;
                const float a = ex2(x.top[c] - base), b = ex2(top - base);
                x.top[c] = now;
                x.sum[c] = fmaf(x.sum[c], a, at[(kOut + 2 + c) * 32] * b);
#pragma unroll
                for (int e = 0; e < DIM / 16; ++e)
#pragma unroll
                    for (int h = 0; h < 4; h += 2)
                        x.out[e][h + c] =
                            fmaf(x.out[e][h + c], a, at[(e * 4 + h + c) * 32] * b);
            }
        }
        ptx::named_barrier_sync(1, 32 * kWarps);
    }
}

template <int DIM>
__global__ void __launch_bounds__(kThreads8, Attn8Smem<DIM>::kCtas)
    paged_attention_fp8_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                               const Attn8Params p)
{
    using L = Attn8Smem<DIM>;
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
            // Entries of the table, 32 at a time (a tile has at most 8) and those behind them under way: the loop does not wait
            // for a load (pages of 16: 111 us for 103).  -1 past the sequence's end.
            const int known_pages = (it.kv + p.page_size - 1) >> p.page_shift;
            auto entry = [&](int index) { return index < known_pages ? pages[index] : -1; };
            int window = ((it.first_tile + from) * kTileKeys >> p.page_shift) >> 5;
            int held = entry(32 * window + lane), ahead = entry(32 * window + 32 + lane);
            for (int j = from; j < from + n; ++j, ++i) {
                const int key0 = (it.first_tile + j) * kTileKeys, index = key0 >> p.page_shift;
                if (index >> 5 != window) {
                    ++window;
                    held = ahead;
                    ahead = entry(32 * window + 32 + lane);
                }
                const int box = __shfl_sync(0xffffffffu, held, boxes > 1 ? index + mine : index);
                const uint32_t s = i % L::kStages;
                if (!wait_short(bar_empty + 8 * s, ((i / L::kStages) & 1) ^ 1)) {
                    ok = false;
                    atomicOr(p.status, kErrAttn8Ring);
                }
                ok = __all_sync(0xffffffffu, ok);
                if (!ok)
                    break;
                const int used = min(boxes, max(1, (it.kv - key0 + box_keys - 1) / box_keys));   // pages past the end are not requested
                if (lane == 0)
                    ptx::mbar_arrive_expect_tx(bar_full + 8 * s, 2u * used * box_keys * DIM);
                __syncwarp();
                if (lane < 16 && mine < used)
                    tma_load_4d(sbase + s * 2 * L::kTileBytes + at, map, 0, key0 & (p.page_size - 1), it.head, box, bar_full + 8 * s);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int key = key0 + 32 * h + lane;
                    const int page = __shfl_sync(0xffffffffu, held, key >> p.page_shift);
                    const bool known = page >= 0 && page < p.num_pages;
                    const int64_t pg = known ? page : 0;
                    const int64_t block = (key & (p.page_size - 1)) >> p.block_shift;
                    const uint32_t to = sbase + L::kScales + (s * 2 * kTileKeys + 32 * h + lane) * 4;
                    copy_async_4(to, p.k_scale + pg * p.ks_page + block * p.ks_block + it.head * p.ks_head, known ? 4 : 0);
                    copy_async_4(to + kTileKeys * 4, p.v_scale + pg * p.vs_page + block * p.vs_block + it.head * p.vs_head, known ? 4 : 0);
                }
                copies_arrive(bar_full + 8 * s);
            }
        } while (ok && next_piece(p, c, end));
        // No copy may land after the CTA has ended: normally all were consumed long ago.
        for (uint32_t j = i > L::kStages ? i - L::kStages : 0; j < i; ++j)
            (void)wait_short(bar_full + 8 * (j % L::kStages), (j / L::kStages) & 1);
        return;
    }
    // ---------------------------------------------------------------- rows
    float4 *keys = reinterpret_cast<float4 *>(smem + L::kKeys) + warp * kUnitKeys;
    float *merge = reinterpret_cast<float *>(smem + L::kMerge);
    const int g = lane >> 2, t = lane & 3;
    do {
        const int from = c.from, n = c.to - c.from;
        const int in_item = min(p.kRows, it.q_len * p.group - it.q_tile * p.kRows);
        int row_tiles = 1;
        while (row_tiles * kWarpRows < in_item)
            row_tiles *= 2;
        const int sharing = kWarps / row_tiles, rt = warp % row_tiles, part = warp / row_tiles;
        const bool has_rows = rt * kWarpRows < in_item;
        const Seen seen = seen_by(p, it);
        Rows8<DIM> x;
        load_rows<DIM>(p, it, rt * kWarpRows, x);
        for (int j = 0; j < n; ++j, ++i) {
            const uint32_t s = i % L::kStages;
            if (ok && !wait_short(bar_full + 8 * s, (i / L::kStages) & 1)) {
                ok = false;
                atomicOr(p.status, kErrAttn8Full);
            }
            ok = __all_sync(0xffffffffu, ok);
            const uint8_t *k_tile = smem + s * 2 * L::kTileBytes;
            const float *scales = reinterpret_cast<const float *>(smem + L::kScales) + s * 2 * kTileKeys;
#pragma unroll 1
            for (int h = 0; h < kTileKeys / kUnitKeys; ++h)
                if (ok && has_rows && ((2 * j + h) & (sharing - 1)) == part)
                    attend<DIM>(x, seen, (it.first_tile + from + j) * kTileKeys + kUnitKeys * h, kUnitKeys * h, k_tile,
                                   k_tile + L::kTileBytes, scales, keys, p.scale_log2);
            __syncwarp();
            if (lane == 0)
                ptx::mbar_arrive(bar_empty + 8 * s);
        }
        if (sharing > 1)
            join_warps<DIM>(x, merge, sharing, row_tiles, warp);
        // The item's rows: finished here, or a part for the join.
        const bool whole = n == it.tiles;
        const int64_t slot = 2 * (int64_t)blockIdx.x + (from == 0 ? 1 : 0);
        if (threadIdx.x == 0 && from == 0 && !whole)
            p.cuts[blockIdx.x] = {(it.start + p.kCost + it.tiles - 1) / share - (int)blockIdx.x + 1, it.q0, it.q_len, it.head,
                                  it.q_tile};
        if (part > 0)
            continue;
        constexpr int N = DIM / 8;           // elements a thread holds of a row
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float sum = x.sum[c];
#pragma unroll
            for (int o = 4; o < 32; o *= 2)
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const int r = rt * kWarpRows + 2 * t + c;
            const Row row = row_of(p, it, r);
            if (!row.valid)
                continue;
            if (whole) {
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                alignas(16) __nv_bfloat162 v[N / 2];
#pragma unroll
                for (int e = 0; e < N / 2; ++e)
                    v[e] = __floats2bfloat162_rn(x.out[e][c] * inv, x.out[e][2 + c] * inv);
                __nv_bfloat16 *o = p.out + row.token * p.o_ts + row.q_head * p.o_hs + N * g;
                if (p.out_vec) {
#pragma unroll
                    for (int e = 0; e < N; e += 8)
                        *reinterpret_cast<uint4 *>(o + e) = *reinterpret_cast<const uint4 *>(v + e / 2);
                } else {
#pragma unroll
                    for (int e = 0; e < N / 2; ++e) {
                        o[2 * e] = v[e].x;
                        o[2 * e + 1] = v[e].y;
                    }
                }
                if (p.lse && g == 0)
                    p.lse[(int64_t)row.token * p.heads + row.q_head] =
                        sum == 0.f ? -CUDART_INF_F : (x.top[c] - kWeightLog2 + log2f(sum)) * CUDART_LN2_F;
            } else {
                float *o = p.parts + (slot * p.slot_rows + r) * DIM + N * g;
#pragma unroll
                for (int e = 0; e < N / 2; e += 2)
                    *reinterpret_cast<float4 *>(o + 2 * e) = make_float4(x.out[e][c], x.out[e][2 + c],
                                                                         x.out[e + 1][c], x.out[e + 1][2 + c]);
                if (g == 0)
                    reinterpret_cast<float2 *>(p.parts + 2 * (int64_t)gridDim.x * p.slot_rows * DIM)[slot * p.slot_rows + r] =
                        make_float2(x.top[c], sum);
            }
        }
    } while (next_piece(p, c, end));
}

// Joins the parts of the items that shares cut: CTA c owns the one that begins in share c and ends in a later one.  A
// thread owns four elements of a row.  Part i counts 2^(its maximum - the largest one), and the parts add in the order
// of the keys.
constexpr int kJoinThreads8 = 256, kJoinSplit8 = 4;

template <int DIM>
__global__ void __launch_bounds__(kJoinThreads8) join_parts_fp8_kernel(const Attn8Params p, int ctas)
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
    const CutItem cut = p.cuts[blockIdx.x];
    if (cut.parts == 0)
        return;
    const float2 *ml = reinterpret_cast<const float2 *>(p.parts + 2 * (int64_t)ctas * p.slot_rows * DIM);
    const int rows = min(p.kRows, cut.q_len * p.group - cut.q_tile * p.kRows);
    auto slot = [&](int i) { return 2 * (int64_t)(blockIdx.x + i) + (i == 0 ? 1 : 0); };
    for (int c = threadIdx.x + blockIdx.y * kJoinThreads8; c < rows * (DIM / 4); c += kJoinSplit8 * kJoinThreads8) {
        const int r = c / (DIM / 4), d = c % (DIM / 4) * 4;
        const int row = cut.q_tile * p.kRows + r, t = cut.q0 + row / p.group, h = cut.head * p.group + row % p.group;
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

// ------------------------------------------------------------------ chunks: the cache widened first
// Where sequences bring many rows a head, the keys and values that they see are written out in bf16 once, in pages of 64
// tokens, and the tcgen05 attention of paged_attention.cu runs on those: it does 1.2 PFLOP/s where the registers' products
// reach 0.15; but writing and reading 2 bytes an element takes its time, and a launch more.  A code times a power of two is
// a bf16 number, so K and V keep their scales' powers of two, and the mantissas, in [1, 2), multiply scores and weights (V
// rounded with its scale made the result's error 0.0027 of it where its own rounding is 0.0017).  A tile of the copy has one
// scale where a block is not shorter, else one for each four keys, or for each.
// The rule counts the multiply-adds of all rows with all keys that the table has room for (a key's exponentials as 64 of
// them): us in the registers and widened at 8 sequences x 16 tokens x 4000 keys (of 32 / 8 heads of 128) 40, 58; 8 x 32 x
// 16000 175, 141; 8 x 64 x 8000 250, 135; 2 x 64 x 4000 54, 47; 1 x 300 x 1000 (16 / 8 heads) 30, 35.
constexpr int kWideRows = 96;                // rows a sequence and head bring on average, at least
constexpr double kWideWork = 1.3e10;         // and multiply-adds in all, times four
// The copy has room for as many keys as the table (or, with a window, as its rows can see), in kWideBytes at most: where that
// is not enough for all, sequences and heads take turns, three launches each.  The host only knows how many turns it may take;
// the device gives a turn as many sequences as there is room for, and turns without any do nothing.
constexpr int64_t kWideBytes = (int64_t)1 << 30;
constexpr int kWideKeys = 64;                // tokens of a page of the copy

struct WidenParams {
    const uint8_t *k, *v;
    const float *k_scale, *v_scale;
    int64_t k_page, k_place, k_head, v_page, v_place, v_head, ks_page, ks_block, ks_head, vs_page, vs_block, vs_head;
    int64_t table_stride, num_pages;
    const int32_t *table, *kv_lens, *cu_q;
    __nv_bfloat16 *wide_k, *wide_v;          // [pages][kv_heads][64][dim]
    float *factors;                          // [pages][kv_heads], as in CacheCopy
    int32_t *wide_table;                     // [batch][table_pages]
    int page_shift, block_shift, batch, q_tokens, kv_heads, window, capacity, table_pages;
    int pages;                               // of the copy that a sequence needs at most: the first of sequence b is b * pages,
    int32_t *places, *turns;                 // or, in turns, places[b]; a turn's sequences are turns[turn] .. turns[turn + 1] - 1,
    int32_t *turn_cu_q;                      // and this is cu_q with the others' rows left out
    int turn, room;                          // pages of a turn
    int tokens_a_factor;                     // 64, 4 or 1
    float scale_inverse;                     // of attend_pages
};

// The pages of the copy that a sequence has, from `first` on: those with keys that its rows see, and one where it has new
// tokens but no keys (for the factors, which its rows' masked tile meets).
__device__ __forceinline__ int pages_to_widen(const WidenParams &p, int b, int &first, int &kv)
{
    const int q0 = min(max(p.cu_q[b], 0), p.q_tokens), q_len = min(max(p.cu_q[b + 1], q0), p.q_tokens) - q0;
    kv = min(max(p.kv_lens[b], 0), p.capacity);
    first = p.window > 0 ? max(kv - q_len - p.window + 1, 0) / kWideKeys : 0;
    return q_len == 0 ? 0 : (max(kv, 1) + kWideKeys - 1) / kWideKeys - first;
}

// The turns: in order, as many sequences each as there is room for.
constexpr int kPlanThreads = 256;

__global__ void __launch_bounds__(kPlanThreads) plan_turns_kernel(const WidenParams p, int turns)
{
    __shared__ int pages[kPlanThreads];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    int turn = 0, used = 0;
    for (int b0 = 0; b0 < p.batch; b0 += kPlanThreads) {
        int first, kv;
        const int b = b0 + threadIdx.x;
        pages[threadIdx.x] = b < p.batch ? pages_to_widen(p, b, first, kv) : 0;
        __syncthreads();
        if (threadIdx.x == 0)
            for (int i = 0; i < min(kPlanThreads, p.batch - b0); ++i) {
                if (used + pages[i] > p.room && turn + 1 < turns) {      // (never more turns than the host counted)
                    p.turns[++turn] = b0 + i;
                    used = 0;
                }
                p.places[b0 + i] = used;
                used += pages[i];
            }
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        p.turns[0] = 0;
        while (turn < turns)
            p.turns[++turn] = p.batch;
    }
}

__device__ __forceinline__ void widen_16(uint4 codes, float scale, uint4 *to)
{
    const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
    alignas(16) __nv_bfloat162 out[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 a = __half22float2(e4m3x2_to_half2(w[i] & 0xffffu)), b = __half22float2(e4m3x2_to_half2(w[i] >> 16));
        out[2 * i] = __floats2bfloat162_rn(a.x * scale, a.y * scale);
        out[2 * i + 1] = __floats2bfloat162_rn(b.x * scale, b.y * scale);
    }
    to[0] = reinterpret_cast<const uint4 *>(out)[0];
    to[1] = reinterpret_cast<const uint4 *>(out)[1];
}

// A scale as a power of two, with its sign, times the rest in [1, 2); 0, infinities, NaN and what is below 2^-126 are left whole.
__device__ __forceinline__ float split_scale(float scale, float &rest)
{
    const uint32_t bits = __float_as_uint(scale), exponent = bits & 0x7f800000u;
    const bool normal = exponent != 0 && exponent != 0x7f800000u;
    rest = normal ? __uint_as_float((bits & 0x007fffffu) | 0x3f800000u) : 1.f;
    return normal ? __uint_as_float(bits & 0xff800000u) : scale;
}

// A CTA widens one head of 64 tokens of a sequence at a time, 16 elements a thread and step.
constexpr int kWidenThreads = 256;

template <int DIM>
__global__ void __launch_bounds__(kWidenThreads) widen_kernel(const WidenParams p)
{
    constexpr int kChunks = DIM / 16, kKeysAtOnce = kWidenThreads / kChunks, kSteps = kWideKeys / kKeysAtOnce;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int chunk = threadIdx.x % kChunks, mine = threadIdx.x / kChunks;
    int begin = 0, stop = p.batch;
    if (p.places) {
        begin = p.turns[p.turn];
        stop = p.turns[p.turn + 1];
        for (int i = (int)((blockIdx.y * gridDim.x + blockIdx.x) * kWidenThreads + threadIdx.x); i <= p.batch;
             i += (int)(gridDim.x * gridDim.y * kWidenThreads))
            p.turn_cu_q[i] = p.cu_q[min(max(i, begin), stop)];
    }
    for (int b = begin + (int)blockIdx.y; b < stop; b += (int)gridDim.y) {
        int first, kv;
        const int tasks = pages_to_widen(p, b, first, kv) * p.kv_heads, place = p.places ? p.places[b] : b * p.pages;
        for (int i = (int)blockIdx.x; i < tasks; i += (int)gridDim.x) {
            const int nth = i / p.kv_heads, head = i - nth * p.kv_heads, j = first + nth, wide = place + nth;    // page of the copy
            const int64_t task = (int64_t)wide * p.kv_heads + head;
            if (threadIdx.x == 0 && head == 0)
                p.wide_table[(int64_t)b * p.table_pages + j] = wide;
            const int key0 = j * kWideKeys, end = min(kv, key0 + kWideKeys);
            uint4 k[kSteps], v[kSteps];
            float ks[kSteps], vs[kSteps];
#pragma unroll
            for (int u = 0; u < kSteps; ++u) {
                const int key = key0 + u * kKeysAtOnce + mine;
                k[u] = v[u] = make_uint4(0, 0, 0, 0);
                ks[u] = vs[u] = 1.f;
                if (key >= end)
                    continue;
                const int64_t page = p.table[b * p.table_stride + (key >> p.page_shift)];
                const int place = key & ((1 << p.page_shift) - 1), block = place >> p.block_shift;
                if (page < 0 || page >= p.num_pages)                             // reads as zeros
                    continue;
                k[u] = *reinterpret_cast<const uint4 *>(p.k + page * p.k_page + place * p.k_place + head * p.k_head + 16 * chunk);
                v[u] = *reinterpret_cast<const uint4 *>(p.v + page * p.v_page + place * p.v_place + head * p.v_head + 16 * chunk);
                ks[u] = p.k_scale[page * p.ks_page + block * p.ks_block + head * p.ks_head];
                vs[u] = p.v_scale[page * p.vs_page + block * p.vs_block + head * p.vs_head];
            }
#pragma unroll
            for (int u = 0; u < kSteps; ++u) {
                const int key = u * kKeysAtOnce + mine;
                float k_rest, v_rest;
                const float k_power = split_scale(ks[u], k_rest);
                const float v_power = split_scale(is_value_scale(vs[u]) ? fmaxf(vs[u], 1.f / kMaxScale) : CUDART_NAN_F, v_rest);
                if (chunk == 0 && key % p.tokens_a_factor == 0) {
                    if (p.tokens_a_factor == kWideKeys) {
                        reinterpret_cast<float4 *>(p.factors)[task] = make_float4(k_rest, log2f(v_rest), 1.f / v_rest, 0.f);
                    } else if (p.tokens_a_factor == 4) {
                        float *to = p.factors + 3 * task * (kWideKeys / 4) + key / 4;
                        to[0] = k_rest;
                        to[kWideKeys / 4] = log2f(v_rest) * p.scale_inverse;
                        to[2 * kWideKeys / 4] = 1.f / v_rest;
                    } else {
                        p.factors[2 * task * kWideKeys + key] = k_rest;
                        p.factors[(2 * task + 1) * kWideKeys + key] = v_rest;
                    }
                }
                if (key0 + key >= end)
                    continue;
                const int64_t to = (task * kWideKeys + key) * DIM + 16 * chunk;
                widen_16(k[u], k_power, reinterpret_cast<uint4 *>(p.wide_k + to));
                widen_16(v[u], v_power, reinterpret_cast<uint4 *>(p.wide_v + to));
            }
        }
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
    return (int)std::min<int64_t>(kWarps * kWarpRows, std::max<int64_t>(1, (int64_t)q_tokens * (heads / kv_heads)));
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
               dim == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_64B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? LOWM_OK
               : LOWM_ERR_CUDA;
}

template <int DIM>
lowm_status_t launch_fp8(const CUtensorMap &map_k, const CUtensorMap &map_v, const Attn8Params &p, int sms, void *stream)
{
    static SmemOptIn opt_in;
    if (!opt_in.set(reinterpret_cast<const void *>(paged_attention_fp8_kernel<DIM>), Attn8Smem<DIM>::kBytes))
        return LOWM_ERR_CUDA;
    const int ctas = std::min(Attn8Smem<DIM>::kCtas * sms, kMaxCtas);
    if (p.batch > 0) {
        const lowm_status_t st = launch_pdl(paged_attention_fp8_kernel<DIM>, dim3((unsigned)ctas), dim3(kThreads8),
                                            Attn8Smem<DIM>::kBytes, stream, map_k, map_v, p);
        if (st != LOWM_OK)
            return st;
    }
    return launch_pdl(join_parts_fp8_kernel<DIM>, dim3((unsigned)ctas, kJoinSplit8), dim3(kJoinThreads8), 0, stream, p,
                      ctas);
}

}  // namespace
}  // namespace lowm

namespace lowm {
namespace {

int64_t wide_pages(int page_size, int table_width)
{
    const int64_t capacity = std::min<int64_t>((int64_t)table_width * page_size, kMaxKeys);
    return (capacity + kWideKeys - 1) / kWideKeys;
}

// A call's scratch memory for the copy and how it is used.
struct WidePlan {
    int64_t head_pages;                      // 64 keys of one head each
    int64_t tensor, factors, tables, lists;  // bytes of K or V, of the factors, of the table, of what the turns need
    int heads, turns;                        // at a time; of the sequences
    int64_t pages;                           // of a turn

    int64_t bytes() const { return 2 * tensor + factors + tables + lists; }
};

int64_t sixteens(int64_t bytes) { return (bytes + 15) / 16 * 16; }

// `pages` of the copy a sequence and `table_pages` in its table.  Without room for one head of a sequence: no heads.
WidePlan plan_copy(int batch, int kv_heads, int dim, int64_t pages, int64_t table_pages)
{
    const int64_t one = 2 * kWideKeys * dim * 2 + 2 * kWideKeys * 4;         // bytes of a head's page
    WidePlan plan;
    plan.tables = sixteens(batch * table_pages * 4);
    plan.lists = 3 * sixteens((int64_t)(batch + 1) * 4);                     // places, turns, turn_cu_q
    plan.head_pages = std::min(batch * kv_heads * table_pages, std::max<int64_t>(kWideBytes - plan.tables - plan.lists, 0) / one);
    plan.tensor = plan.head_pages * kWideKeys * dim * 2;
    plan.factors = plan.head_pages * 2 * kWideKeys * 4;
    plan.heads = (int)std::min<int64_t>(kv_heads, plan.head_pages / pages);
    plan.pages = plan.heads ? plan.head_pages / plan.heads : 0;
    const int64_t sequences = plan.pages / pages;                            // in one turn, at least
    plan.turns = plan.heads ? (int)((batch + sequences - 1) / sequences) : 0;
    return plan;
}

// The plan of a call whose rows may see all of the table; with a window they need less of the same memory.
WidePlan plan_whole_copy(int batch, int kv_heads, int dim, int page_size, int table_width)
{
    const int64_t pages = wide_pages(page_size, table_width);
    return plan_copy(batch, kv_heads, dim, pages, pages);
}

// Whether a call widens the cache first.
bool widens(int batch, int q_tokens, int heads, int kv_heads, int dim, int page_size, int table_width)
{
    const double keys = (double)wide_pages(page_size, table_width) * kWideKeys;
    return batch > 0 && (int64_t)q_tokens * (heads / kv_heads) >= (int64_t)kWideRows * batch &&
           4.0 * q_tokens * heads * keys * (dim + 64) >= kWideWork &&
           plan_whole_copy(batch, kv_heads, dim, page_size, table_width).heads > 0;
}

}  // namespace
}  // namespace lowm

extern "C" size_t lowm_paged_attention_fp8_workspace(int batch, int q_tokens, int heads, int kv_heads, int dim, int page_size,
                                                     int table_width)
{
    using namespace lowm;
    if (!attention_fp8_shape_ok(batch, q_tokens, heads, kv_heads, dim) || page_size <= 0 || table_width < 0)
        return 0;
    if (widens(batch, q_tokens, heads, kv_heads, dim, page_size, table_width))
        return (size_t)plan_whole_copy(batch, kv_heads, dim, page_size, table_width).bytes() +
               lowm_paged_attention_workspace(batch, q_tokens, heads, kv_heads, dim);
    return (size_t)2 * kMaxCtas * slot_rows_fp8(q_tokens, heads, kv_heads) * (dim + 2) * sizeof(float) + kMaxCtas * sizeof(CutItem);
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
    if (workspace_bytes < lowm_paged_attention_fp8_workspace(batch, q_tokens, heads, kv_heads, dim, page_size, table_width))
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
    const int64_t q_tiles = (int64_t)q_tokens * group / (kWarps * kWarpRows) + batch;
    if ((double)q_tiles * kv_heads * (double)(capacity / kTileKeys + 2 + kItemCost8) > (double)(INT_MAX - kMinShare8 * kMaxCtas))
        return LOWM_ERR_UNSUPPORTED_SHAPE;
    int sms = 0;
    lowm_status_t st = host_check_device(&sms);
    if (st != LOWM_OK)
        return st;
    auto log2_of = [](int n) {
        int shift = 0;
        while ((1 << shift) < n)
            ++shift;
        return shift;
    };
    if (widens(batch, q_tokens, heads, kv_heads, dim, page_size, table_width)) {
        WidenParams w;
        w.k_page = k_page_stride;
        w.k_place = k_place_stride;
        w.k_head = k_cache_head_stride;
        w.v_page = v_page_stride;
        w.v_place = v_place_stride;
        w.v_head = v_cache_head_stride;
        w.ks_page = ks_page_stride;
        w.ks_block = ks_block_stride;
        w.ks_head = ks_head_stride;
        w.vs_page = vs_page_stride;
        w.vs_block = vs_block_stride;
        w.vs_head = vs_head_stride;
        w.table_stride = page_table_stride;
        w.num_pages = num_pages;
        w.scale_inverse = 1.f / attend_scale_log2(scale);
        w.tokens_a_factor = block >= kWideKeys ? kWideKeys : (block >= 4 ? 4 : 1);
        w.page_shift = log2_of(page_size);
        w.block_shift = log2_of(block);
        w.q_tokens = q_tokens;
        w.window = window < kMaxKeys ? window : 0;
        w.capacity = (int)capacity;
        w.table_pages = (int)wide_pages(page_size, table_width);
        // With a window a sequence's rows see window + q_len - 1 keys at most.
        w.pages = w.window ? (int)std::min<int64_t>(w.table_pages, ((int64_t)w.window + q_tokens) / kWideKeys + 2) : w.table_pages;
        const WidePlan plan = plan_copy(batch, kv_heads, dim, w.pages, w.table_pages);
        uint8_t *at = static_cast<uint8_t *>(workspace);
        auto take = [&](int64_t bytes) {
            uint8_t *here = at;
            at += bytes;
            return here;
        };
        w.wide_k = reinterpret_cast<__nv_bfloat16 *>(take(plan.tensor));
        w.wide_v = reinterpret_cast<__nv_bfloat16 *>(take(plan.tensor));
        w.factors = reinterpret_cast<float *>(take(plan.factors));
        w.wide_table = reinterpret_cast<int32_t *>(take(plan.tables));
        int32_t *lists = reinterpret_cast<int32_t *>(take(plan.lists));
        const int list = (int)(plan.lists / 3 / 4);
        const bool turns = plan.turns > 1;
        w.places = turns ? lists : nullptr;
        w.turns = lists + list;
        w.turn_cu_q = lists + 2 * list;
        w.table = page_table;
        w.kv_lens = kv_lens;
        w.cu_q = cu_q;
        w.batch = batch;
        w.room = (int)plan.pages;
        const int32_t *rows = turns ? w.turn_cu_q : cu_q;
        const CacheCopy copy = {w.factors, w.tokens_a_factor, capacity, cu_q, heads};
        const int64_t head = (int64_t)kWideKeys * dim;
        const int y = std::min(batch, 1024), x = (int)std::min<int64_t>((16 * sms + y - 1) / y, (int64_t)w.pages * plan.heads);
        if (turns && (st = launch_pdl(plan_turns_kernel, dim3(1), dim3(kPlanThreads), 0, stream, w, plan.turns)) != LOWM_OK)
            return st;
        for (int h = 0; h < kv_heads; h += plan.heads)
            for (w.turn = 0; w.turn < plan.turns; ++w.turn) {
                const int some = std::min(plan.heads, kv_heads - h);
                const int64_t q_head = (int64_t)h * group;
                w.k = static_cast<const uint8_t *>(k_cache) + h * k_cache_head_stride;
                w.v = static_cast<const uint8_t *>(v_cache) + h * v_cache_head_stride;
                w.k_scale = k_scale + h * ks_head_stride;
                w.v_scale = v_scale + h * vs_head_stride;
                w.kv_heads = some;
                st = launch_pdl(dim == 64 ? widen_kernel<64> : widen_kernel<128>, dim3((unsigned)x, (unsigned)y), dim3(kWidenThreads), 0,
                                stream, w);
                if (st != LOWM_OK)
                    return st;
                st = attend_pages(static_cast<const __nv_bfloat16 *>(q) + q_head * q_head_stride, q_token_stride, q_head_stride, w.wide_k,
                                  some * head, dim, head, w.wide_v, some * head, dim, head, plan.pages, kWideKeys, w.wide_table,
                                  w.table_pages, w.table_pages, kv_lens, rows,
                                  static_cast<__nv_bfloat16 *>(out) + q_head * out_head_stride, out_token_stride, out_head_stride,
                                  lse ? lse + q_head : nullptr, batch, q_tokens, some * group, some, dim, scale, window, &copy, at,
                                  workspace_bytes - plan.bytes(), stream);
                if (st != LOWM_OK)
                    return st;
            }
        return LOWM_OK;
    }
    unsigned int *status = host_status_word();
    if (!status)
        return LOWM_ERR_CUDA;
    CUtensorMap map_k, map_v;
    if ((st = encode_codes(k_cache, k_page_stride, k_place_stride, k_cache_head_stride, num_pages, page_size, kv_heads, dim,
                           &map_k)) != LOWM_OK ||
        (st = encode_codes(v_cache, v_page_stride, v_place_stride, v_cache_head_stride, num_pages, page_size, kv_heads, dim,
                           &map_v)) != LOWM_OK)
        return st;

    Attn8Params p;
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
    p.page_shift = log2_of(page_size);
    p.block_shift = log2_of(block);
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
    p.cuts = reinterpret_cast<CutItem *>(static_cast<uint8_t *>(workspace) +
                                          (size_t)2 * kMaxCtas * p.slot_rows * (dim + 2) * sizeof(float));
    p.status = status;
    return dim == 64 ? launch_fp8<64>(map_k, map_v, p, sms, stream) : launch_fp8<128>(map_k, map_v, p, sms, stream);
}
