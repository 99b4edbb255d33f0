// Host helpers shared by the decoder-layer operators (residual_norm.cu,
// rope_append.cu, paged_attention.cu, moe.cu): device check, status word, the
// driver's tensor-map encoder and a launch with programmatic dependent launch.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstring>

#include "../../include/lowm_layer.h"

namespace lowm {

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Defined in lowm_gemm.cu, which caches what they look up.
lowm_status_t host_check_device(int *sms);   // LOWM_OK on sm_103; the SM count
unsigned int *host_status_word();            // device address of the status word, or nullptr
EncodeTiledFn host_encode_fn();              // cuTensorMapEncodeTiled (for any host thread), or nullptr

// What attend_pages takes scores to exponents of 2 with; their sign is in Q.  Never 0, so that a masked score (-inf) stays one.
inline float attend_scale_log2(float scale)
{
    return std::max((scale < 0.f ? -scale : scale) * 1.44269504088896340736f, 1e-30f);
}

// A cache that was copied to pages of 64 tokens with factors in [1, 2) of a key's scores (f) and of its value (v), for some of
// a call's sequences (the others have no rows in the cu_q that goes with it) and heads.
struct CacheCopy {
    // fp32 and 16-byte aligned, [num_pages][kv_heads] of: f, log2(v), 1 / v and an unused number for the page
    // (tokens_a_factor 64); 16 f, 16 log2(v) / attend_scale_log2 and 16 1 / v, for four keys each (4); 64 f and 64 v (1).  The
    // first page of a sequence with new tokens is read even where it has no keys: its factors are finite.
    const float *factors;
    int tokens_a_factor;
    int64_t capacity;                        // keys a sequence can have
    const int32_t *cu_q;                     // the whole call's: rows of none of its sequences become zeros
    int heads;                               // the whole call's
};

// Defined in paged_attention.cu: lowm_paged_attention, of a copy when that is not NULL.
lowm_status_t attend_pages(const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *k_cache, int64_t k_page_stride,
                           int64_t k_place_stride, int64_t k_cache_head_stride, const void *v_cache, int64_t v_page_stride,
                           int64_t v_place_stride, int64_t v_cache_head_stride, int64_t num_pages, int page_size,
                           const int32_t *page_table, int64_t page_table_stride, int table_width, const int32_t *kv_lens,
                           const int32_t *cu_q, void *out, int64_t out_token_stride, int64_t out_head_stride, float *lse, int batch,
                           int q_tokens, int heads, int kv_heads, int dim, float scale, int window, const CacheCopy *copy,
                           void *workspace, size_t workspace_bytes, void *stream);

inline bool is_aligned(const void *p, uintptr_t bytes)
{
    return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

// The opt-in of one kernel to more than 48 KiB of dynamic shared memory, made
// once per device.
class SmemOptIn {
public:
    bool set(const void *kernel, int bytes)
    {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
            return false;
        if (done_[dev].load(std::memory_order_acquire))
            return true;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
            return false;
        done_[dev].store(true, std::memory_order_release);
        return true;
    }

private:
    std::atomic<bool> done_[64] = {};
};

// One launch on `stream`, allowed to start while its predecessor drains.  Every
// kernel here waits (griddepcontrol.wait) before it touches what another may
// write, and lets its successor start only after that wait: what a kernel does
// before its own wait then sees everything that came before its predecessor,
// as the GEMM's launch flags for A and W promise.
template <typename... KArgs, typename... Args>
lowm_status_t launch_pdl(void (*fn)(KArgs...), dim3 grid, dim3 block, size_t smem, void *stream, Args... args)
{
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, static_cast<KArgs>(args)...) == cudaSuccess ? LOWM_OK : LOWM_ERR_CUDA;
}

}  // namespace lowm
