// Host helpers shared by the decoder-layer operators (residual_norm.cu,
// rope_append.cu, paged_attention.cu, moe.cu): device check, status word, the
// driver's tensor-map encoder and a launch with programmatic dependent launch.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

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
