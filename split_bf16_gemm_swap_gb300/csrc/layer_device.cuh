// Device helpers shared by the decoder-layer kernels that run on the tensor
// cores (paged_attention.cu, moe.cu).
#pragma once

#include "lowm_kernel.cuh"

namespace lowm {

// A value that all lanes of a warp hold, so that the compiler knows it, too.
template <typename T>
__device__ __forceinline__ T uniform(T x)
{
    return __shfl_sync(0xffffffffu, x, 0);
}

// One try_wait that lets the hardware suspend the thread for up to `ns` until the phase completes.
__device__ __forceinline__ bool mbar_try_wait_for(uint32_t bar, uint32_t parity, uint32_t ns)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(ns)
        : "memory");
    return ok != 0;
}

// The rest of wait_short: not inlined, so that the many waits of a kernel share it.
static __device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity)
{
    const uint64_t t0 = ptx::globaltimer();
    do {
        for (int i = 0; i < 64; ++i)
            if (mbar_try_wait_for(bar, parity, 100000u))
                return true;
    } while (ptx::globaltimer() - t0 < kDefaultTimeoutNs);
    return false;
}

// A bounded wait (about 2 s) for kernels that meet many waits.
__device__ __forceinline__ bool wait_short(uint32_t bar, uint32_t parity)
{
    constexpr uint32_t kSuspendNs = 10000000u;
    if (mbar_try_wait_for(bar, parity, kSuspendNs))
        return true;
    return wait_slow(bar, parity);
}

}  // namespace lowm
