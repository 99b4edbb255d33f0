// Device helpers of the 8-bit operators: e4m3 codes and their power-of-two scales.
//
// A scale is the smallest power of two that brings the largest magnitude of
// its block to 448, e4m3's largest value, or less.  Dividing by it and, when a
// block's scale grows, moving older codes to the new one change exponents only:
// nothing is rounded but what falls below e4m3's smallest step, and the scale is
// the same number in any precision.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

namespace lowm {

constexpr int kMinScaleExponent = -100, kMaxScaleExponent = 120;   // normal floats, and so are their inverses

// The exponent of the scale of a block whose largest finite magnitude is amax.
__device__ __forceinline__ int scale_exponent(float amax)
{
    const uint32_t bits = __float_as_uint(amax);
    const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u);   // 448 = 1.75 * 2^8
    return min(max(e, kMinScaleExponent), kMaxScaleExponent);
}

__device__ __forceinline__ float power_of_two(int e)
{
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// The magnitude that counts for a scale: 0 for what is not finite.
__device__ __forceinline__ float finite_magnitude(float x)
{
    const float a = fabsf(x);
    return a < __uint_as_float(0x7f800000u) ? a : 0.f;
}

// e4m3 has no infinities: what is not finite becomes NaN, not the largest value.
__device__ __forceinline__ float nan_unless_finite(float x)
{
    return fabsf(x) < __uint_as_float(0x7f800000u) ? x : __uint_as_float(0x7fffffffu);
}

// Two values rounded to nearest even, the first one in the low byte.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Exact: e4m3 is a subset of fp16.
__device__ __forceinline__ __half2 e4m3x2_to_half2(uint32_t x)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)x));
    return *reinterpret_cast<const __half2 *>(&r);
}

}  // namespace lowm
