// Device helpers of the 8-bit KV cache: E4M3 codes, block scales, the position
// rotation.  Shared by the cache writer and the tree attention.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "w12_internal.h"

namespace w12d {

__device__ __forceinline__ float bf16_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

// two floats -> two E4M3 codes (round to nearest even; |x| <= 448 here, NaN -> NaN), `lo` in the low byte
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi)
{
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

// A value that is not finite has no code under a finite scale: it is stored as NaN.
__device__ __forceinline__ uint8_t to_e4m3(float x)
{
    if (fabsf(x) == INFINITY) x = __int_as_float(0x7FC00000);
    return (uint8_t)(to_e4m3x2(x, 0.f) & 0xFFu);
}

// two E4M3 codes -> f16x2 (exact: every E4M3 value is an f16 value)
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t codes)
{
    uint32_t d;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"((uint16_t)codes));
    return d;
}

__device__ __forceinline__ float2 f16x2_f32(uint32_t h)
{
    float2 f;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
        : "=f"(f.x), "=f"(f.y)
        : "r"(h));
    return f;
}

__device__ __forceinline__ float e4m3_f32(uint8_t code)
{
    return f16x2_f32(e4m3x2_f16x2(code)).x;
}

// The least power of two s with top <= 448 s, not under 2^-32 (a block of
// zeros, or of values so small that their absolute error no longer matters).
__device__ __forceinline__ float block_scale(float top)
{
    const uint32_t u = __float_as_uint(top);
    const int e = (int)(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);   // 448 = 1.75 * 2^8
    return __uint_as_float((uint32_t)(e < 95 ? 95 : e) << 23);                  // 95: 2^-32
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

}  // namespace w12d
