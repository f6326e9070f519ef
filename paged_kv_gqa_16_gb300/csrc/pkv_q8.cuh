// pkv_q8.cuh -- the 8-bit cache's number format, shared by the kernels that
// write, read back and attend over it.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

#include "pkv_device.cuh"

namespace pkv {

// Exponents of a head vector's scale (a byte 127 + e): values up to 448 2^40
// are held, and the attention's sums over any two scales stay in fp32 range.
constexpr int kQ8MinExp = -40;
constexpr int kQ8MaxExp = 40;

// The scale byte 127 + clamp(ceil(log2(amax / 448)), min, max).  448 = 1.75 *
// 2^8: for amax = 1.f * 2^n the power is n - 8, one more if 1.f > 1.75.
__device__ __forceinline__ int q8_scale_byte(float amax)
{
    const unsigned u = __float_as_uint(amax);
    const int n = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return 127 + min(max(n, kQ8MinExp), kQ8MaxExp);
}

// Two floats to two e4m3 codes (low byte first), nearest even, saturating.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Eight values times f (> 0) to codes at scale byte sb; with `inf`, infinite
// values become NaN (they would saturate).
__device__ __forceinline__ uint2 q8_encode8(const float (&x)[8], float f, int sb, bool inf)
{
    const float by = f * __uint_as_float((unsigned)(254 - sb) << 23);   // f 2^(127 - sb)
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        y[j] = x[j] * by;
    if (inf) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (fabsf(y[j]) == INFINITY)
                y[j] = __uint_as_float(0x7fffffffu);
    }
    uint2 r;
    r.x = e4m3x2(y[0], y[1]) | (e4m3x2(y[2], y[3]) << 16);
    r.y = e4m3x2(y[4], y[5]) | (e4m3x2(y[6], y[7]) << 16);
    return r;
}

// Two e4m3 codes (the low 16 bits of w) to f16x2, exactly.
__device__ __forceinline__ uint32_t f16x2_of_e4m3x2(uint32_t w)
{
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(w));
    return r;
}

// The same for the high 16 bits.
__device__ __forceinline__ uint32_t f16x2_of_e4m3x2_hi(uint32_t w)
{
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(w));
    return r;
}

// 2^(byte - 127) as fp32, for bytes 1 to 254.
__device__ __forceinline__ float q8_scale(unsigned byte)
{
    return __uint_as_float(byte << 23);
}

} // namespace pkv
