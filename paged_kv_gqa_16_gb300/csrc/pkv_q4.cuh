// pkv_q4.cuh -- the 4-bit cache's number format, shared by the kernels that
// write, read back and attend over it: e2m1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and
// their negatives), two to a byte, the first in the low half, and one e8m0
// scale for each 32 elements of a head vector.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

#include "pkv_device.cuh"

namespace pkv {

constexpr int kQ4Group = 32;             // elements of a scale
// Exponents of a scale (a byte 127 + e): values up to 6 2^40 are held, and the
// attention's sums over any two scales stay in fp32 range.
constexpr int kQ4MinExp = -40;
constexpr int kQ4MaxExp = 40;

// The scale byte 127 + clamp(ceil(log2(amax / 6)), min, max) of a group whose
// largest magnitude has the bits `amax`; 255 if one is infinite or NaN (as bits
// they are above all others).  6 = 1.5 * 2^2: for amax = 1.f * 2^n the power is
// n - 2, one more if 1.f > 1.5.
__device__ __forceinline__ int q4_scale_byte(unsigned amax)
{
    const int n = (int)(amax >> 23) - 127 - 2 + ((amax & 0x7fffffu) > 0x400000u ? 1 : 0);
    return amax >= 0x7f800000u ? 255 : 127 + min(max(n, kQ4MinExp), kQ4MaxExp);
}

// 2^(127 - byte), what a value is multiplied with before it is rounded to a code.
__device__ __forceinline__ float q4_unscale(int byte)
{
    return __uint_as_float((unsigned)(254 - byte) << 23);
}

// Two floats to two e2m1 codes (the low four bits first), nearest even, saturating.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi)
{
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\t"
        "cvt.u32.u8 %0, b;\n\t}" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Eight values (already scaled) to eight codes.
__device__ __forceinline__ uint32_t e2m1x8(const float (&y)[8])
{
    return e2m1x2(y[0], y[1]) | e2m1x2(y[2], y[3]) << 8 | e2m1x2(y[4], y[5]) << 16 |
           e2m1x2(y[6], y[7]) << 24;
}

// Byte B of w, two codes, to f16x2, exactly.
template <int B>
__device__ __forceinline__ uint32_t f16x2_of_e2m1x2(uint32_t w)
{
    uint32_t r;
    if constexpr (B == 0)
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(r) : "r"(w));
    else if constexpr (B == 1)
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(r) : "r"(w));
    else if constexpr (B == 2)
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(r) : "r"(w));
    else
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, d;\n\t}" : "=r"(r) : "r"(w));
    return r;
}

} // namespace pkv
