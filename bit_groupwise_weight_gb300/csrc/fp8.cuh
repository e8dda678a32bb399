// fp8.cuh -- conversions between e4m3 codes, fp16 and fp32 (one instruction each
// way on sm_103a), for the kernels over the 8-bit key-value cache.
//
// A cached value is code * 2^e: code an e4m3 number (4 significant bits, largest
// 448, subnormals down to 2^-9, no infinity, NaN 0x7F), e one exponent for each
// page of tokens and head.  With the scale a power of two, scaling is exact, and
// a page whose exponent has to grow moves its codes' exponents: only codes that
// become subnormal are rounded again.
#pragma once

#include <cstdint>

namespace lowbit {

constexpr int kExpMin = -64, kExpMax = 64;   // limits of a page's exponent

// The smallest e in [kExpMin, kExpMax] with amax <= 448 * 2^e, amax >= 0 finite:
// 448 = 1.75 * 2^8, so e is amax's binary exponent - 8, and one more past 1.75.
__device__ __forceinline__ int page_exponent(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return min(max(e, kExpMin), kExpMax);
}

// 2^e for e in [-126, 127].
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Four fp32 -> four e4m3 codes, nearest even, values past 448 stored as 448, NaN as 0x7F.
__device__ __forceinline__ uint32_t f32x4_to_e4m3x4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
        "mov.b32 %0, {l, h};\n\t}"
        : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

// Four e4m3 codes -> two fp16 pairs (exact).
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t v, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(v));
}

// Two fp32 -> an fp16 pair, nearest even.
__device__ __forceinline__ uint32_t f32x2_to_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t f32x2_to_bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

}  // namespace lowbit
