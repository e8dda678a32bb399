// int4.cuh -- the 4-bit format of the key-value cache.
//
// A token's head is cut into groups of 32 values that share a scale s, an e5m2 number
// (5 bits of exponent, 2 of mantissa: its byte is the upper byte of an fp16, so one byte
// permutation turns it into one).  value = (code - 8) s, codes 1 .. 15 (0 reads as -8), two
// to a byte, the even value in the low bits.  s is the smallest e5m2 number of at least 2^-14
// with amax <= 7.5 s: the largest value then rounds to 7 like any other, within half a step
// (with amax <= 7 s steps are a fourteenth wider for nothing).  A group that holds a NaN has
// s = NaN and reads as NaN; infinities are stored as 7 s.
// Groups of 32 and not whole heads, because keys' channels differ in size: where they do so by
// e^(0.7 n), n normal, the stored keys are 16 dB over their rounding, 13 dB with a scale a head.
//
// (code - 8) s has at most 3 + 3 significant bits: exact in fp16 and in bf16.
#pragma once

#include <cstdint>

#include "common.cuh"
#include "ptx.cuh"

namespace lowbit {

constexpr int kGroup4 = 32;                      // values that share a scale
constexpr float kScaleMin = 6.103515625e-5f, kScaleMax = 57344.f;

// The scale for a largest finite magnitude.  The product only guesses; the comparison decides
// (7.5 times an e5m2 number is exact).
__device__ __forceinline__ float scale4(float amax) {
    float s = __uint_as_float(__float_as_uint(amax * (1.f / 7.5f)) & 0xFFE00000u);
    if (7.5f * s < amax) s = __uint_as_float(__float_as_uint(s) + 0x00200000u);
    return fminf(fmaxf(s, kScaleMin), kScaleMax);
}

// The byte of a scale (a normal e5m2 number).
__device__ __forceinline__ uint32_t scale4_byte(float s) { return (__float_as_uint(s) >> 21) - ((127u - 15u) << 2); }

// The codes of eight values, packed: round_half_even(x / s) + 8, within 1 .. 15.  The quotient is
// corrected by its remainder (1 / s rounded alone would put ties next to where they are).
__device__ __forceinline__ uint32_t codes4(const float (&x)[8], float s) {
    const float inv = __frcp_rn(s), top = 7.f * s;
    const float2 s2 = make_float2(-s, -s), inv2 = make_float2(inv, inv), to_int = make_float2(12582920.f, 12582920.f);
    uint32_t w = 0u;
#pragma unroll
    for (int i = 6; i >= 0; i -= 2) {
        const float2 a = make_float2(fminf(fmaxf(x[i], -top), top), fminf(fmaxf(x[i + 1], -top), top)), t = ptx::fmul2(a, inv2);
        float2 q;
        ptx::ffma2(q, t, s2, a);
        ptx::ffma2(q, q, inv2, t);
        q = ptx::fadd2(q, to_int);                                        // 1.5 * 2^23 + 8: rounds to whole numbers
        w = w * 256u + (__float_as_uint(q.y) & 15u) * 16u + (__float_as_uint(q.x) & 15u);
    }
    return w;
}

}  // namespace lowbit
