// append.cuh -- what the writes into the 8-bit cache (cache.cu) and into the 4-bit cache
// (cache4.cu) share: rows of heads in vectors of 8, their norms, and the angles.
#pragma once

#include "common.cuh"
#include "ptx.cuh"

namespace lowbit {
namespace append {

// How rows are read and rotated: any layout value by value, or in 16-byte vectors
// with the pairs' halves, or neighbours, in whole vectors.
enum Form { kAny, kHalves, kNeighbours };

__device__ __forceinline__ void widen(const uint4 &v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
    }
}

// Eight consecutive bf16 values, as they are.
template <Form FORM>
__device__ __forceinline__ uint4 load8(const uint16_t *p) {
    if constexpr (FORM != kAny) return *reinterpret_cast<const uint4 *>(p);
    return make_uint4(p[0] | (uint32_t)p[1] << 16, p[2] | (uint32_t)p[3] << 16, p[4] | (uint32_t)p[5] << 16,
                      p[6] | (uint32_t)p[7] << 16);
}

// 1 / sqrt(v), root and reciprocal rounded to nearest each.  Within the range that rows have in earnest by Newton
// steps from the approximate inverse root, their remainders exact in a fused operation (P. Markstein, "Computation
// of elementary functions on the IBM RISC System/6000 processor", 1990), one for the root and two for the reciprocal: some
// fifteen instructions, where the two functions take some sixty.  A reciprocal step does not round right for a mantissa of ones,
// which the root of v next below a power of 4 has.  (Compared with the two functions for every float that is not negative;
// with one step for the reciprocal 400 of 1.7e9 were the float beside.)
__device__ __forceinline__ float inverse_root(float v) {
    const uint32_t u = __float_as_uint(v);
    if (u - 0x0D800000u >= 0x64000000u || (u & 0xFFFFFEu) == 0x7FFFFEu) return __frcp_rn(__fsqrt_rn(v));     // 2^-100 .. 2^100
    const float y = rsqrtf(v), s0 = v * y, s = fmaf(fmaf(-s0, s0, v), 0.5f * y, s0), r = fmaf(fmaf(-s, y, 1.f), y, y);
    return fmaf(fmaf(-s, r, 1.f), r, r);
}

// 1 / sqrt(mean of squares + eps) of a row held by LANES lanes, 8 values each.  Every operation
// is rounded by itself, the squares are added in pairs: the codes of a key that is not turned are then
// the same in any implementation, also next to a border between two (cosines and sines are not
// rounded to nearest).  The lanes of `mask` call, whole rows of them.
template <int LANES>
__device__ __forceinline__ float row_norm(const float (&x)[8], float eps, uint32_t mask) {
    float s[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float2 a = make_float2(x[i], x[i + 1]), b = ptx::fmul2(a, a);
        s[i] = b.x, s[i + 1] = b.y;
    }
    float t = __fadd_rn(__fadd_rn(__fadd_rn(s[0], s[1]), __fadd_rn(s[2], s[3])),
                        __fadd_rn(__fadd_rn(s[4], s[5]), __fadd_rn(s[6], s[7])));
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) t = __fadd_rn(t, __shfl_xor_sync(mask, t, o));
    return inverse_root(__fadd_rn(__fmul_rn(t, 1.f / (8 * LANES)), eps));
}

// x times `norm`, times the weights from wt (16-byte aligned) on.
__device__ __forceinline__ void weigh(float (&x)[8], float norm, const float *wt) {
    const float4 a = *reinterpret_cast<const float4 *>(wt), b = *reinterpret_cast<const float4 *>(wt + 4);
    const float w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float2 y = ptx::fmul2(ptx::fmul2(make_float2(x[i], x[i + 1]), make_float2(norm, norm)), make_float2(w[i], w[i + 1]));
        x[i] = y.x, x[i + 1] = y.y;
    }
}

// Norm weight d of q or k.
__device__ __forceinline__ float norm_weight(const void *w, int dtype, int d) {
    if (dtype == LOWBIT_DTYPE_F32) return static_cast<const float *>(w)[d];
    const uint16_t h = static_cast<const uint16_t *>(w)[d];
    return dtype == LOWBIT_DTYPE_BF16 ? __uint_as_float((uint32_t)h << 16) : __half2float(__ushort_as_half(h));
}

// Where token `token` at place `pos` of its sequence stands for pair j's rotation.
__device__ __forceinline__ int position_of(const AppendArgs &p, int64_t token, int pos, int j) {
    if (p.positions == nullptr) return pos;
    const int axis = p.axis == nullptr ? 0 : min((int)p.axis[j], p.axes - 1);
    return p.positions[token * p.positions_token + axis];
}

// Cosine and sine of pair j at a position, times the factor.
__device__ __forceinline__ void turn_of(const AppendArgs &p, int position, int j, float &cs, float &sn) {
    // As a signed fraction of a turn, the nearest way round.
    const int32_t ph = (int32_t)(((uint64_t)(int64_t)position * (uint64_t)p.turns[j]) >> 32);
    float c, s;                          // (cs and sn may be places in shared memory)
    sincosf((float)ph * 1.4629180792671596e-9f, &s, &c);          // 2 pi / 2^32
    cs = __fmul_rn(c, p.factor);
    sn = __fmul_rn(s, p.factor);
}

}  // namespace append
}  // namespace lowbit
