// attention.cuh -- shared by the attention kernels over a paged cache of 8 or 4 bits
// (attention_few.cuh: few query rows a sequence; attention_prompt.cu: many).
#pragma once

#include "common.cuh"
#include "fp8.cuh"
#include "ptx.cuh"

namespace lowbit {

// Grid of the prompt kernel: row tiles over all sequences (an upper bound when the
// sequences are ragged), splits of the keys, and where its workspace begins (floats).
struct PromptGrid {
    int tiles, splits;
    int64_t workspace;
};
PromptGrid prompt_grid(int64_t T, int B, int max_q, bool uniform, int Hq, int Hk, int64_t max_len);
size_t prompt_workspace_bytes(const PromptGrid &g, int Hk, int D);
cudaError_t launch_prompt(const AttentionArgs &p, const PromptGrid &g, cudaStream_t stream);
uint32_t prompt_timeouts(bool reset);
// Few query rows a sequence over a 4-bit cache (attention4.cu).
cudaError_t launch_attention4(const AttentionArgs &p, cudaStream_t stream);
uint32_t attention4_timeouts(bool reset);
size_t attention4_workspace_bytes(int max_q, int G, int D);

namespace attn {

constexpr int kSms = 152;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void sts_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// A row's weights are 2^(s + ve - m), as fp16 for the product: m is set 2^kStart below the largest
// s + ve when that has passed m + kPeak, so that they lie below 2^kPeak (fp16 holds less than
// 2^16), the largest at 2^kStart at least.  fp16 then holds them to 2^-11 of themselves down to
// 2^-21 of the largest, and to 2^-32 of it below.  (A kStart of 11 or 13 holds 4 or 6 bits more, but
// m moves more often: a prompt of 4096 tokens takes 140 or 150 us instead of 125, 8 sequences of 5
// guessed tokens 19.2 or 19.9 instead of 18.7.)
constexpr float kStart = 7.f, kPeak = 15.f;
// Scores less m by one fused operation are differences of the exact products, m comes from a rounded one.  Up to this
// size of m the two are half a unit apart at most, past it any number of them, and what is below kPeak in one
// way overflows, or counts for nothing, in the other: there products are rounded first.  (kPeak is compared with the
// difference as the exponential takes it: m + kPeak may be rounded to 16 more than m.)
constexpr float kFar = 4194304.f;
// The weights' sum l does not have ve in it, and what counts in it may count for nothing in the
// product (a page of zeros).  For ve below kDeep, where the weight may be under fp32's range, it
// takes 2^(s - m) by itself; and l is rescaled in two halves of the exponent, which may be past -126.
constexpr float kDeep = -38.f;
struct Rescale {
    float half;
    __device__ __forceinline__ explicit Rescale(float exponent) : half(ex2(0.5f * exponent)) {}
    __device__ __forceinline__ float of_o() const { return half * half; }
    __device__ __forceinline__ float of_l(float l) const { return l * half * half; }
};

// Where a sequence's new tokens lie, and its length with them.  Of tokens past max_q, which are
// left out, neither n nor len counts any: the first one stands at len - n either way.
struct Span { int start, n, len; };

__device__ __forceinline__ Span span(const AttentionArgs &p, int b) {
    Span s;
    int over = 0;
    if (p.cu_q == nullptr) {
        s.n = p.n;
        s.start = b * s.n;
    } else {
        s.start = min(max(p.cu_q[b], 0), p.T);
        const int all = max(min(p.cu_q[b + 1], p.T) - s.start, 0);
        s.n = min(all, p.max_q);
        over = all - s.n;
    }
    s.len = min(max(p.lens[b], 0), p.width * p.P) - over;     // below 0: all before position 0
    return s;
}

// Power of two that brings a row of q whose largest finite magnitude is amax into
// [2^10, 2^11): bf16's 8 bits are then exact in fp16 down to 2^-28 of it (2^-17, fp16's last
// bit being 2^-24), and what is smaller is off by 2^-35 of it at most.
__device__ __forceinline__ int query_shift(float amax) { return min(10 + 127 - (int)(__float_as_uint(amax) >> 23), 100); }

}  // namespace attn
}  // namespace lowbit
