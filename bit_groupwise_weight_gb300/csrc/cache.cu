// cache.cu -- rotary positions and the write into the 8-bit paged cache, in one
// kernel (lowbit_kv_append).
//
// Mathematics.  Token i of a sequence's n new tokens stands at position
// pos = len - n + i.  Pair j of its rotated part turns by the angle
//     2 pi * frac(pos * turns_j / 2^64),
// turns_j being the pair's frequency in turns per position times 2^64: the
// 64-bit product wraps exactly at whole turns, so the angle of position 2^30 is
// as good as that of position 1 (an fp32 product would be off by radians).
//     (a, b) -> ((a cos - b sin), (a sin + b cos)),  cos and sin times `factor`.
// Keys (rotated) and values then go into the sequence's pages as e4m3 codes with
// one exponent e per page and head (fp8.cuh).  A page whose first slot is among
// the new tokens starts afresh; one that holds older tokens keeps the larger of
// its exponent and the new tokens', and where that grows the older codes are
// moved to it.  Rotation and amax are in fp32, rounded once to the output.
//
// Work split.  One CTA takes one page of one sequence and one key-value head:
// the new tokens of that page, their K and V rows of the head and the q rows of
// its group.  So a page's amax, its exponent and its older codes belong to one
// CTA (no atomics, no second launch), and the cos/sin table of the page's tokens
// is computed once for all of its rows.
//
// Bound: HBM (T D (4 Hq + 6 Hk) bytes) for prompts, launch latency for decode.
#include <algorithm>

#include "common.cuh"
#include "fp8.cuh"
#include "ptx.cuh"

namespace lowbit {
namespace {

constexpr int kChunk = 64;               // tokens of a page handled at a time
constexpr int kVecs = 4;                 // 8-value vectors a thread holds of a chunk's rows
constexpr int kBigThreads = 256;         // kChunk * 128 / 8 / kVecs
constexpr int kSmallThreads = 64;

struct Seq { int start, n, len; };

__device__ __forceinline__ int floor_div(int a, int b) {
    const int q = a / b;
    return q - (a - q * b < 0);
}

// Where a sequence's new tokens lie in q, k and v, and its length with them.
__device__ __forceinline__ Seq sequence(const AppendArgs &p, int b) {
    Seq s;
    if (p.cu_q == nullptr) {
        s.n = p.T / p.B;
        s.start = b * s.n;
    } else {
        s.start = min(max(p.cu_q[b], 0), p.T);
        s.n = min(max(min(p.cu_q[b + 1], p.T) - s.start, 0), p.max_q);
    }
    s.len = max(p.lens[b], 0);
    return s;
}

// Eight consecutive bf16 values as fp32.
__device__ __forceinline__ void load8(const uint16_t *p, bool vec, float (&x)[8]) {
    if (vec) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf16_lo(w[i]);
            x[2 * i + 1] = bf16_hi(w[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __uint_as_float((uint32_t)p[i] << 16);
    }
}

__device__ __forceinline__ void store8(uint16_t *p, bool vec, const float (&x)[8]) {
    if (vec) {
        uint4 v;
        v.x = f32x2_to_bf16x2(x[0], x[1]);
        v.y = f32x2_to_bf16x2(x[2], x[3]);
        v.z = f32x2_to_bf16x2(x[4], x[5]);
        v.w = f32x2_to_bf16x2(x[6], x[7]);
        *reinterpret_cast<uint4 *>(p) = v;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = float_to_bf16_bits(x[i]);
    }
}

// Values d0 .. d0+7 of a row, rotated.  cs: the token's (cos, sin) per pair.
__device__ __forceinline__ void load_rotated(const AppendArgs &p, const uint16_t *row, int d0, bool vec,
                                             const float2 *cs, float (&x)[8]) {
    load8(row + d0, vec, x);
    if (d0 >= p.R) return;
    if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; i += 2)
            if (d0 + i < p.R) {
                const float2 c = cs[(d0 + i) >> 1];
                const float a = x[i], b = x[i + 1];
                x[i] = __fsub_rn(__fmul_rn(a, c.x), __fmul_rn(b, c.y));
                x[i + 1] = __fadd_rn(__fmul_rn(a, c.y), __fmul_rn(b, c.x));
            }
        return;
    }
    const int half = p.R >> 1;
    if (vec && (half & 7) == 0) {                 // the partners are a vector too
        const bool upper = d0 >= half;
        const int j0 = upper ? d0 - half : d0;
        float y[8];
        load8(row + (upper ? j0 : d0 + half), true, y);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 c = cs[j0 + i];
            const float t = __fmul_rn(x[i], c.x), u = __fmul_rn(y[i], c.y);
            x[i] = upper ? __fadd_rn(u, t) : __fsub_rn(t, u);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int d = d0 + i;
        if (d < p.R) {
            const bool upper = d >= half;
            const int j = upper ? d - half : d;
            const float y = __uint_as_float((uint32_t)row[upper ? j : d + half] << 16);
            const float2 c = cs[j];
            const float t = __fmul_rn(x[i], c.x), u = __fmul_rn(y, c.y);
            x[i] = upper ? __fadd_rn(u, t) : __fsub_rn(t, u);
        }
    }
}

__device__ __forceinline__ float finite_max(float m, const float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float a = fabsf(x[i]);
        m = a <= 3.402823466e38f ? fmaxf(m, a) : m;    // false for infinities and NaN
    }
    return m;
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS) kv_append_kernel(const AppendArgs p) {
    extern __shared__ float2 table[];                 // [kChunk][R / 2] (cos, sin)
    __shared__ float red[2][THREADS / 32];
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();

    // This CTA's sequence and page.  With ragged sequences, sequence b owns the
    // CTAs from cu_q[b] / P + 2 b on: as many as the pages its tokens can touch,
    // found by bisection without any table of page counts.
    const int P = p.P;
    int b, j;
    if (p.cu_q == nullptr) {
        b = blockIdx.x / p.units;
        j = blockIdx.x - b * p.units;
    } else {
        int lo = 0, hi = p.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (min(max(p.cu_q[mid], 0), p.T) / P + 2 * mid <= (int)blockIdx.x) lo = mid;
            else hi = mid - 1;
        }
        b = lo;
        j = (int)blockIdx.x - (min(max(p.cu_q[b], 0), p.T) / P + 2 * b);
    }
    const Seq s = sequence(p, b);
    if (s.n == 0) return;
    const int first = s.len - s.n;                    // position of the first new token
    const int slot = floor_div(first, P) + j;         // page of the sequence
    const int lo = max(slot * P, first), hi = min(slot * P + P, s.len);
    if (lo >= hi) return;                             // also what negative j gives: nothing
    const int head = blockIdx.y, G = p.Hq / p.Hk;
    const bool stored = slot >= 0 && slot < p.width;
    const int page = stored ? p.page_table[(int64_t)b * p.table_stride + slot] : -1;
    const bool write = page >= 0 && page < p.pages;
    const int older = lo - slot * P;                  // slots that hold older tokens

    const int vpr = p.D >> 3;                         // vectors of a row: 8 or 16
    const int vshift = vpr == 16 ? 4 : 3;
    const int tid = threadIdx.x;
    const int half = p.R >> 1;
    int8_t *exps[2] = {p.k_exp + (int64_t)page * p.Hk + head, p.v_exp + (int64_t)page * p.Hk + head};
    const int old_k = write && older ? *exps[0] : kExpMin, old_v = write && older ? *exps[1] : kExpMin;
    const int chunks = (hi - lo + kChunk - 1) / kChunk;

    float m[2] = {0.f, 0.f};                          // amax of K and V
    float held[2][kVecs][8];                          // the chunk's K and V values
    auto rows = [&](int c, bool want_max) {           // load chunk c: the table, K, V (and q on the way)
        const int t0 = lo + c * kChunk, nt = min(kChunk, hi - t0);
        __syncthreads();
        for (int i = tid; i < nt * half; i += THREADS) {
            const int t = i / half, jj = i - t * half;
            // As a signed fraction of a turn, the nearest way round.
            const int32_t ph = (int32_t)(((uint64_t)(int64_t)(t0 + t) * (uint64_t)p.turns[jj]) >> 32);
            float sn, cs;
            sincosf((float)ph * 1.4629180792671596e-9f, &sn, &cs);        // 2 pi / 2^32
            table[i] = make_float2(__fmul_rn(cs, p.factor), __fmul_rn(sn, p.factor));
        }
        __syncthreads();
        const int64_t tok0 = s.start + (t0 - first);
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            const int i = v * THREADS + tid, t = i >> vshift, d0 = (i & (vpr - 1)) << 3;
            if (t < nt) {
                load_rotated(p, p.k + (tok0 + t) * p.k_token + head * p.k_head, d0, p.kvec, table + t * half, held[0][v]);
                load8(p.v + (tok0 + t) * p.v_token + head * p.v_head + d0, p.vvec, held[1][v]);
                if (want_max) {
                    m[0] = finite_max(m[0], held[0][v]);
                    m[1] = finite_max(m[1], held[1][v]);
                }
            }
        }
    };
    auto turn_q = [&](int c) {
        const int t0 = lo + c * kChunk, nt = min(kChunk, hi - t0);
        const int64_t tok0 = s.start + (t0 - first);
        // A row's vectors lie in one warp and are all loaded before any is
        // stored, so q may be rotated in place.
        const int items = nt << vshift;
        for (int g = 0; g < G; ++g) {
            const int h = head * G + g;
            for (int i0 = 0; i0 < items; i0 += THREADS) {
                const int i = i0 + tid, t = i >> vshift, d0 = (i & (vpr - 1)) << 3;
                float x[8];
                if (i < items)
                    load_rotated(p, p.q + (tok0 + t) * p.q_token + h * p.q_head, d0, p.qvec, table + t * half, x);
                __syncwarp();
                if (i < items) store8(p.q_out + (tok0 + t) * p.o_token + h * p.o_head + d0, p.ovec, x);
            }
        }
    };
    // Pages of more than kChunk tokens: one pass for the amax (and q), one to store.
    for (int c = 0; c < chunks; ++c) {
        rows(c, true);
        turn_q(c);
    }
    if (!write) return;

#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m[w] = fmaxf(m[w], __shfl_xor_sync(~0u, m[w], o));
    if ((tid & 31) == 0) {
        red[0][tid >> 5] = m[0];
        red[1][tid >> 5] = m[1];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
        m[0] = fmaxf(m[0], red[0][i]);
        m[1] = fmaxf(m[1], red[1][i]);
    }
    const int e[2] = {max(page_exponent(m[0]), old_k), max(page_exponent(m[1]), old_v)};
    const int was[2] = {old_k, old_v};
    uint8_t *cache[2] = {p.k_cache + (int64_t)page * p.page_stride + (int64_t)head * p.head_stride,
                         p.v_cache + (int64_t)page * p.page_stride + (int64_t)head * p.head_stride};
    if (tid < 2) *exps[tid] = (int8_t)e[tid];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        if (older == 0 || e[w] == was[w]) continue;
        const float scale = exp2_int(max(was[w] - e[w], -126));
        for (int i = tid; i < older << vshift; i += THREADS) {           // 8 codes at a time
            uint2 *at = reinterpret_cast<uint2 *>(cache[w] + (int64_t)i * 8);
            const uint2 v = *at;
            uint32_t in[2] = {v.x, v.y}, out[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t l, h;
                e4m3x4_to_f16x2(in[k], l, h);
                const float2 a = __half22float2(*reinterpret_cast<__half2 *>(&l));
                const float2 c = __half22float2(*reinterpret_cast<__half2 *>(&h));
                out[k] = f32x2_to_e4m3x2(a.x * scale, a.y * scale) | f32x2_to_e4m3x2(c.x * scale, c.y * scale) << 16;
            }
            *at = make_uint2(out[0], out[1]);
        }
    }
    for (int c = 0; c < chunks; ++c) {
        if (chunks > 1) rows(c, false);
        const int t0 = lo + c * kChunk, nt = min(kChunk, hi - t0);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const float scale = exp2_int(-e[w]);
#pragma unroll
            for (int v = 0; v < kVecs; ++v) {
                const int i = v * THREADS + tid, t = i >> vshift, d0 = (i & (vpr - 1)) << 3;
                if (t < nt) {
                    const float(&x)[8] = held[w][v];
                    uint2 o;
                    o.x = f32x2_to_e4m3x2(x[0] * scale, x[1] * scale) | f32x2_to_e4m3x2(x[2] * scale, x[3] * scale) << 16;
                    o.y = f32x2_to_e4m3x2(x[4] * scale, x[5] * scale) | f32x2_to_e4m3x2(x[6] * scale, x[7] * scale) << 16;
                    *reinterpret_cast<uint2 *>(cache[w] + (int64_t)(t0 - slot * P + t) * p.D + d0) = o;
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs &args, cudaStream_t stream) {
    AppendArgs p = args;
    const int n = p.cu_q == nullptr ? p.T / p.B : p.max_q;
    // CTAs for the pages a sequence's n tokens can touch.
    p.units = n == 1 ? 1 : (n - 1) / p.P + 2;
    const int64_t gx = p.cu_q == nullptr ? (int64_t)p.B * p.units : (int64_t)p.T / p.P + 2 * (int64_t)p.B;
    const dim3 grid((unsigned)gx, (unsigned)p.Hk);
    // A thread holds kVecs vectors of K and of V: the small CTA covers 16 tokens.
    const bool small = (int64_t)std::min(n, p.P) * p.D <= (int64_t)kSmallThreads * kVecs * 8;
    const size_t smem = (size_t)(small ? std::min(n, p.P) : kChunk) * (size_t)(p.R / 2) * sizeof(float2);
    if (small) return launch_pdl(kv_append_kernel<kSmallThreads>, grid, dim3(kSmallThreads), smem, stream, p);
    return launch_pdl(kv_append_kernel<kBigThreads>, grid, dim3(kBigThreads), smem, stream, p);
}

}  // namespace lowbit
