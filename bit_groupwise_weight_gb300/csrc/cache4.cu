// cache4.cu -- rotary positions and the write into the 4-bit paged cache, in one kernel
// (lowbit_kv_append4), and the values that a cache of either kind holds (lowbit_cache_values,
// lowbit_cache4_values).
//
// Mathematics: norms (optional) and rotation as in cache.cu (append.cuh), then k and v into
// codes of 4 bits with a scale for each 32 values (int4.cuh).  No token's codes depend on
// another's, unlike the 8-bit cache's, whose exponent is a page's.
//
// Work split.  A CTA takes a few tokens and, when there are few of them, a part of their rows
// (the heads of q, k and v); a row is held by D / 8 neighbouring lanes, 8 values each, so that
// norms and scales are shuffles.  A thread keeps to one row at a time and goes through the
// tokens, four loads ahead of the work.  Cosines and sines are computed once a CTA for all its
// rows.  Where the vectors allow it a value's mate of the rotation comes by a shuffle, else (odd
// sizes, unaligned rows) by way of shared memory.
#include <algorithm>

#include "append.cuh"
#include "fp8.cuh"
#include "int4.cuh"
#include "ptx.cuh"

namespace lowbit {
namespace {

using namespace append;

constexpr int kThreads = 256, kMostTokens = 8, kAhead = 4;
constexpr int kCtasToFill = 152 * 4;             // fewer CTAs than this: fewer tokens each, then rows divided

struct Token {
    int live;                            // whether it is of a sequence, and not past max_q
    int pos;                             // its place in the sequence
    int page, slot;                      // where its codes go; page -1: nowhere
};

// Where token `at` of q, k and v stands: by bisection of cu_q.
__device__ __forceinline__ Token token_of(const AppendArgs &p, int at) {
    Token t{0, 0, -1, 0};
    int b, i, all;
    if (p.cu_q == nullptr) {
        b = at / p.n, i = at - b * p.n, all = p.n;
    } else {
        int lo = 0, hi = p.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (p.cu_q[mid] <= at) lo = mid;
            else hi = mid - 1;
        }
        b = lo;
        const int start = min(max(p.cu_q[b], 0), p.T);
        i = at - start, all = min(p.cu_q[b + 1], p.T) - start;
        if (i < 0 || i >= min(all, p.max_q)) return t;
    }
    t.live = 1;
    t.pos = max(p.lens[b], 0) - all + i;
    const int page = t.pos >> p.pshift;
    if (t.pos >= 0 && page < p.width) {
        const int id = p.page_table[(int64_t)b * p.table_stride + page];
        if (id >= 0 && id < p.pages) t.page = id, t.slot = t.pos & (p.P - 1);
    }
    return t;
}

template <int D, Form FORM>
__global__ void __launch_bounds__(kThreads, 4) kv_append4_kernel(const AppendArgs p) {
    constexpr int kRow = D / 8, kRows = kThreads / kRow;                  // lanes of a row, rows of a CTA at once
    extern __shared__ __align__(16) float table[];                       // [tokens][R / 2] cosines, then sines
    __shared__ __align__(16) float weights[2][D];                        // of the norms of q and k
    __shared__ Token tokens[kMostTokens];
    __shared__ float whole[FORM == kAny ? kRows : 1][FORM == kAny ? D : 1];
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();
    const int tid = threadIdx.x, half = p.R >> 1, first = blockIdx.x * p.table_tokens, nt = min(p.table_tokens, p.T - first);
    const bool normed = p.q_norm != nullptr || p.k_norm != nullptr;
    if (tid < nt) tokens[tid] = token_of(p, first + tid);
    if (normed)
        for (int i = tid; i < 2 * D; i += kThreads) {
            const void *w = i < D ? p.q_norm : p.k_norm;
            weights[i / D][i % D] = w == nullptr ? 1.f : norm_weight(w, p.norm_dtype, i % D);
        }
    __syncthreads();
    for (int i = tid; i < nt * half; i += kThreads) {
        const int t = i / half, j = i - t * half;
        turn_of(p, position_of(p, first + t, tokens[t].pos, j), j, table[i], table[p.table_tokens * half + i]);
    }
    __syncthreads();

    const int lane_in = tid % kRow, d0 = lane_in * 8;
    const uint32_t mask = row_mask<kRow>();
    const bool upper = d0 >= half;
    const int mate_at = upper ? d0 - half : d0 + half;                   // where kHalves' mates are
    for (int r = blockIdx.y * kRows + tid / kRow; r < p.Hq + 2 * p.Hk; r += gridDim.y * kRows) {
        const int kind = r < p.Hq ? 0 : (r < p.Hq + p.Hk ? 1 : 2);       // of q, k or v
        const int head = kind == 0 ? r : (kind == 1 ? r - p.Hq : r - p.Hq - p.Hk);
        const int64_t pitch = kind == 0 ? p.q_token : (kind == 1 ? p.k_token : p.v_token);
        const uint16_t *row = (kind == 0 ? p.q + head * p.q_head : (kind == 1 ? p.k + head * p.k_head : p.v + head * p.v_head)) +
                              first * pitch + d0;
        const bool norm = kind == 0 ? p.q_norm != nullptr : (kind == 1 && p.k_norm != nullptr);
        const float *wt = weights[kind == 1];
        for (int t0 = 0; t0 < nt; t0 += kAhead) {
            uint4 v[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (t0 + u < nt) v[u] = load8<FORM>(row + (t0 + u) * pitch);
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int t = t0 + u;
                if (t >= nt) break;
                const Token tok = tokens[t];
                if (!tok.live || (kind != 0 && tok.page < 0)) continue;  // the same for the row's lanes
                float x[8];
                widen(v[u], x);
                if (kind != 2) {
                    float by = 1.f;
                    if (norm) {
                        by = row_norm<kRow>(x, p.eps);
                        weigh(x, by, wt + d0);
                    }
                    const float *cs = table + t * half, *sn = table + (p.table_tokens + t) * half;
                    if constexpr (FORM == kHalves) {
                        const int from = d0 < p.R ? mate_at >> 3 : lane_in;
                        const uint32_t flip = upper ? 0u : 0x80008000u;
                        float y[8];
                        widen(make_uint4(__shfl_sync(mask, v[u].x, from, kRow) ^ flip, __shfl_sync(mask, v[u].y, from, kRow) ^ flip,
                                         __shfl_sync(mask, v[u].z, from, kRow) ^ flip, __shfl_sync(mask, v[u].w, from, kRow) ^ flip), y);
                        if (d0 < p.R) {
                            if (norm) weigh(y, by, wt + mate_at);
                            const int j0 = upper ? mate_at : d0;
#pragma unroll
                            for (int i = 0; i < 8; i += 4) {
                                const float4 c = *reinterpret_cast<const float4 *>(cs + j0 + i), s = *reinterpret_cast<const float4 *>(sn + j0 + i);
                                const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                                for (int k = 0; k < 4; ++k) x[i + k] = __fadd_rn(__fmul_rn(x[i + k], cc[k]), __fmul_rn(y[i + k], ss[k]));
                            }
                        }
                    } else if constexpr (FORM == kNeighbours) {
                        if (d0 < p.R) {
                            const float4 c = *reinterpret_cast<const float4 *>(cs + (d0 >> 1)), s = *reinterpret_cast<const float4 *>(sn + (d0 >> 1));
                            const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float a = x[2 * k], b = x[2 * k + 1];
                                x[2 * k] = __fsub_rn(__fmul_rn(a, cc[k]), __fmul_rn(b, ss[k]));
                                x[2 * k + 1] = __fadd_rn(__fmul_rn(a, ss[k]), __fmul_rn(b, cc[k]));
                            }
                        }
                    } else {
                        float *all = whole[tid / kRow];
                        __syncwarp(mask);
#pragma unroll
                        for (int i = 0; i < 8; ++i) all[d0 + i] = x[i];
                        __syncwarp(mask);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int d = d0 + i;
                            if (d >= p.R) continue;
                            const bool second = p.interleaved ? d & 1 : d >= half;
                            const int m = p.interleaved ? d ^ 1 : (second ? d - half : d + half), j = p.interleaved ? d >> 1 : (second ? m : d);
                            const float a = __fmul_rn(x[i], cs[j]), b = __fmul_rn(all[m], sn[j]);
                            x[i] = second ? __fadd_rn(b, a) : __fsub_rn(a, b);
                        }
                    }
                }
                if (kind == 0) {
                    uint16_t *to = p.q_out + (int64_t)(first + t) * p.o_token + head * p.o_head + d0;
                    const uint32_t w[4] = {f32x2_to_bf16x2(x[0], x[1]), f32x2_to_bf16x2(x[2], x[3]), f32x2_to_bf16x2(x[4], x[5]),
                                           f32x2_to_bf16x2(x[6], x[7])};
                    if constexpr (FORM != kAny) {
                        *reinterpret_cast<uint4 *>(to) = make_uint4(w[0], w[1], w[2], w[3]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) to[i] = (uint16_t)(w[i >> 1] >> (i & 1 ? 16 : 0));
                    }
                    continue;
                }
                // The group's largest magnitude: as bits, over the four lanes that hold it.
                const uint32_t four = 0xFu << (tid & 28);
                uint32_t top = 0u;
#pragma unroll
                for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
                top = max(top, __shfl_xor_sync(four, top, 1));
                top = max(top, __shfl_xor_sync(four, top, 2));
                bool nan = false;
                if (top >= 0x7F800000u) {                                // not all of it finite
                    nan = top > 0x7F800000u;
                    top = 0u;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t a = __float_as_uint(x[i]) & 0x7FFFFFFFu;
                        top = max(top, a < 0x7F800000u ? a : 0u);
                    }
                    top = max(top, __shfl_xor_sync(four, top, 1));
                    top = max(top, __shfl_xor_sync(four, top, 2));
                }
                const float s = scale4(__uint_as_float(top));
                uint8_t *codes = (kind == 1 ? p.k_cache : p.v_cache) + tok.page * p.page_stride + head * p.head_stride + tok.slot * (D / 2);
                uint8_t *scales = (kind == 1 ? p.k_scale : p.v_scale) + tok.page * p.scale_page_stride + head * p.scale_head_stride + tok.slot * (D / kGroup4);
                *reinterpret_cast<uint32_t *>(codes + lane_in * 4) = codes4(x, s);
                if ((tid & 3) == 0) scales[lane_in / 4] = (uint8_t)(nan ? 0x7Fu : scale4_byte(s));
            }
        }
    }
}

template <int D>
cudaError_t launch(const AppendArgs &p, cudaStream_t stream) {
    constexpr int kRows = kThreads / (D / 8);
    const bool vec = p.qvec && p.kvec && p.vvec && p.ovec;
    const auto kernel = vec && p.interleaved && p.R % 8 == 0 ? kv_append4_kernel<D, kNeighbours>
                        : vec && !p.interleaved && p.R % 16 == 0 ? kv_append4_kernel<D, kHalves>
                                                                 : kv_append4_kernel<D, kAny>;
    AppendArgs a = p;
    const int passes = (p.Hq + 2 * p.Hk + kRows - 1) / kRows;
    a.table_tokens = kMostTokens;
    while (a.table_tokens > 1 && p.T < (int64_t)a.table_tokens * kCtasToFill) a.table_tokens /= 2;
    const int64_t gx = (p.T + a.table_tokens - 1) / a.table_tokens;
    const int gy = gx >= kCtasToFill ? 1 : (int)std::min<int64_t>(passes, (kCtasToFill + gx - 1) / gx);
    return launch_pdl(kernel, dim3((unsigned)gx, (unsigned)gy), dim3(kThreads), (size_t)a.table_tokens * p.R * sizeof(float),
                      stream, (const AppendArgs)a);
}

// Eight values a thread.  Bound: HBM, mostly the 16-bit values that are written.
template <int D, bool FOUR>
__global__ void __launch_bounds__(256) cache_values_kernel(const ValuesArgs p) {
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();
    const int64_t n = (int64_t)p.pages * p.Hk * p.P * (D / 8);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int d8 = (int)(i % (D / 8));
        const int64_t row = i / (D / 8), place = row / p.P;              // place: page and head
        const int slot = (int)(row - place * p.P), head = (int)(place % p.Hk);
        const int64_t page = place / p.Hk;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const uint8_t *codes = (which ? p.v : p.k) + page * p.page_stride + head * p.head_stride;
            float x[8];
            if constexpr (FOUR) {
                const uint8_t *scales = (which ? p.v_scale : p.k_scale) + page * p.scale_page_stride + head * p.scale_head_stride;
                const uint32_t w = *reinterpret_cast<const uint32_t *>(codes + slot * (D / 2) + d8 * 4);
                const float s = __half2float(__ushort_as_half((uint16_t)(scales[slot * (D / kGroup4) + d8 / 4] << 8)));
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = (float)((int)(w >> (4 * k) & 15u) - 8) * s;
            } else {
                const uint2 w = *reinterpret_cast<const uint2 *>(codes + slot * D + d8 * 8);
                const int e = (which ? p.v_exp : p.k_exp)[place];
                const float s = exp2_int(min(max(e, kExpMin), kExpMax));
                uint32_t h[4];
                e4m3x4_to_f16x2(w.x, h[0], h[1]);
                e4m3x4_to_f16x2(w.y, h[2], h[3]);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&h[k]));
                    x[2 * k] = y.x * s, x[2 * k + 1] = y.y * s;
                }
            }
            *reinterpret_cast<uint4 *>((which ? p.v_out : p.k_out) + i * 8) =
                make_uint4(f32x2_to_bf16x2(x[0], x[1]), f32x2_to_bf16x2(x[2], x[3]), f32x2_to_bf16x2(x[4], x[5]),
                           f32x2_to_bf16x2(x[6], x[7]));
        }
    }
}

}  // namespace

cudaError_t launch_kv_append4(const AppendArgs &args, cudaStream_t stream) {
    AppendArgs p = args;
    p.n = p.cu_q == nullptr ? p.T / p.B : 0;
    p.pshift = 0;
    while ((1 << p.pshift) < p.P) ++p.pshift;
    return p.D == 128 ? launch<128>(p, stream) : launch<64>(p, stream);
}

cudaError_t launch_cache_values(const ValuesArgs &p, cudaStream_t stream) {
    const bool four = p.k_scale != nullptr;
    const auto kernel = p.D == 128 ? (four ? cache_values_kernel<128, true> : cache_values_kernel<128, false>)
                                   : (four ? cache_values_kernel<64, true> : cache_values_kernel<64, false>);
    const int64_t n = (int64_t)p.pages * p.Hk * p.P * (p.D / 8);
    return launch_pdl(kernel, dim3((unsigned)std::min<int64_t>((n + 255) / 256, 152 * 8 * 8)), dim3(256), 0, stream, p);
}

}  // namespace lowbit
