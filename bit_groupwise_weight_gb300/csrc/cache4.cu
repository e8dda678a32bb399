// cache4.cu -- rotary positions and the write into the 4-bit paged cache, in one kernel
// (lowbit_kv_append4), and the values that a cache of either kind holds (lowbit_cache_values,
// lowbit_cache4_values).  Its part for queries serves the 8-bit write too (launch_append_queries).
//
// Mathematics: norms (optional) and rotation as in cache.cu (append.cuh), then k and v into
// codes of 4 bits with a scale for each 32 values (int4.cuh).  No token's codes depend on
// another's, unlike the 8-bit cache's, whose exponent is a page's.
//
// Work split.  A warp takes one token, or a part of its rows (the heads of q, k and v) when
// there are few tokens; a row is held by D / 8 neighbouring lanes, 8 values each, so that norms and
// scales are shuffles, and so are a value's mates in the rotation.  A lane holds the same values of
// every row: its cosines and sines stay in registers for all of them.  Rows come by asynchronous
// copies into a ring in shared memory, each lane's own bytes, as far ahead as the ring is long, the
// first ones before the token's place is known.  Odd sizes and unaligned rows are read directly
// and find their mates by way of shared memory.
//
// Bound: instructions (0.8 issued a cycle and scheduler; some 190 for two rows of q of 128 values with norm and rotation).
// 15502 tokens of 32 + 8 heads of 128 with norms take 78 us, 4.3 TB/s; 5003 of 28 + 4 heads with positions of three axes
// 21; one token 3.5, a launch's shortest.  Steps on the way: tokens' tables in shared memory read for every row 141 us; rows of
// different kinds in one loop, with shuffles of half warps, 116; loads ahead in registers 97; a ring of eight rows instead
// of four 1 us more.
#include <algorithm>
#include <type_traits>

#include "append.cuh"
#include "fp8.cuh"
#include "int4.cuh"
#include "ptx.cuh"

namespace lowbit {
namespace {

using namespace append;

constexpr int kThreads = 256, kWarps = kThreads / 32, kAhead = 4;
// Fewer warps than this: the rows of a token are divided.  A warp a token from 4864 on: 4800 and 4864 tokens take 28.9 and
// 28.5 us (32 + 8 heads of 128, norms; 28 + 4, three axes: 19.4 and 17.5), 4900 and 5500, a few CTAs past the 608 that the SMs hold,
// 33.4 and 34.3 (20.4 and 22.0), 8000 43.8 (27.5).
constexpr int kWarpsToFill = 152 * 32;

struct Token {
    bool live;                           // whether it is of a sequence, and not past max_q
    int pos;                             // its place in the sequence
    int page, slot;                      // where its codes go; page -1: nowhere
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Where token `at` of q, k and v stands.  A whole warp looks: 32 places of cu_q at a time.
__device__ __forceinline__ Token token_of(const AppendArgs &p, int at) {
    Token t{false, 0, -1, 0};
    int b = 0, i = at, all = p.n;
    if (p.cu_q == nullptr) {
        if (p.B > 1) b = at / p.n, i = at - b * p.n;
    } else {
        int n = p.B;                     // the last sequence that begins at `at` or before, among n from b on
        while (n > 1) {
            const int step = (n + 31) / 32, mine = (int)(threadIdx.x & 31) * step;
            const uint32_t begun = __ballot_sync(~0u, mine < n && (mine == 0 || p.cu_q[b + mine] <= at));
            const int last = (31 - __clz(begun)) * step;
            b += last, n = min(step, n - last);
        }
        const int start = min(max(p.cu_q[b], 0), p.T);
        i = at - start, all = min(p.cu_q[b + 1], p.T) - start;
        if (i < 0 || i >= min(all, p.max_q)) return t;
    }
    t.live = true;
    t.pos = max(p.lens[b], 0) - all + i;
    const int page = t.pos >> p.pshift;
    if (t.pos >= 0 && page < p.width) {
        const int id = p.page_table[(int64_t)b * p.table_stride + page];
        if (id >= 0 && id < p.pages) t.page = id, t.slot = t.pos & (p.P - 1);
    }
    return t;
}

// The largest magnitude of three, NaN if one is.
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(fabsf(a)), "f"(fabsf(b)), "f"(fabsf(c)));
    return d;
}

// Eight values of a group of 32 (held by four lanes) into their codes, and the group's scale; the
// whole warp calls, and what is not `stored` is not written.
__device__ __forceinline__ void store_codes(const float (&x)[8], bool stored, uint8_t *codes, uint8_t *scale) {
    float top = max3(max3(max3(0.f, x[0], x[1]), x[2], x[3]), max3(max3(0.f, x[4], x[5]), x[6], x[7]), 0.f);
    top = max3(top, __shfl_xor_sync(~0u, top, 1), 0.f);
    top = max3(top, __shfl_xor_sync(~0u, top, 2), 0.f);
    const bool nan = top != top;
    if (__any_sync(~0u, !(top < INFINITY))) {        // not all of it finite
        top = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fabsf(x[i]) < INFINITY ? fmaxf(top, fabsf(x[i])) : top;
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
    }
    const float s = scale4(top);
    const uint32_t w = codes4(x, s);
    if (stored) {
        *reinterpret_cast<uint32_t *>(codes) = w;
        if ((threadIdx.x & 3) == 0) *scale = (uint8_t)(nan ? 0x7Fu : scale4_byte(s));
    }
}

enum Kind { kQuery, kKey, kValue };

// FULL: the whole head is rotated.
template <int D, Form FORM, bool FULL>
__global__ void __launch_bounds__(kThreads, 4) kv_append4_kernel(const AppendArgs p) {
    constexpr int kRow = D / 8, kRows = 32 / kRow;                       // lanes of a row, rows of a warp
    __shared__ __align__(16) float turns[kWarps][2][D / 2];              // cosines and sines of the warp's token
    __shared__ __align__(16) float weights[2][D];                        // of the norms of q and k
    __shared__ float whole[FORM == kAny ? kThreads / kRow : 1][FORM == kAny ? D : 1];
    __shared__ uint4 ring[FORM == kAny ? 1 : kWarps][FORM == kAny ? 1 : kAhead][32];
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, lane_in = lane % kRow, row_in = lane / kRow, d0 = lane_in * 8;
    const int half = p.R >> 1, unit = blockIdx.x * kWarps + warp, at = unit / p.units, part = unit - at * p.units;
    if (p.q_norm != nullptr || p.k_norm != nullptr) {
        for (int i = tid; i < 2 * D; i += kThreads) {
            const void *w = i < D ? p.q_norm : p.k_norm;
            weights[i / D][i % D] = w == nullptr ? 1.f : norm_weight(w, p.norm_dtype, i % D);
        }
        __syncthreads();
    }
    if (at >= p.T) return;
    // The warp's share of the rows, in sets of kRows of one kind.
    const int q_sets = (p.Hq + kRows - 1) / kRows, k_sets = p.q_only ? 0 : (p.Hk + kRows - 1) / kRows, sets = q_sets + 2 * k_sets;
    const int begin = (int)((int64_t)sets * part / p.units);
    const int end = (int)((int64_t)sets * (part + 1) / p.units);
    // The next row to come: where it is, how far the following one of its kind, how many rows are left of it.
    const uint16_t *coming;
    int64_t pitch;
    int left, coming_set = begin;
    auto find = [&] {
        const int kind = coming_set < q_sets ? kQuery : (coming_set < q_sets + k_sets ? kKey : kValue);
        const int r = (coming_set - (kind == kQuery ? 0 : (kind == kKey ? q_sets : q_sets + k_sets))) * kRows + row_in;
        const int64_t head = kind == kQuery ? p.q_head : (kind == kKey ? p.k_head : p.v_head);
        coming = (kind == kQuery ? p.q + at * p.q_token : (kind == kKey ? p.k + at * p.k_token : p.v + at * p.v_token)) + r * head + d0;
        pitch = head * kRows, left = (kind == kQuery ? p.Hq : p.Hk) - r;
    };
    auto advance = [&] {
        coming += pitch, left -= kRows;
        if (++coming_set == q_sets || coming_set == q_sets + k_sets) find();
    };
    uint32_t slot = 0, taken = 0;                                        // of the ring, for what comes and what is next
    auto fetch = [&] {
        if constexpr (FORM != kAny) {
            if (coming_set < end) {
                if (left > 0) cp_async16(ptx::smem_u32(&ring[warp][slot][lane]), coming);
                advance();
            }
            slot = (slot + 1) % kAhead;
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    };
    auto next = [&] {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if constexpr (FORM == kAny) {
            if (left > 0) v = load8<FORM>(coming);
            advance();
        } else {
            asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
            v = ring[warp][taken][lane];
            taken = (taken + 1) % kAhead;
        }
        return v;
    };
    find();
#pragma unroll
    for (int u = 0; u < kAhead; ++u) fetch();
    const Token tok = token_of(p, at);
    if (!tok.live) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        return;
    }
    for (int j = lane; j < half; j += 32) turn_of(p, position_of(p, at, tok.pos, j), j, turns[warp][0][j], turns[warp][1][j]);
    __syncwarp();

    // What the lane's values are multiplied by in the rotation: kHalves x cos + mate sin (the lower half's
    // sines turned around), kNeighbours four pairs.  Not turned: by 1 and 0.
    const bool upper = d0 >= half, turned = FULL || d0 < p.R;
    const int mate_lane = FORM == kHalves && turned ? (upper ? d0 - half : d0 + half) >> 3 : lane_in;
    constexpr int kAngles = FORM == kHalves ? 8 : (FORM == kNeighbours ? 4 : 1);
    float cs[kAngles], sn[kAngles];
    if constexpr (FORM != kAny) {
        const int j0 = FORM == kHalves ? (upper ? d0 - half : d0) : d0 >> 1;
#pragma unroll
        for (int k = 0; k < kAngles; ++k) {
            cs[k] = turned ? turns[warp][0][j0 + k] : 1.f, sn[k] = turned ? turns[warp][1][j0 + k] : 0.f;
            if (FORM == kHalves && !upper) sn[k] = -sn[k];
        }
    }
    auto rows = [&]<int KIND>(std::integral_constant<int, KIND>) {
        const int before = KIND == kQuery ? 0 : (KIND == kKey ? q_sets : q_sets + k_sets), count = KIND == kQuery ? p.Hq : p.Hk;
        const int first = max(begin - before, 0), last = min(end - before, KIND == kQuery ? q_sets : k_sets);
        if (first >= last) return;
        const int r0 = first * kRows + row_in;
        uint16_t *to = p.q_out + at * p.o_token + r0 * p.o_head + d0;
        uint8_t *codes = (KIND == kKey ? p.k_cache : p.v_cache) + tok.page * p.page_stride + r0 * p.head_stride + tok.slot * (D / 2) + lane_in * 4;
        uint8_t *scale = (KIND == kKey ? p.k_scale : p.v_scale) + tok.page * p.scale_page_stride + r0 * p.scale_head_stride +
                         tok.slot * (D / kGroup4) + lane_in / 4;
        const bool norm = KIND == kQuery ? p.q_norm != nullptr : (KIND == kKey && p.k_norm != nullptr);
        float wt[KIND == kValue ? 1 : 8];
        if constexpr (KIND != kValue) {
            if (norm) {
#pragma unroll
                for (int k = 0; k < 8; ++k) wt[k] = weights[KIND][d0 + k];
            }
        }
        for (int set = first; set < last; ++set) {
            const bool live = set * kRows + row_in < count && (KIND == kQuery || tok.page >= 0);   // the last set may have fewer rows
            float x[8];
            widen(next(), x);
            fetch();
            if constexpr (KIND != kValue) {
                if (norm) {
                    const float by = row_norm<kRow>(x, p.eps, ~0u);
#pragma unroll
                    for (int k = 0; k < 8; k += 2) {
                        const float2 y = ptx::fmul2(ptx::fmul2(make_float2(x[k], x[k + 1]), make_float2(by, by)), make_float2(wt[k], wt[k + 1]));
                        x[k] = y.x, x[k + 1] = y.y;
                    }
                }
                if constexpr (FORM == kHalves) {
#pragma unroll
                    for (int k = 0; k < 8; k += 2) {
                        const float2 y = make_float2(__shfl_sync(~0u, x[k], mate_lane, kRow), __shfl_sync(~0u, x[k + 1], mate_lane, kRow));
                        const float2 a = ptx::fmul2(make_float2(x[k], x[k + 1]), make_float2(cs[k], cs[k + 1]));
                        const float2 b = ptx::fmul2(y, make_float2(sn[k], sn[k + 1]));
                        // (Sums two at a time would be contracted with the products.)
                        x[k] = turned ? __fadd_rn(a.x, b.x) : x[k], x[k + 1] = turned ? __fadd_rn(a.y, b.y) : x[k + 1];
                    }
                } else if constexpr (FORM == kNeighbours) {
                    if (turned) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float a = x[2 * k], b = x[2 * k + 1];
                            x[2 * k] = __fsub_rn(__fmul_rn(a, cs[k]), __fmul_rn(b, sn[k]));
                            x[2 * k + 1] = __fadd_rn(__fmul_rn(a, sn[k]), __fmul_rn(b, cs[k]));
                        }
                    }
                } else {
                    float *all = whole[tid / kRow];
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8; ++i) all[d0 + i] = x[i];
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int d = d0 + i;
                        if (d >= p.R) continue;
                        const bool second = p.interleaved ? d & 1 : d >= half;
                        const int m = p.interleaved ? d ^ 1 : (second ? d - half : d + half), j = p.interleaved ? d >> 1 : (second ? m : d);
                        const float a = __fmul_rn(x[i], turns[warp][0][j]), b = __fmul_rn(all[m], turns[warp][1][j]);
                        x[i] = second ? __fadd_rn(b, a) : __fsub_rn(a, b);
                    }
                }
            }
            if constexpr (KIND == kQuery) {
                const uint32_t w[4] = {f32x2_to_bf16x2(x[0], x[1]), f32x2_to_bf16x2(x[2], x[3]), f32x2_to_bf16x2(x[4], x[5]),
                                       f32x2_to_bf16x2(x[6], x[7])};
                if (!live) {
                } else if constexpr (FORM != kAny) {
                    *reinterpret_cast<uint4 *>(to) = make_uint4(w[0], w[1], w[2], w[3]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) to[i] = (uint16_t)(w[i >> 1] >> (i & 1 ? 16 : 0));
                }
                to += kRows * p.o_head;
            } else {
                store_codes(x, live, codes, scale);
                codes += kRows * p.head_stride, scale += kRows * p.scale_head_stride;
            }
        }
    };
    rows(std::integral_constant<int, kQuery>{});
    rows(std::integral_constant<int, kKey>{});
    rows(std::integral_constant<int, kValue>{});
}

template <int D>
cudaError_t launch(const AppendArgs &p, cudaStream_t stream) {
    constexpr int kRows = 32 / (D / 8);
    const bool vec = p.qvec && p.kvec && p.vvec && p.ovec;
    const bool full = p.R == D;
    const auto kernel = vec && p.interleaved && p.R % 8 == 0 ? (full ? kv_append4_kernel<D, kNeighbours, true> : kv_append4_kernel<D, kNeighbours, false>)
                        : vec && !p.interleaved && p.R % 16 == 0 ? (full ? kv_append4_kernel<D, kHalves, true> : kv_append4_kernel<D, kHalves, false>)
                                                                 : kv_append4_kernel<D, kAny, false>;
    AppendArgs a = p;                    // units: warps of a token
    const int64_t sets = (p.Hq + kRows - 1) / kRows + (p.q_only ? 0 : 2 * (int64_t)((p.Hk + kRows - 1) / kRows));
    a.units = (int)std::min<int64_t>(sets, (kWarpsToFill + (int64_t)p.T - 1) / p.T);
    const int64_t ctas = ((int64_t)p.T * a.units + kWarps - 1) / kWarps;
    return launch_pdl(kernel, dim3((unsigned)ctas), dim3(kThreads), 0, stream, (const AppendArgs)a);
}

// Eight values of K and of V a thread; a page's head is 2^place_bits of such.  Bound: HBM, mostly the 16-bit
// values that are written: 250 pages of 64 tokens, 8 heads of 128, 12.8 us, 2000 99, 6.7 TB/s, a copy's rate.
template <int D, bool FOUR>
__global__ void __launch_bounds__(256) cache_values_kernel(const ValuesArgs p, int place_bits) {
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();
    const int64_t n = ((int64_t)p.pages * p.Hk) << place_bits;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const uint32_t place = (uint32_t)(i >> place_bits), in = (uint32_t)i & ((1u << place_bits) - 1u);
        const uint32_t page = place / (uint32_t)p.Hk, head = place - page * (uint32_t)p.Hk;
        uint32_t w[2][2], scale[2];
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const uint8_t *codes = (which ? p.v : p.k) + page * p.page_stride + head * p.head_stride;
            if constexpr (FOUR) {
                w[which][0] = *reinterpret_cast<const uint32_t *>(codes + in * 4);
                scale[which] = ((which ? p.v_scale : p.k_scale) + page * p.scale_page_stride + head * p.scale_head_stride)[in / 4];
            } else {
                const uint2 v = *reinterpret_cast<const uint2 *>(codes + in * 8);
                w[which][0] = v.x, w[which][1] = v.y;
                scale[which] = (uint32_t)(which ? p.v_exp : p.k_exp)[place];
            }
        }
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            uint4 &to = *reinterpret_cast<uint4 *>((which ? p.v_out : p.k_out) + i * 8);
            if constexpr (FOUR) {
                // A nibble in the mantissa of bf16's 128 is 128 + code; less 136, times the scale: exact each.
                const __nv_bfloat162 s = __float2bfloat162_rn(__half2float(__ushort_as_half((uint16_t)(scale[which] << 8))));
                uint32_t y[4];                                           // values k and k + 4
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t in = ptx::lop3_and_or(w[which][0] >> (4 * k), 0x000F000Fu, 0x43004300u);
                    const __nv_bfloat162 x = __hmul2(__hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&in), __float2bfloat162_rn(136.f)), s);
                    y[k] = *reinterpret_cast<const uint32_t *>(&x);
                }
                to = make_uint4(ptx::prmt(y[0], y[1], 0x5410u), ptx::prmt(y[2], y[3], 0x5410u), ptx::prmt(y[0], y[1], 0x7632u),
                                ptx::prmt(y[2], y[3], 0x7632u));
            } else {
                const float s = exp2_int(min(max((int)scale[which], kExpMin), kExpMax));
                uint32_t h[4];
                e4m3x4_to_f16x2(w[which][0], h[0], h[1]);
                e4m3x4_to_f16x2(w[which][1], h[2], h[3]);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 x = ptx::fmul2(__half22float2(*reinterpret_cast<const __half2 *>(&h[k])), make_float2(s, s));
                    h[k] = f32x2_to_bf16x2(x.x, x.y);
                }
                to = make_uint4(h[0], h[1], h[2], h[3]);
            }
        }
    }
}

}  // namespace

cudaError_t launch_append_queries(const AppendArgs &args, cudaStream_t stream) {
    AppendArgs p = args;
    p.q_only = true;
    return launch_kv_append4(p, stream);
}

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
    int bits = 0;
    while (1 << bits < p.P * (p.D / 8)) ++bits;
    const int64_t n = (int64_t)p.pages * p.Hk << bits;
    return launch_pdl(kernel, dim3((unsigned)std::min<int64_t>((n + 255) / 256, 152 * 128)), dim3(256), 0, stream, p, bits);
}

}  // namespace lowbit
