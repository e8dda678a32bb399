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
// Work split.  One CTA takes one page of one sequence and one key-value head: the new
// tokens of that page, their K and V rows of the head and the q rows of its group.  So
// a page's amax, its exponent and its older codes belong to one CTA (no atomics, no
// second launch).  The cosines and sines of the page's tokens are computed once for the
// head's rows (sharing them over a cluster of the heads' CTAs was slower: 101 against
// 88 us for 16002 tokens).  Rows are loaded one set ahead of the one in work.
// With norms or positions of the caller's own, prompts go another way: the rows of q through cache4.cu's kernel,
// and here a CTA takes the keys or the values of a page, of several heads with one table (15502 tokens with norms 103
// us, with positions 94; all in one kernel 169, a CTA a head for keys and values 128).  Pages of more tokens than a CTA holds at
// once (64 of 128 values) are read twice, with a table for each head and set of rows: with pages of 128 and 256 tokens
// it is 169 and 171 us.
//
// Bound: HBM (T D (4 Hq + 6 Hk) bytes) for prompts, launch latency for decode.  16002 tokens
// of 32 + 8 heads of 128 take 84.5 us, 4.1 TB/s (0.61 of a copy's rate: the CTAs of an SM hold
// too few loads in flight this way); one token 3.9 us.
#include <algorithm>
#include <type_traits>

#include "append.cuh"
#include "fp8.cuh"
#include "ptx.cuh"

namespace lowbit {
namespace {

using namespace append;

// The big CTA holds 64 tokens of 128 values (128 of 64) in vectors of 8, the small one
// 4 (8): fewer registers and instructions for decode (5.4 -> 4.5 us a call).
constexpr int kBigThreads = 256, kSmallThreads = 64;
template <int THREADS>
constexpr int kVecsOf = THREADS == kBigThreads ? 4 : 1;       // vectors of a thread
template <int THREADS>
constexpr int kPerSm = 512 / THREADS;                         // CTAs of an SM

enum Kind { kKey, kValue, kQuery };
constexpr int kCtasToFill = 152 * 4;

struct Seq { int start, n, len; };

// Where a sequence's new tokens lie in q, k and v, and its length with them.  Of tokens past
// max_q, which are left out, neither n nor len counts any: the first one stands at len - n.
__device__ __forceinline__ Seq sequence(const AppendArgs &p, int b) {
    Seq s;
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
    s.len = max(p.lens[b], 0) - over;
    return s;
}

// A thread's vectors of a set of rows: its own values and, for kHalves, their mates.
template <Form FORM, int kVecs>
struct Rows {
    uint4 own[kVecs];
    uint4 mate[FORM == kHalves ? kVecs : 1];
};

// Values d0 .. d0+7 of a row, rotated.  cs, sn: the token's cosines and sines, one a
// pair.  Products and sums are rounded one by one, so that the page's exponent follows from
// the same fp32 values in any implementation, but for kHalves without PRE: there they are taken
// two at a time, and the compiler makes one rounding of a product and the sum.  With PRE, x comes
// normed, and its mates are: times `norm`, times their weights `wt`.
template <Form FORM, bool PRE>
__device__ __forceinline__ void rotate(const AppendArgs &p, const uint16_t *row, int d0, const uint4 &mate, const float *cs,
                                       const float *sn, float (&x)[8], float norm, const float *wt) {
    if (d0 >= p.R) return;
    const int half = p.R >> 1;
    if constexpr (FORM == kHalves) {
        const bool upper = d0 >= half;
        const int j0 = upper ? d0 - half : d0;
        const uint32_t flip = upper ? 0u : 0x80008000u;
        float y[8];
        widen(make_uint4(mate.x ^ flip, mate.y ^ flip, mate.z ^ flip, mate.w ^ flip), y);
        if constexpr (PRE) weigh(y, norm, wt + (upper ? j0 : d0 + half));
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            const float4 c = *reinterpret_cast<const float4 *>(cs + j0 + i), s = *reinterpret_cast<const float4 *>(sn + j0 + i);
            const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int k = 0; k < 4; k += 2) {     // x cos -+ y sin
                if constexpr (PRE) {
                    x[i + k] = __fadd_rn(__fmul_rn(x[i + k], cc[k]), __fmul_rn(y[i + k], ss[k]));
                    x[i + k + 1] = __fadd_rn(__fmul_rn(x[i + k + 1], cc[k + 1]), __fmul_rn(y[i + k + 1], ss[k + 1]));
                    continue;
                }
                const float2 a = ptx::fmul2(make_float2(x[i + k], x[i + k + 1]), make_float2(cc[k], cc[k + 1]));
                const float2 b = ptx::fmul2(make_float2(y[i + k], y[i + k + 1]), make_float2(ss[k], ss[k + 1]));
                const float2 r = ptx::fadd2(a, b);
                x[i + k] = r.x, x[i + k + 1] = r.y;
            }
        }
    } else if constexpr (FORM == kNeighbours) {
        const float4 c = *reinterpret_cast<const float4 *>(cs + (d0 >> 1)), s = *reinterpret_cast<const float4 *>(sn + (d0 >> 1));
        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = x[2 * i], b = x[2 * i + 1];
            x[2 * i] = __fsub_rn(__fmul_rn(a, cc[i]), __fmul_rn(b, ss[i]));
            x[2 * i + 1] = __fadd_rn(__fmul_rn(a, ss[i]), __fmul_rn(b, cc[i]));
        }
    } else if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; i += 2)
            if (d0 + i < p.R) {
                const float a = x[i], b = x[i + 1], c = cs[(d0 + i) >> 1], s = sn[(d0 + i) >> 1];
                x[i] = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
                x[i + 1] = __fadd_rn(__fmul_rn(a, s), __fmul_rn(b, c));
            }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int d = d0 + i;
            if (d < p.R) {
                const bool upper = d >= half;
                const int j = upper ? d - half : d;
                float y = __uint_as_float((uint32_t)row[upper ? j : d + half] << 16);
                if constexpr (PRE) y = __fmul_rn(__fmul_rn(y, norm), wt[upper ? j : d + half]);
                const float t = __fmul_rn(x[i], cs[j]), u = __fmul_rn(y, sn[j]);
                x[i] = upper ? __fadd_rn(u, t) : __fsub_rn(t, u);
            }
        }
    }
}

// PRE: with norms of q or k, or positions of the caller's own.
template <int THREADS, int D, Form FORM, bool PRE>
__global__ void __launch_bounds__(THREADS, kPerSm<THREADS>) kv_append_kernel(const AppendArgs p) {
    constexpr int kVecs = kVecsOf<THREADS>;
    constexpr int kRow = D / 8, kStep = THREADS / kRow, kChunk = kStep * kVecs;      // vectors of a row; tokens apart; of a set
    extern __shared__ __align__(16) float table[];        // [tokens][R / 2] cosines, then sines
    __shared__ float red[2][THREADS / 32];
    __shared__ __align__(16) float weights[2][PRE ? D : 4];              // of the norms of q and k
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();

    // This CTA's sequence and page.  With ragged sequences, sequence b owns the
    // CTAs from cu_q[b] / P + 2 b on: as many as the pages its tokens can touch,
    // found by bisection without any table of page counts.
    int b, j;
    if (p.cu_q == nullptr) {
        b = p.units == 1 ? (int)blockIdx.x : (int)blockIdx.x / p.units;
        j = (int)blockIdx.x - b * p.units;
    } else {
        int lo = 0, hi = p.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if ((min(max(p.cu_q[mid], 0), p.T) >> p.pshift) + 2 * mid <= (int)blockIdx.x) lo = mid;
            else hi = mid - 1;
        }
        b = lo;
        j = (int)blockIdx.x - ((min(max(p.cu_q[b], 0), p.T) >> p.pshift) + 2 * b);
    }
    const Seq s = sequence(p, b);
    if (s.n == 0) return;
    const int P = 1 << p.pshift, first = s.len - s.n;     // position of the first new token
    const int slot = (first >> p.pshift) + j;             // page of the sequence (rounded down)
    if (slot > (s.len - 1) >> p.pshift) return;           // past the last token: slot * P may not be an int
    const int lo = max(slot * P, first), hi = slot * P + min(P, s.len - slot * P);
    if (lo >= hi) return;                                 // also what negative j gives: nothing
    const bool stored = slot >= 0 && slot < p.width;
    const int page = stored ? p.page_table[(int64_t)b * p.table_stride + slot] : -1;
    const bool write = page >= 0 && page < p.pages;
    const int older = write ? lo - slot * P : 0;          // slots that hold older tokens

    // Without rows of q (PRE, G = 0) a CTA takes the keys or the values (blockIdx.z) of several heads, with one table.
    const bool apart = PRE && p.G == 0;
    const int tid = threadIdx.x, half = p.R >> 1;
    int head = apart ? (int)blockIdx.y * p.heads_each : (int)blockIdx.y;
    const int d0 = (tid % kRow) * 8, t_in = tid / kRow;
    const int j0 = FORM == kHalves ? (d0 >= half ? d0 - half : d0 + half) : 0;       // where the mates are
    const bool mated = FORM == kHalves && d0 < p.R;
    const int chunks = (hi - lo + kChunk - 1) / kChunk;
    int8_t *k_exp = p.k_exp + (int64_t)page * p.Hk + head, *v_exp = p.v_exp + (int64_t)page * p.Hk + head;
    const int was_k = older ? *k_exp : kExpMin, was_v = older ? *v_exp : kExpMin;
    int phase = 0;
    if constexpr (PRE) {
        for (int i = tid; i < 2 * D; i += THREADS) {
            const void *w = i < D ? p.q_norm : p.k_norm;
            weights[i / D][i % D] = w == nullptr ? 1.f : norm_weight(w, p.norm_dtype, i % D);
        }
        __syncthreads();
    }

    // Cosines and sines of tokens t0 .. t0 + nt.
    auto make_table = [&](int t0, int nt) {
        if (half == 0) return;
        __syncthreads();
        for (int i = tid; i < nt * half; i += THREADS) {
            const int t = i / half, jj = i - t * half;
            const int pos = PRE ? position_of(p, s.start + (t0 - first) + t, t0 + t, jj) : t0 + t;
            turn_of(p, pos, jj, table[i], table[p.table_tokens * half + i]);
        }
        __syncthreads();
    };
    // Token t0 + t_in of a set of rows; `pitch` from one of its vectors to the next.
    auto load = [&](Rows<FORM, kVecs> &r, const uint16_t *row, int64_t pitch, int nt, bool rotated) {
#pragma unroll
        for (int v = 0; v < kVecs; ++v, row += pitch) {
            const bool in = t_in + v * kStep < nt;
            r.own[v] = in ? load8<FORM>(row + d0) : make_uint4(0u, 0u, 0u, 0u);
            if constexpr (FORM == kHalves)
                if (rotated && mated && in) r.mate[v] = *reinterpret_cast<const uint4 *>(row + j0);
        }
    };
    auto turned = [&](const Rows<FORM, kVecs> &r, int v, const uint16_t *row, int t, float (&x)[8], int kind) {
        widen(r.own[v], x);
        const float *wt = weights[kind == kQuery ? 0 : 1];
        float norm = 1.f;
        if constexpr (PRE) {
            if ((kind == kQuery ? p.q_norm : p.k_norm) != nullptr) norm = row_norm<kRow>(x, p.eps, ((1u << kRow) - 1u) << (tid & 31 & ~(kRow - 1)));
            weigh(x, norm, wt + d0);
        }
        rotate<FORM, PRE>(p, row, d0, r.mate[FORM == kHalves ? v : 0], table + t * half, table + (p.table_tokens + t) * half, x,
                          norm, wt);
    };
    // Largest value over the CTA.
    auto reduce = [&](float m) {
        const uint32_t u = __reduce_max_sync(~0u, __float_as_uint(m));    // not negative: ordered like integers
        float *r = red[phase ^= 1];                       // two buffers: one barrier a reduction
        if ((tid & 31) == 0) r[tid >> 5] = __uint_as_float(u);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < THREADS / 32; ++i) m = fmaxf(m, r[i]);
        return m;
    };
    const uint16_t *k0 = p.k + (int64_t)s.start * p.k_token + head * p.k_head, *v0 = p.v + (int64_t)s.start * p.v_token + head * p.v_head;
    auto k_row = [&](int t0) { return k0 + (int64_t)(t0 - first + t_in) * p.k_token; };
    auto v_row = [&](int t0) { return v0 + (int64_t)(t0 - first + t_in) * p.v_token; };

    // K or V rows: the page's exponent, older codes moved to it if it grew, then codes.  With
    // one chunk `r` holds the rows; more are read again, first for the magnitude, then to store.
    auto write_rows = [&]<int kind>(std::integral_constant<int, kind>, Rows<FORM, kVecs> &r) {
        const int64_t pitch = (kind == kKey ? p.k_token : p.v_token) * kStep;
        float x[kVecs][8];
        auto values = [&](int c) {
            const int t0 = lo + c * kChunk, nt = min(kChunk, hi - t0);
            const uint16_t *row = kind == kKey ? k_row(t0) : v_row(t0);
            if (chunks > 1) {
                if (kind == kKey) make_table(t0, nt);
                load(r, row, pitch, nt, kind == kKey);
            }
#pragma unroll
            for (int v = 0; v < kVecs; ++v) {
                const int t = t_in + v * kStep;
                if (kind == kKey && t < nt) turned(r, v, row + v * pitch, t, x[v], kKey);
                else widen(r.own[v], x[v]);
            }
        };
        float m = 0.f;                                    // fmaxf leaves NaN out
        for (int c = 0; c < chunks; ++c) {
            values(c);
#pragma unroll
            for (int v = 0; v < kVecs; ++v)
#pragma unroll
                for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[v][i]));
        }
        const int was = apart ? (older ? *(kind == kKey ? k_exp : v_exp) : kExpMin) : (kind == kKey ? was_k : was_v);
        m = reduce(m);
        if (m == INFINITY) {                              // infinities count for nothing either
            m = 0.f;
            for (int c = 0; c < chunks; ++c) {
                if (chunks > 1) values(c);
#pragma unroll
                for (int v = 0; v < kVecs; ++v)
#pragma unroll
                    for (int i = 0; i < 8; ++i) m = fabsf(x[v][i]) < INFINITY ? fmaxf(m, fabsf(x[v][i])) : m;
            }
            m = reduce(m);
        }
        const int e = max(page_exponent(m), was);
        if (tid == 0) *(kind == kKey ? k_exp : v_exp) = (int8_t)e;
        uint8_t *cache = (kind == kKey ? p.k_cache : p.v_cache) + (int64_t)page * p.page_stride + (int64_t)head * p.head_stride;
        if (older != 0 && e != was) {
            const float scale = exp2_int(max(was - e, -126));
            for (int i = tid; i < older * kRow; i += THREADS) {          // 8 codes at a time
                uint2 *at = reinterpret_cast<uint2 *>(cache + (int64_t)i * 8);
                const uint2 v = *at;
                uint32_t in[2] = {v.x, v.y}, out[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    uint32_t l, h;
                    e4m3x4_to_f16x2(in[k], l, h);
                    const float2 a = __half22float2(*reinterpret_cast<__half2 *>(&l));
                    const float2 c = __half22float2(*reinterpret_cast<__half2 *>(&h));
                    out[k] = f32x4_to_e4m3x4(a.x * scale, a.y * scale, c.x * scale, c.y * scale);
                }
                *at = make_uint2(out[0], out[1]);
            }
        }
        const float scale = exp2_int(-e);
        const float2 ss = make_float2(scale, scale);
        for (int c = 0; c < chunks; ++c) {
            const int t0 = lo + c * kChunk, nt = min(kChunk, hi - t0);
            if (chunks > 1) values(c);
            uint8_t *to = cache + (t0 - slot * P + t_in) * D + d0;
#pragma unroll
            for (int v = 0; v < kVecs; ++v) {
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const float2 y = ptx::fmul2(make_float2(x[v][i], x[v][i + 1]), ss);
                    x[v][i] = y.x, x[v][i + 1] = y.y;
                }
                if (t_in + v * kStep < nt)
                    *reinterpret_cast<uint2 *>(to + v * kStep * D) = make_uint2(f32x4_to_e4m3x4(x[v][0], x[v][1], x[v][2], x[v][3]),
                                                                               f32x4_to_e4m3x4(x[v][4], x[v][5], x[v][6], x[v][7]));
            }
        }
    };

    Rows<FORM, kVecs> r[2];
    for (int c = 0; c < chunks; ++c) {
        const int t0 = lo + c * kChunk, nt = min(kChunk, hi - t0);
        // The rows in order K, V, the group's q; while one is in work the next are on their way.
        const int64_t tok0 = s.start + (t0 - first) + t_in;
        const uint16_t *q = p.q + tok0 * p.q_token + (int64_t)head * p.G * p.q_head;
        uint16_t *o = p.q_out + tok0 * p.o_token + (int64_t)head * p.G * p.o_head + d0;
        const bool keys = write && chunks == 1;
        if (apart) break;
        if (keys) load(r[0], k_row(t0), p.k_token * kStep, nt, true);
        make_table(t0, nt);
        if (keys) {
            load(r[1], v_row(t0), p.v_token * kStep, nt, false);
            write_rows(std::integral_constant<int, kKey>{}, r[0]);
        }
        load(r[0], q, p.q_token * kStep, nt, true);
        if (keys) write_rows(std::integral_constant<int, kValue>{}, r[1]);
        // A row's vectors lie in one warp and are all loaded before any is stored, so q may
        // be rotated in place.
        auto turn = [&](const Rows<FORM, kVecs> &x, int h) {
            __syncwarp();
#pragma unroll
            for (int v = 0; v < kVecs; ++v) {
                const int t = t_in + v * kStep;
                float y[8];
                if (t < nt) turned(x, v, q + h * p.q_head + v * kStep * p.q_token, t, y, kQuery);
                if (FORM == kAny) __syncwarp();
                if (t < nt) {
                    uint16_t *to = o + h * p.o_head + v * kStep * p.o_token;
                    const uint32_t w[4] = {f32x2_to_bf16x2(y[0], y[1]), f32x2_to_bf16x2(y[2], y[3]), f32x2_to_bf16x2(y[4], y[5]),
                                           f32x2_to_bf16x2(y[6], y[7])};
                    if constexpr (FORM != kAny) {
                        *reinterpret_cast<uint4 *>(to) = make_uint4(w[0], w[1], w[2], w[3]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) to[i] = (uint16_t)(w[i >> 1] >> (i & 1 ? 16 : 0));
                    }
                }
            }
        };
        for (int h = 0; h < p.G; h += 2) {
            if (h + 1 < p.G) load(r[1], q + (h + 1) * p.q_head, p.q_token * kStep, nt, true);
            turn(r[0], h);
            if (h + 2 < p.G) load(r[0], q + (h + 2) * p.q_head, p.q_token * kStep, nt, true);
            if (h + 1 < p.G) turn(r[1], h + 1);
        }
    }
    if constexpr (PRE) {
        if (apart) {
            if (!write) return;
            const int nt = hi - lo, last = min(head + p.heads_each, p.Hk);
            auto each = [&]<int kind>(std::integral_constant<int, kind> which) {
                const int64_t pitch = kind == kKey ? p.k_token : p.v_token, next = kind == kKey ? p.k_head : p.v_head;
                if (chunks == 1) {
                    load(r[0], kind == kKey ? k_row(lo) : v_row(lo), pitch * kStep, nt, kind == kKey);
                    if (kind == kKey) make_table(lo, nt);
                }
                while (head < last) {
                    if (chunks == 1 && head + 1 < last) load(r[1], (kind == kKey ? k_row(lo) : v_row(lo)) + next, pitch * kStep, nt, kind == kKey);
                    write_rows(which, r[0]);
                    r[0] = r[1];
                    ++head, ++k_exp, ++v_exp, k0 += p.k_head, v0 += p.v_head;
                }
            };
            if (blockIdx.z == 0) each(std::integral_constant<int, kKey>{});
            else each(std::integral_constant<int, kValue>{});
            return;
        }
    }
    if (write && chunks > 1) {
        write_rows(std::integral_constant<int, kKey>{}, r[0]);
        write_rows(std::integral_constant<int, kValue>{}, r[0]);
    }
}

template <int THREADS, int D, bool PRE>
cudaError_t launch(AppendArgs &p, int n, int64_t gx, cudaStream_t stream) {
    constexpr int kChunk = THREADS / (D / 8) * kVecsOf<THREADS>;
    const bool vec = p.qvec && p.kvec && p.vvec && p.ovec;
    const auto kernel = vec && p.interleaved && p.R % 8 == 0 ? kv_append_kernel<THREADS, D, kNeighbours, PRE>
                        : vec && !p.interleaved && p.R % 16 == 0 ? kv_append_kernel<THREADS, D, kHalves, PRE>
                                                                 : kv_append_kernel<THREADS, D, kAny, PRE>;
    p.table_tokens = std::min(std::min(n, p.P), kChunk);
    static_assert(kChunk * D * sizeof(float) <= 48 * 1024, "the table fits what a kernel may use without asking");
    const size_t smem = (size_t)p.table_tokens * (size_t)p.R * sizeof(float);
    if (PRE && p.G == 0) {                                // CTAs to fill the GPU a few times, of as many heads as leaves
        p.heads_each = (int)std::min<int64_t>(p.Hk, std::max<int64_t>(1, gx * p.Hk * 2 / kCtasToFill));
        return launch_pdl(kernel, dim3((unsigned)gx, (unsigned)((p.Hk + p.heads_each - 1) / p.heads_each), 2), dim3(THREADS), smem,
                          stream, (const AppendArgs)p);
    }
    return launch_pdl(kernel, dim3((unsigned)gx, (unsigned)p.Hk), dim3(THREADS), smem, stream, (const AppendArgs)p);
}

template <bool PRE>
cudaError_t launch_sized(AppendArgs &p, int n, int64_t gx, bool small, cudaStream_t stream) {
    if (p.D == 128)
        return small ? launch<kSmallThreads, 128, PRE>(p, n, gx, stream) : launch<kBigThreads, 128, PRE>(p, n, gx, stream);
    return small ? launch<kSmallThreads, 64, PRE>(p, n, gx, stream) : launch<kBigThreads, 64, PRE>(p, n, gx, stream);
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs &args, cudaStream_t stream) {
    AppendArgs p = args;
    p.G = p.Hq / p.Hk;
    p.n = p.cu_q == nullptr ? p.T / p.B : 0;
    p.pshift = 0;
    while ((1 << p.pshift) < p.P) ++p.pshift;
    const int n = p.cu_q == nullptr ? p.n : p.max_q;
    // CTAs for the pages a sequence's n tokens can touch.
    p.units = n == 1 ? 1 : (n - 1) / p.P + 2;
    const int64_t gx = p.cu_q == nullptr ? (int64_t)p.B * p.units : (int64_t)p.T / p.P + 2 * (int64_t)p.B;
    const bool small = std::min(n, p.P) * p.D <= kSmallThreads * kVecsOf<kSmallThreads> * 8;
    const bool pre = p.q_norm != nullptr || p.k_norm != nullptr || p.positions != nullptr;
    if (!pre) return launch_sized<false>(p, n, gx, small, stream);
    // With norms or positions the big CTAs take keys and values alone, and the rows of q go through the
    // 4-bit write's kernel, in a launch of their own: prompts of 64, 256, 1024 and 8001 tokens (32 heads of 128
    // over 8) take 14.0, 16.1, 19.1 and 72.9 us, 18.6, 23.6, 24.5 and 96.6 all in one.
    if (small) return launch_sized<true>(p, n, gx, small, stream);
    const cudaError_t e = launch_append_queries(args, stream);
    if (e != cudaSuccess) return e;
    p.G = 0;
    return launch_sized<true>(p, n, gx, small, stream);
}

}  // namespace lowbit
