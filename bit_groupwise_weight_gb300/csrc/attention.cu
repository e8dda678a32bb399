// attention.cu -- softmax attention of the new tokens' queries over the 8-bit
// paged cache (lowbit_attention), for few query rows a sequence, on the warp-level
// tensor cores.
//
// Mathematics.  Row r (query token i, head h) at position pos sees the keys
// t <= pos, t > pos - window (window > 0), t < len.  With codes Kc, Vc and page
// exponents ke, ve, in powers of two throughout:
//     s_t = scale log2(e) 2^ke(t) (q . Kc_t)
//     out = sum_t 2^s_t 2^ve(t) Vc_t / sum_t 2^s_t.
// The products run on the codes themselves: an e4m3 code is an fp16 number, so
// the dequantised operands are exact and one conversion instruction covers two
// of them; both scales are applied in fp32.  V's exponent goes into the softmax
// exponent, so that one weight serves the product:
//     w_t = 2^(s_t + ve(t) - m),  O += fp16(w_t) Vc_t,  l += w_t 2^-ve(t),
//     out = O / l,  lse = ln2 (m + log2 l),
// m following the maximum of s_t + ve(t) when that has outgrown it (attention.cuh): fp16
// holds w to 2^-11 of itself, or to 2^-32 of the row's largest where that is more, and
// most steps need neither a reduction over the warp nor a rescaling.  m, l, O are fp32.  q is multiplied by a power of two per row that puts its largest value
// into [2^10, 2^11): its 8 significant bits fit fp16's 11.
//
// A row that sees nothing has l = 0: out = 0, lse = -inf.  Masked scores are
// replaced, not added to, and V codes past a sequence's end are zeroed, so what
// a page holds there (NaN codes among it) does not reach the sums; a NaN in V that
// some rows of a slice see and others do not is handled apart (edge slices).
//
// Work split.  An item is (sequence, kv head, tile of 8 or 16 rows), the rows being
// the new tokens times the heads of the group; its keys come in tiles of 64.  All
// items' tiles form one list, each item's preceded by kItemCost units that stand for
// its other cost, and the list is cut into equal ranges, one per CTA: sequences of any
// lengths fill the machine evenly.  The CTAs of an item that cuts divide leave their
// parts' (m, l, O) in the workspace; the last of them, when its own range is done, waits
// for the others (which came before it in the grid, and leave their parts before they
// wait for any) and joins the parts.  A part's flag holds a
// number of the call's own, so that the workspace may come with any content, and is
// cleared by who reads it, so that a captured call may run again.  Items in many parts
// (few items, long ones) are joined by a second launch instead, many CTAs to an item: the
// 57 parts of each of 8 heads over 131001 keys cost 6 us more in one CTA, while for fewer
// parts the second launch costs more (3 us, most of it on the host).
//
// A CTA: one producer warp (TMA: K and V tile of 64 keys per stage, 128- or 64-byte
// swizzle; pages smaller than a tile take one copy each) and four consumer warps of
// 16 keys each with their own running (m, l, O), joined at the item's end.  The
// products are transposed, S^T = K q^T and O^T = V^T P^T: the 16 rows of the MMA's A
// operand are keys (values), its 8 columns query rows, so that a group of up to 8
// heads wastes nothing.
// Bound: HBM, 2 D bytes per key and kv head, for long sequences (one of 131001 keys, 8 kv
// heads of 128: 49.7 us, 5.4 TB/s, 0.80 of a copy's rate); for many and short ones what an item
// costs beside its tiles (queries, first tiles' latency, the join of the warps: some 6 tiles'
// time): 48 sequences of up to 8192 keys 25.5 us, 3.8 TB/s; 96 windows of 1000 keys of 64 values
// in pages of 16 17.5 us, 1.5 TB/s; one sequence of 257 keys 7.4 us, of which 5 are one
// launch's shortest.  (More CTAs of an SM for 64 values, four for three: 16.8 for 17.4 us, and
// 10.5 for 9.3 with few sequences.)
#include <algorithm>
#include <atomic>
#include <chrono>

#include "attention.cuh"

namespace lowbit {
namespace {

using namespace attn;

typedef unsigned long long u64;
constexpr int kTile = 64;                        // keys of a stage
constexpr int kWarps = 4;                        // consumer warps, 16 keys each
constexpr int kThreads = 32 * (kWarps + 1);
// What an item costs beside its tiles, in tiles: with 3 and 9 instead of 6, 48 sequences of up to
// 8192 keys take 26.8 and 25.9 us instead of 25.5, 96 windows of 1000 keys 16.9 and 18.4 instead of
// 17.3, one sequence of 257 keys 9.2 and 7.6 instead of 7.5, 7 sequences of 10 tokens 12.6 and 8.7
// instead of 8.6.
constexpr int kItemCost = 6;
// The least range of a CTA: 3 and 12 instead of 6 give 7.1 and 10.1 us for 257 keys, 18.6 and 19.7
// for 8 sequences of 5 tokens (18.7), 9.6 and 12.5 for a window of 3778 keys in one sequence (11.3);
// a step of it is a CTA more to wait for.
constexpr int kMinChunk = 6;
constexpr int kCtas = kSms * 3;                  // at most

__device__ unsigned int g_attn_timeouts;

// CTAs of an SM (what registers allow) and stages: about 150 KB of loads in flight.
template <int D, int ROWS>
constexpr int kPerSm = D == 128 && ROWS == 16 ? 2 : 3;
template <int D, int ROWS>
constexpr int kStages = D == 64 ? 6 : (ROWS == 16 ? 5 : 3);

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// Transpose of an 8 x 8 matrix of 16-bit values held one row per four lanes.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
// Bytes that hold an e4m3 NaN (0x7F or 0xFF), as 0x01 each.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t v) { return (((v & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7; }

// ---------------------------------------------------------------------------
// The list of tiles.

struct Seq : Span {
    int lo, nt;             // first key tile and number of tiles
    int rt;                 // row tiles; none for a sequence of the prompt kernel
    __device__ long long units(const AttentionArgs &p) const { return (long long)(kItemCost + nt) * (rt * p.Hk); }
};

template <int ROWS>
__device__ __forceinline__ Seq sequence(const AttentionArgs &p, int b) {
    Seq s;
    static_cast<Span &>(s) = span(p, b);
    const int n = s.n * p.G;
    s.lo = p.window > 0 ? max(s.len - s.n - p.window + 1, 0) / kTile : 0;
    s.nt = max((s.len + kTile - 1) / kTile - s.lo, 1);           // an empty sequence still writes its rows
    s.rt = n > p.few_rows ? 0 : (n + ROWS - 1) / ROWS;
    return s;
}

// A place in the list: sequence b, item (h, rt) and tile t of it (below 0: before its
// first tile); `before`: units of earlier sequences.
struct Place { int b, h, rt, t; long long before; };

// Moves pl forward to the place `idx`.
template <int ROWS>
__device__ __forceinline__ Seq locate(const AttentionArgs &p, long long idx, Place &pl) {
    Seq s = sequence<ROWS>(p, pl.b);
    while (idx - pl.before >= s.units(p) && pl.b + 1 < p.B) {
        pl.before += s.units(p);
        s = sequence<ROWS>(p, ++pl.b);
    }
    const uint32_t in = (uint32_t)(idx - pl.before), each = (uint32_t)(kItemCost + s.nt), item = in / each;
    pl.t = (int)(in - item * each) - kItemCost;
    pl.h = s.rt > 1 ? (int)item / s.rt : (int)item;
    pl.rt = (int)item - pl.h * s.rt;
    return s;
}

// A CTA's range of the list and the sequence in which it begins.  Each warp works it
// out by itself.
struct Plan { long long begin, end, chunk; Place pl; };

template <int ROWS>
__device__ __forceinline__ Plan make_plan(const AttentionArgs &p, int cta, int ctas) {
    const int lane = threadIdx.x & 31;
    auto weight = [&](int b) { return b < p.B ? sequence<ROWS>(p, b).units(p) : 0ll; };
    const long long w0 = weight(lane);
    long long total = w0;
    for (int b = lane + 32; b < p.B; b += 32) total += weight(b);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(~0u, total, o);
    Plan r;
    r.chunk = total <= (long long)ctas * kMinChunk ? kMinChunk : (total + ctas - 1) / ctas;
    r.begin = min((long long)cta * r.chunk, total);
    r.end = min(r.begin + r.chunk, total);
    r.pl = Place{0, 0, 0, 0, 0};
    if (r.begin >= r.end || p.B == 1) return r;
    for (int b0 = 0;; b0 += 32) {
        const long long w = b0 == 0 ? w0 : weight(b0 + lane);
        long long inc = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(~0u, inc, o);
            if (lane >= o) inc += v;
        }
        const unsigned hit = __ballot_sync(~0u, r.begin < r.pl.before + inc);
        if (hit != 0u || b0 + 32 >= p.B) {
            const int l = hit != 0u ? __ffs(hit) - 1 : 31;
            r.pl.b = min(b0 + l, p.B - 1);
            r.pl.before += __shfl_sync(~0u, inc - w, l);
            return r;
        }
        r.pl.before += __shfl_sync(~0u, inc, 31);
    }
}

// ---------------------------------------------------------------------------
// Shared memory of a CTA.

template <int D, int ROWS>
struct Smem {
    alignas(1024) uint8_t k[kStages<D, ROWS>][kTile * D];
    alignas(1024) uint8_t v[kStages<D, ROWS>][kTile * D];
    float o[kWarps][8][D + 4];                   // the warps' sums at an item's end, 8 rows at a time
    float m[kWarps][8], l[kWarps][8];
    int2 exps[kStages<D, ROWS>][kWarps];               // (ke, ve) of each 16 keys
    alignas(8) uint64_t full[kStages<D, ROWS>], empty[kStages<D, ROWS>];
};

// What the second launch needs to know of an item: written by the CTA that ends it, from
// CTA `begun` on (below 0: none).
struct Join { int begun, start, nrows, row0, h, pad; };
// More CTAs than this for each item that the page table allows: a second launch joins the parts.
// (By the last CTA always, 131001 keys take 55.6 us instead of 49.6; with 4 or 48 instead of 12 no
// measured case changes by more than 1.2 us.  The lengths may be far below the table's width, and
// the second launch is then for little: 66 keys take 5.6 us with a table of 2 pages, 9.6 with 2048.)
constexpr int kManyParts = 12;

// Workspace: a flag and a Join per CTA, then two slots per CTA: for the part of an item that it leaves
// to a later CTA (it leaves one at most), and for the part of the item that it joins
// itself.  A slot: ROWS x D sums, then ROWS (m, l) pairs.
__device__ __forceinline__ u64 *flag_of(const AttentionArgs &p, int cta) { return reinterpret_cast<u64 *>(p.workspace) + cta; }
__device__ __forceinline__ Join *join_of(const AttentionArgs &p, int cta) { return reinterpret_cast<Join *>(p.workspace + kCtas * 2) + cta; }
template <int D, int ROWS>
__device__ __forceinline__ float *slot_of(const AttentionArgs &p, int slot) {
    return p.workspace + kCtas * (2 + (int)sizeof(Join) / 4) + (int64_t)slot * (ROWS * (D + 2));
}
__device__ __forceinline__ u64 load_acquire(const u64 *at) {
    u64 v;
    asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(at) : "memory");
    return v;
}
__device__ __forceinline__ void store_release(u64 *at, u64 v) {
    asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(at), "l"(v) : "memory");
}

// Four values of a row's result.
__device__ __forceinline__ void write_row(const AttentionArgs &p, int start, int h, int row, int d, float4 o, float m, float l) {
    const int i = row / p.G, token = start + i, head = h * p.G + row - i * p.G;
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);          // NaN stays
    const uint32_t a = f32x2_to_bf16x2(o.x * inv, o.y * inv), c = f32x2_to_bf16x2(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2 *>(p.out + token * p.o_token + head * p.o_head + d) = make_uint2(a, c);
    if (d == 0 && p.lse != nullptr) p.lse[token * p.lse_token + head] = l == 0.f ? -INFINITY : kLn2 * (m + log2f(l));
}

// A consumer warp's state of an item.  Lane (g, t) = (lane / 4, lane % 4); column pair
// n: query rows 8n + 2t and 8n + 2t + 1.
template <int D, int ROWS>
struct State {
    static constexpr int KS = D / 16, N = ROWS / 8;
    uint32_t q[KS][N][2];                        // B fragments of q^T
    float qs[N][2];                              // factor of the row's scores
    int pos[N][2];
    float o[KS][N][4];                           // O^T: values 16c + 2g (+ 1) of the rows
    float m[N][2], l[N][2];
};

// One slice of 16 keys.  EDGE: some row does not see some key of it.
template <int D, int ROWS, bool EDGE>
__device__ __forceinline__ void slice(const AttentionArgs &p, State<D, ROWS> &st, uint32_t kat, uint32_t vat, int2 e, int key0,
                                      int len) {
    constexpr int KS = D / 16, N = ROWS / 8;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    // S^T: two chains of products for each column pair.
    float sc[N][2][4];
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < 8; ++i) sc[n][i >> 2][i & 3] = 0.f;
#pragma unroll
    for (int c = 0; c < KS; c += 2) {
        uint32_t r[4], a[8];
        ldsm_x4(kat ^ (c << 4), r);              // (keys 0-7, chunk c), (8-15, c), (0-7, c+1), (8-15, c+1)
#pragma unroll
        for (int i = 0; i < 4; ++i) e4m3x4_to_f16x2(r[i], a[2 * i], a[2 * i + 1]);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            ptx::mma_16816_f16(sc[n][0], a[0], a[2], a[1], a[3], st.q[c][n][0], st.q[c][n][1]);
            ptx::mma_16816_f16(sc[n][1], a[4], a[6], a[5], a[7], st.q[c + 1][n][0], st.q[c + 1][n][1]);
        }
    }
    const float kf = exp2_int(e.x), ve = (float)e.y;
    float x[N][4];
    uint32_t seen[N];                            // bit i: value i of the pair is seen
    bool grown = false;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        seen[n] = 0xFu;
        const float f0 = st.qs[n][0] * kf, f1 = st.qs[n][1] * kf;
#pragma unroll
        for (int i = 0; i < 4; ++i) {            // (key g, row 2t), (g, 2t+1), (g+8, 2t), (g+8, 2t+1)
            x[n][i] = fmaf(sc[n][0][i] + sc[n][1][i], i & 1 ? f1 : f0, ve);
            if constexpr (EDGE) {
                const int key = key0 + g + 8 * (i >> 1), pos = st.pos[n][i & 1];
                const bool see = key <= pos && (p.window == 0 || key > pos - p.window);
                if (!see) x[n][i] = -INFINITY, seen[n] &= ~(1u << i);
            }
        }
        grown |= fmaxf(x[n][0], x[n][2]) > st.m[n][0] + kPeak || fmaxf(x[n][1], x[n][3]) > st.m[n][1] + kPeak;
    }
    if (__any_sync(~0u, grown)) {                // rows whose maximum has outgrown m (the first keys seen: from -inf)
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float mx = fmaxf(x[n][c], x[n][c + 2]);
                mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 16));
                const float to = fmaxf(mx - kStart, st.m[n][c]);
                const Rescale by(to == st.m[n][c] ? 0.f : st.m[n][c] - to);
                const float a = by.of_o();
                st.m[n][c] = to;
                st.l[n][c] = by.of_l(st.l[n][c]);
#pragma unroll
                for (int k = 0; k < KS; ++k) st.o[k][n][c] *= a, st.o[k][n][c + 2] *= a;
            }
    }
    const bool deep = ve < kDeep;
    const float back = deep ? 0.f : exp2_int(-e.y);
    if (__builtin_expect(deep, 0)) {
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float ref = ve + (EDGE && st.m[n][c] == -INFINITY ? 0.f : st.m[n][c]);
                st.l[n][c] += ex2(x[n][c] - ref) + ex2(x[n][c + 2] - ref);
            }
    }
    uint32_t pb[N][2];                           // P^T: B fragments
#pragma unroll
    for (int n = 0; n < N; ++n) {
        // A row that has seen nothing has m = -inf; its scores are -inf as well.
        const float m0 = EDGE && st.m[n][0] == -INFINITY ? 0.f : st.m[n][0], m1 = EDGE && st.m[n][1] == -INFINITY ? 0.f : st.m[n][1];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[n][i] = ex2(x[n][i] - (i & 1 ? m1 : m0));
        st.l[n][0] = fmaf(x[n][0] + x[n][2], back, st.l[n][0]);
        st.l[n][1] = fmaf(x[n][1] + x[n][3], back, st.l[n][1]);
        pb[n][0] = transpose8(f32x2_to_f16x2(x[n][0], x[n][1]));
        pb[n][1] = transpose8(f32x2_to_f16x2(x[n][2], x[n][3]));
    }
    // V codes past the sequence's end are cleared (keys 2t, 2t+1 and 2t+8, 2t+9).
    uint32_t keep[2] = {~0u, ~0u};
    bool apart = false;                          // a NaN that not all rows see
    if constexpr (EDGE) {
        uint32_t nan = 0u;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int key = key0 + 8 * i + 2 * t;
            keep[i] = (key < len ? 0xFFFFu : 0u) | (key + 1 < len ? 0xFFFF0000u : 0u);
        }
#pragma unroll 1
        for (int c = 0; c < KS; c += 2) {
            uint32_t r[4];
            ldsm_x4_trans(vat ^ (c << 4), r);
            nan |= nan_bytes(r[0] & keep[0]) | nan_bytes(r[1] & keep[1]) | nan_bytes(r[2] & keep[0]) | nan_bytes(r[3] & keep[1]);
        }
        apart = __any_sync(~0u, nan != 0u);
    }
#pragma unroll
    for (int c = 0; c < KS; c += 2) {
        uint32_t r[4];
        ldsm_x4_trans(vat ^ (c << 4), r);
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            uint32_t a[4], bad[2] = {0u, 0u};
            if constexpr (EDGE) {
                r[i] &= keep[0], r[i + 1] &= keep[1];
                if (apart) {                     // NaN codes out, a flag (1.0 as e4m3) in their place
                    bad[0] = nan_bytes(r[i]) * 0x38u, bad[1] = nan_bytes(r[i + 1]) * 0x38u;
                    r[i] &= ~(nan_bytes(r[i]) * 0xFFu), r[i + 1] &= ~(nan_bytes(r[i + 1]) * 0xFFu);
                }
            }
            // Bytes (key, d), (key, d+1), (key+1, d), (key+1, d+1) -> key pairs of d and of d+1.
            e4m3x4_to_f16x2(ptx::prmt(r[i], 0u, 0x3120u), a[0], a[1]);
            e4m3x4_to_f16x2(ptx::prmt(r[i + 1], 0u, 0x3120u), a[2], a[3]);
#pragma unroll
            for (int n = 0; n < N; ++n)
                ptx::mma_16816_f16(st.o[c + (i >> 1)][n], a[0], a[1], a[2], a[3], pb[n][0], pb[n][1]);
            if constexpr (EDGE) {
                if (apart) {                     // rows that see a flagged key take NaN
                    uint32_t f[4];
                    e4m3x4_to_f16x2(ptx::prmt(bad[0], 0u, 0x3120u), f[0], f[1]);
                    e4m3x4_to_f16x2(ptx::prmt(bad[1], 0u, 0x3120u), f[2], f[3]);
#pragma unroll
                    for (int n = 0; n < N; ++n) {
                        float hits[4] = {0.f, 0.f, 0.f, 0.f};
                        const uint32_t s0 = (seen[n] & 1u ? 0x3C00u : 0u) | (seen[n] & 2u ? 0x3C000000u : 0u);
                        const uint32_t s1 = (seen[n] & 4u ? 0x3C00u : 0u) | (seen[n] & 8u ? 0x3C000000u : 0u);
                        ptx::mma_16816_f16(hits, f[0], f[1], f[2], f[3], transpose8(s0), transpose8(s1));
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (hits[k] > 0.f) st.o[c + (i >> 1)][n][k] = __int_as_float(0x7FFFFFFF);
                    }
                }
            }
        }
    }
}

template <int D, int ROWS>
__global__ void __launch_bounds__(kThreads, kPerSm<D, ROWS>)
    attention_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                     const AttentionArgs p) {
    constexpr int S = kStages<D, ROWS>, KS = D / 16, N = ROWS / 8;
    extern __shared__ uint8_t raw[];
    Smem<D, ROWS> &sm = *reinterpret_cast<Smem<D, ROWS> *>(raw + ((1024 - (ptx::smem_u32(raw) & 1023)) & 1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            ptx::mbar_init(ptx::smem_u32(&sm.full[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&sm.empty[i]), kWarps);
        }
        ptx::fence_mbar_init();
        ptx::prefetch_tensormap(&kmap);
        ptx::prefetch_tensormap(&vmap);
    }
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();
    const Plan plan = make_plan<ROWS>(p, blockIdx.x, gridDim.x);
    if (plan.begin >= plan.end) {
        if (p.defer && tid == 0) join_of(p, blockIdx.x)->begun = -1;
        return;
    }
    __syncthreads();
    Place pl = plan.pl;

    if (warp == kWarps) {
        // ------------- producer.  Lanes look up the pages of the next tiles (one
        // page, or one part of a large page, a lane) a window ahead of their use.
        const int pshift = p.pshift, page_keys = 1 << pshift;
        const int parts = page_keys < kTile ? kTile >> pshift : 1;       // pages of a tile
        const int pbits = page_keys < kTile ? 6 - pshift : 0, part = lane & (parts - 1);
        const int box = min(page_keys, kTile);
        const uint32_t off = (uint32_t)(part * box * D);
        int n_page = -1, n_row = 0, n_head = 0, n_ke = 0, n_ve = 0, n_tiles = 0;
        long long next = plan.begin;                                     // unit from which the next window's tiles are counted
        auto look_up = [&] {
            long long u = next;
            int i = lane >> pbits;                                       // this lane's tile of the window
            bool found = false;
            n_page = -1;                                                 // nothing to fetch
            while (u < plan.end) {
                const Seq s = locate<ROWS>(p, u, pl);
                const int t = max(pl.t, 0), left = (int)min((long long)(s.nt - t), plan.end - u - (t - pl.t));
                u += t - pl.t;
                if (i < left) {
                    u += i;
                    found = true;
                    const int key = (s.lo + t + i) * kTile + part * box;
                    n_head = pl.h;
                    n_row = key & (page_keys - 1);
                    if (key < s.len) {
                        n_page = p.page_table[(int64_t)pl.b * p.table_stride + (key >> pshift)];
                        if (n_page < 0) n_page = p.pages;                // outside the cache: read as zeros
                    }
                    break;
                }
                i -= max(left, 0);
                u += max(left, 0);
            }
            n_tiles = __popc(__ballot_sync(~0u, found)) >> pbits;
            next = __shfl_sync(~0u, u, 31) + 1;
        };
        auto look_up_exps = [&] {
            n_ke = n_ve = 0;
            if ((unsigned)n_page < (unsigned)p.pages) {
                n_ke = p.k_exp[(int64_t)n_page * p.Hk + n_head];
                n_ve = p.v_exp[(int64_t)n_page * p.Hk + n_head];
            }
        };
        look_up();
        look_up_exps();
        bool ok = true;
        int issued = 0, st = 0;
        uint32_t round = 1;                                              // parity of the stage's last release
        while (n_tiles > 0 && ok) {
            const int page = n_page, row = n_row, head = n_head, ke = n_ke, ve = n_ve, cnt = n_tiles;
            n_tiles = 0;
            if (cnt == 32 >> pbits && next < plan.end) look_up();
            for (int i = 0; i < cnt; ++i) {
                if (i == cnt / 2 && n_tiles > 0) look_up_exps();
                if (issued >= S)
                    ok = __all_sync(~0u, ptx::mbar_wait(ptx::smem_u32(&sm.empty[st]), round, &g_attn_timeouts));
                if (!ok) break;
                // The copies, then the exponents of the tile's four 16-key slices.
                const bool mine = (lane >> pbits) == i && page >= 0;
                const uint32_t bytes = __popc(__ballot_sync(~0u, mine)) * 2u * box * D;
                const uint32_t bar = ptx::smem_u32(&sm.full[st]);
                if (mine) {
                    ptx::tma_load_4d(ptx::smem_u32(sm.k[st]) + off, &kmap, 0, row, head, page, bar);
                    ptx::tma_load_4d(ptx::smem_u32(sm.v[st]) + off, &vmap, 0, row, head, page, bar);
                }
                const int src = (i << pbits) + ((lane & 3) * parts >> 2);
                const int ske = __shfl_sync(~0u, ke, src), sve = __shfl_sync(~0u, ve, src);
                if (lane < kWarps)
                    sm.exps[st][lane] = make_int2(min(max(ske, kExpMin), kExpMax), min(max(sve, kExpMin), kExpMax));
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_expect_tx(bar, bytes);
                ++issued;
                if (++st == S) st = 0, round ^= 1;
            }
        }
        for (int i = max(0, issued - S); i < issued; ++i)
            if (!ptx::mbar_wait(ptx::smem_u32(&sm.full[i % S]), (i / S) & 1, &g_attn_timeouts)) break;
        return;
    }

    // ---------------- consumers.
    const int g = lane >> 2, t = lane & 3;
    // ldmatrix addresses of the slice, without the chunk: the swizzle only flips bits
    // of the chunk number, so chunk c is at (address ^ c << 4).
    const int mkey = warp * 16 + ((lane >> 3) & 1) * 8 + (lane & 7);
    const uint32_t moff = mkey * D + (((lane >> 4) ^ (D == 128 ? mkey & 7 : (mkey >> 1) & 3)) << 4);
    bool ok = true;
    int st = 0;
    uint32_t round = 0;
    Join join{-1, 0, 0, 0, 0, 0};                                        // the item that this CTA ends and others began
    State<D, ROWS> a;
    for (long long idx = plan.begin; idx < plan.end;) {
        const Seq s = locate<ROWS>(p, idx, pl);
        const int units = (int)min((long long)(s.nt - pl.t), plan.end - idx);
        const int t0 = max(pl.t, 0), cnt = pl.t + units - t0;            // this CTA's tiles of the item
        const long long first_tile = idx - pl.t;                         // place of the item's first tile
        idx += units;
        if (cnt <= 0) continue;
        const int nrows = s.n * p.G, row0 = pl.rt * ROWS, first = s.len - s.n;

        // Query fragments: fp16, each row times a power of two.
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int r = row0 + 8 * n + g;
            const bool live = r < nrows;
            const int i = live ? r / p.G : 0, hq = pl.h * p.G + (live ? r - i * p.G : 0);
            const uint16_t *q = p.q + (int64_t)(s.start + i) * p.q_token + hq * p.q_head + 4 * t;
            uint2 v[KS];
            float amax = 0.f;
#pragma unroll
            for (int c = 0; c < KS; ++c) v[c] = live ? *reinterpret_cast<const uint2 *>(q + 16 * c) : make_uint2(0u, 0u);
#pragma unroll
            for (int c = 0; c < KS; ++c) {
                const float x[4] = {bf16_lo(v[c].x), bf16_hi(v[c].x), bf16_lo(v[c].y), bf16_hi(v[c].y)};
#pragma unroll
                for (int k = 0; k < 4; ++k) amax = fabsf(x[k]) < INFINITY ? fmaxf(amax, fabsf(x[k])) : amax;
            }
            amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 2));
            const int up = query_shift(amax);
            const float f = exp2_int(up), scale = exp2_int(-up) * p.scale_log2;
#pragma unroll
            for (int c = 0; c < KS; ++c) {
                a.q[c][n][0] = f32x2_to_f16x2(bf16_lo(v[c].x) * f, bf16_hi(v[c].x) * f);
                a.q[c][n][1] = f32x2_to_f16x2(bf16_lo(v[c].y) * f, bf16_hi(v[c].y) * f);
            }
            // This lane's columns are rows 2t and 2t + 1.
            const int position = live ? first + i : -1;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                a.qs[n][c] = __shfl_sync(~0u, scale, 8 * t + 4 * c);
                a.pos[n][c] = __shfl_sync(~0u, position, 8 * t + 4 * c);
                a.m[n][c] = -INFINITY, a.l[n][c] = 0.f;
            }
#pragma unroll
            for (int c = 0; c < KS; ++c) a.o[c][n][0] = a.o[c][n][1] = a.o[c][n][2] = a.o[c][n][3] = 0.f;
        }
        const int pos_lo = first + row0 / p.G, pos_hi = first + (min(row0 + ROWS, nrows) - 1) / p.G;

        int key0 = (s.lo + t0) * kTile + warp * 16;
        for (int tile = 0; tile < cnt; ++tile, key0 += kTile) {
            if (ok) ok = ptx::mbar_wait(ptx::smem_u32(&sm.full[st]), round, &g_attn_timeouts);
            const uint32_t kat = ptx::smem_u32(sm.k[st]) + moff, vat = ptx::smem_u32(sm.v[st]) + moff;
            if (key0 + 15 <= pos_lo && (p.window == 0 || key0 > pos_hi - p.window))
                slice<D, ROWS, false>(p, a, kat, vat, sm.exps[st][warp], key0, s.len);
            else if (key0 <= pos_hi && (p.window == 0 || key0 + 15 > pos_lo - p.window))
                slice<D, ROWS, true>(p, a, kat, vat, sm.exps[st][warp], key0, s.len);
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sm.empty[st]));
            if (++st == S) st = 0, round ^= 1;
        }

        // The warps' parts of the item are joined in shared memory, 8 rows at a time.
        const bool continued = t0 > 0, unfinished = t0 + cnt < s.nt;
        float *slot = slot_of<D, ROWS>(p, 2 * (int)blockIdx.x + (unfinished ? 0 : 1));
        if (continued && !unfinished) join = Join{(int)(first_tile / plan.chunk), s.start, nrows, row0, pl.h, 0};
#pragma unroll
        for (int n = 0; n < N; ++n) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) a.l[n][c] += __shfl_xor_sync(~0u, a.l[n][c], o);
                if (g == 0) sm.m[warp][2 * t + c] = a.m[n][c], sm.l[warp][2 * t + c] = a.l[n][c];
#pragma unroll
                for (int k = 0; k < KS; ++k)                              // values 16k + 2g, + 1 of the row
                    *reinterpret_cast<float2 *>(&sm.o[warp][2 * t + c][16 * k + 2 * g]) = make_float2(a.o[k][n][c], a.o[k][n][c + 2]);
            }
            ptx::named_sync(1, kWarps * 32);
            for (int i = tid; i < 8 * (D / 4); i += kWarps * 32) {
                const int r = i / (D / 4), d = (i % (D / 4)) * 4, row = row0 + 8 * n + r;
                if (row >= nrows) break;
                float mm = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sm.m[w][r]);
                const float ref = mm == -INFINITY ? 0.f : mm;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                float ll = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const Rescale by(sm.m[w][r] - ref);
                    const float f = by.of_o();
                    const float4 v = *reinterpret_cast<const float4 *>(&sm.o[w][r][d]);
                    acc.x = fmaf(f, v.x, acc.x), acc.y = fmaf(f, v.y, acc.y);
                    acc.z = fmaf(f, v.z, acc.z), acc.w = fmaf(f, v.w, acc.w);
                    ll += by.of_l(sm.l[w][r]);
                }
                if (continued || unfinished) {
                    *reinterpret_cast<float4 *>(slot + (8 * n + r) * D + d) = acc;
                    if (d == 0) *reinterpret_cast<float2 *>(slot + ROWS * D + 2 * (8 * n + r)) = make_float2(mm, ll);
                } else {
                    write_row(p, s.start, pl.h, row, d, acc, mm, ll);
                }
            }
            ptx::named_sync(1, kWarps * 32);
        }
        if (unfinished && !p.defer) {                                    // nothing follows in this CTA's range
            __threadfence();
            ptx::named_sync(1, kWarps * 32);
            if (tid == 0) store_release(flag_of(p, blockIdx.x), p.call);
        }
    }
    if (p.defer && tid == 0) *join_of(p, blockIdx.x) = join;
    if (p.defer || join.begun < 0) return;

    // The parts of the CTAs before this one have to be there.
    for (int c = join.begun + tid; c < (int)blockIdx.x; c += kWarps * 32) {
        const u64 t0 = ptx::globaltimer_ns();
        while (load_acquire(flag_of(p, c)) != p.call)
            if (ptx::globaltimer_ns() - t0 > ptx::kWaitLimitNs) {
                atomicAdd(&g_attn_timeouts, 1u);
                break;
            }
        *flag_of(p, c) = 0;
    }
    ptx::named_sync(1, kWarps * 32);
    // A thread joins kPer groups of four values; their loads of several parts go out together.
    constexpr int kPer = ROWS * (D / 4) / (kWarps * 32);
    float m[kPer], l[kPer];
    float4 o[kPer];
    int r[kPer];
    const int d = tid % (D / 4) * 4;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
        r[q] = (tid + q * kWarps * 32) / (D / 4);
        m[q] = -INFINITY, l[q] = 0.f, o[q] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll(8 / kPer)
    for (int c = join.begun; c <= (int)blockIdx.x; ++c) {
        const float *part = slot_of<D, ROWS>(p, 2 * c + (c == (int)blockIdx.x));
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
            const float2 ml = __ldcg(reinterpret_cast<const float2 *>(part + ROWS * D + 2 * r[q]));
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(part + r[q] * D + d));
            const float mx = fmaxf(m[q], ml.x), base = mx == -INFINITY ? 0.f : mx;
            const Rescale old(m[q] - base), add(ml.x - base);
            const float e = old.of_o(), f = add.of_o();
            o[q].x = o[q].x * e + v.x * f, o[q].y = o[q].y * e + v.y * f;
            o[q].z = o[q].z * e + v.z * f, o[q].w = o[q].w * e + v.w * f;
            l[q] = old.of_l(l[q]) + add.of_l(ml.y);
            m[q] = mx;
        }
    }
#pragma unroll
    for (int q = 0; q < kPer; ++q)
        if (join.row0 + r[q] < join.nrows) write_row(p, join.start, join.h, join.row0 + r[q], d, o[q], m[q], l[q]);
}

// The second launch: block (c, r) takes row r of the item that CTA c ends.
template <int D, int ROWS>
__global__ void __launch_bounds__(128) attention_join_kernel(const AttentionArgs p) {
    constexpr int kGroups = 128 / (D / 4);                       // parts read at a time
    __shared__ float4 so[kGroups][D / 4];
    __shared__ float2 sml[kGroups];
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();
    const int c = blockIdx.x, r = blockIdx.y;
    const Join join = *join_of(p, c);
    if (join.begun < 0 || join.row0 + r >= join.nrows) return;
    const int grp = threadIdx.x / (D / 4), d = (threadIdx.x % (D / 4)) * 4;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float pm, float pl, float4 po) {
        const float mx = fmaxf(m, pm), ref = mx == -INFINITY ? 0.f : mx;
        const Rescale old(m - ref), more(pm - ref);
        const float a = old.of_o(), b = more.of_o();
        o.x = o.x * a + po.x * b, o.y = o.y * a + po.y * b, o.z = o.z * a + po.z * b, o.w = o.w * a + po.w * b;
        l = old.of_l(l) + more.of_l(pl);
        m = mx;
    };
#pragma unroll 4
    for (int i = join.begun + grp; i <= c; i += kGroups) {
        const float *slot = slot_of<D, ROWS>(p, 2 * i + (i == c));
        const float2 ml = *reinterpret_cast<const float2 *>(slot + ROWS * D + 2 * r);
        add(ml.x, ml.y, *reinterpret_cast<const float4 *>(slot + r * D + d));
    }
    so[grp][d / 4] = o;
    if (d == 0) sml[grp] = make_float2(m, l);
    __syncthreads();
    if (grp == 0) {
#pragma unroll
        for (int k = 1; k < kGroups; ++k) add(sml[k].x, sml[k].y, so[k][d / 4]);
        write_row(p, join.start, join.h, join.row0 + r, d, o, m, l);
    }
}

template <int D, int ROWS>
cudaError_t launch(const AttentionArgs &args, cudaStream_t stream) {
    AttentionArgs p = args;
    const uint32_t box_rows = (uint32_t)std::min(p.P, kTile);
    const uint64_t dims[4] = {(uint64_t)D, (uint64_t)p.P, (uint64_t)p.Hk, (uint64_t)p.pages};
    const uint64_t strides[3] = {(uint64_t)D, (uint64_t)p.head_stride, (uint64_t)p.page_stride};
    const uint32_t box[4] = {(uint32_t)D, box_rows, 1, 1};
    const CUtensorMapSwizzle sw = D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    CUtensorMap kmap, vmap;
    if (!encode_tiled(&kmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, p.k_cache, dims, strides, box, sw) ||
        !encode_tiled(&vmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, p.v_cache, dims, strides, box, sw))
        return cudaErrorInvalidValue;
    const int smem = (int)sizeof(Smem<D, ROWS>) + 1024;
    cudaError_t e = raise_smem_limit((const void *)attention_kernel<D, ROWS>, current_device(), smem);
    if (e != cudaSuccess) return e;
    // No more CTAs than ranges of kMinChunk that the page table allows.
    const int rows_max = (int)std::min<int64_t>((int64_t)p.max_q * p.G, p.few_rows);
    const int64_t items = (int64_t)p.B * p.Hk * ((rows_max + ROWS - 1) / ROWS);
    const int64_t tiles = ((int64_t)p.width * p.P + kTile - 1) / kTile;
    const int ctas = (int)std::min<int64_t>(kSms * kPerSm<D, ROWS>, std::max<int64_t>(1, (items * (kItemCost + tiles) + kMinChunk - 1) / kMinChunk));
    p.defer = ctas > kManyParts * items;
    e = launch_pdl(attention_kernel<D, ROWS>, dim3(ctas), dim3(kThreads), smem, stream, kmap, vmap, (const AttentionArgs)p);
    if (e != cudaSuccess || !p.defer) return e;
    return launch_pdl(attention_join_kernel<D, ROWS>, dim3(ctas, ROWS), dim3(128), 0, stream, (const AttentionArgs)p);
}

// Which kernels a call needs: sequences are sorted by their number of query rows (new
// tokens times heads of a group), on the device when the host does not know it.  Where the two
// cross depends on how much else there is: for 16, 32, 48, 64, 96 and 128 rows a sequence this kernel
// and the prompt kernel (from 32 on) take, in us,
//   8 x 6000 keys of 128 values: 29, 45, 61, 75, 106, 136 and 56, 57, 57, 58, 59;
//   8 x 6000 keys of 64:         18, 25, 34, 43, 59, 75 and 53, 53, 53, 54, 55;
//   1 x 8000 keys of 128:        14, 17, 20, 22, 26, 31 and 32, 33, 33, 35, 35;
//   1 x 300 keys of 128:         10, 11, 11, 11, 12, 12 and 13, 13, 13, 13, 13.
// 64 lies between: full batches of 128 values would cross at 45, of 64 values at 90, single
// sequences at 150.
constexpr int kFewRows = 64;
struct Kernels { bool few, many; int few_rows; };
Kernels kernels_for(int max_q, bool uniform, int G) {
    if ((int64_t)max_q * G <= kFewRows) return {true, false, kFewRows};
    return {!uniform, true, uniform ? 0 : kFewRows};
}

size_t few_workspace_bytes(int max_q, int G, int D) {
    const int rows = (int64_t)max_q * G <= 8 ? 8 : 16;
    return (size_t)kCtas * (sizeof(u64) + sizeof(Join) + 2 * rows * (D + 2) * sizeof(float));
}

}  // namespace

uint32_t attention_timeouts(bool reset) {
    const uint32_t prompt = prompt_timeouts(reset);
    unsigned int v = 0;
    cudaMemcpyFromSymbol(&v, g_attn_timeouts, sizeof(v));
    if (reset) {
        const unsigned int zero = 0;
        cudaMemcpyToSymbol(g_attn_timeouts, &zero, sizeof(zero));
    }
    return v + prompt;
}

size_t attention_workspace_bytes(int64_t T, int B, int max_q, bool uniform, int Hq, int Hk, int D, int64_t max_len) {
    const Kernels k = kernels_for(max_q, uniform, Hq / Hk);
    size_t bytes = k.few ? few_workspace_bytes(max_q, Hq / Hk, D) : 0;
    if (k.many) bytes += prompt_workspace_bytes(prompt_grid(T, B, max_q, uniform, Hq, Hk, max_len), Hk, D);
    return std::max<size_t>(bytes, 16);
}

cudaError_t launch_attention(const AttentionArgs &args, cudaStream_t stream) {
    AttentionArgs p = args;
    const bool uniform = p.cu_q == nullptr;
    p.G = p.Hq / p.Hk;
    p.n = uniform ? p.T / p.B : 0;
    if (uniform) p.max_q = p.n;
    p.pshift = 0;
    while ((1 << p.pshift) < p.P) ++p.pshift;
    const Kernels k = kernels_for(p.max_q, uniform, p.G);
    p.few_rows = k.few_rows;
    // A number that no other call's flags hold, and no other content of the workspace is likely to.
    static std::atomic<u64> calls{(u64)std::chrono::steady_clock::now().time_since_epoch().count() * 0x9E3779B97F4A7C15ull};
    p.call = calls.fetch_add(1, std::memory_order_relaxed) | 1ull << 63;
    if (k.many) {
        PromptGrid g = prompt_grid(p.T, p.B, p.max_q, uniform, p.Hq, p.Hk, (int64_t)p.width * p.P);
        g.workspace = k.few ? (int64_t)(few_workspace_bytes(p.max_q, p.G, p.D) / sizeof(float)) : 0;
        const cudaError_t e = launch_prompt(p, g, stream);
        if (e != cudaSuccess || !k.few) return e;
    }
    const bool half = (int64_t)p.max_q * p.G <= 8;
    if (p.D == 128) return half ? launch<128, 8>(p, stream) : launch<128, 16>(p, stream);
    return half ? launch<64, 8>(p, stream) : launch<64, 16>(p, stream);
}

}  // namespace lowbit
