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
#include <atomic>
#include <chrono>

#include "attention_few.cuh"

namespace lowbit {
namespace {

// Bytes that hold an e4m3 NaN (0x7F or 0xFF), as 0x01 each.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t v) { return (((v & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7; }


// The 8-bit cache.
struct Eight {
    static constexpr int kTile = 64, kTileBits = 6, kWarpKeys = 16;       // keys of a stage, of a warp
    // What an item costs beside its tiles, in tiles: with 3 and 9 instead of 6, 48 sequences of up to
    // 8192 keys take 26.8 and 25.9 us instead of 25.5, 96 windows of 1000 keys 16.9 and 18.4 instead of
    // 17.3, one sequence of 257 keys 9.2 and 7.6 instead of 7.5, 7 sequences of 10 tokens 12.6 and 8.7
    // instead of 8.6.
    static constexpr int kItemCost = 6;
    // The least range of a CTA: 3 and 12 instead of 6 give 7.1 and 10.1 us for 257 keys, 18.6 and 19.7
    // for 8 sequences of 5 tokens (18.7), 9.6 and 12.5 for a window of 3778 keys in one sequence (11.3);
    // a step of it is a CTA more to wait for.
    static constexpr int kMinChunk = 6;
    // CTAs of an SM (what registers allow) and stages: about 150 KB of loads in flight.
    static constexpr int per_sm(int D, int ROWS) { return D == 128 && ROWS == 16 ? 2 : 3; }
    static constexpr int stages(int D, int ROWS) { return D == 64 ? 6 : (ROWS == 16 ? 5 : 3); }
    static constexpr int kCtas = kSms * 3;                                // at most
    static constexpr bool kHold = false;                                   // the list in shared memory during tiles
    static constexpr float kUnit = 1.f;                                   // what a value of V counts in the product
    template <int D>
    static constexpr int kKeyBytes = 2 * D;                               // of K and V

    struct Maps { CUtensorMap k, v; };
    template <int D>
    struct Stage {
        alignas(1024) uint8_t k[kTile * D];
        alignas(1024) uint8_t v[kTile * D];
    };
    struct StageBeside { int2 e[kWarps]; };                               // (ke, ve) of each 16 keys
    struct Beside { int ke, ve; };                                        // of the page that a lane looks up

    static __device__ __forceinline__ void prefetch(const Maps &m) {
        ptx::prefetch_tensormap(&m.k);
        ptx::prefetch_tensormap(&m.v);
    }
    static __device__ __forceinline__ Beside beside(const AttentionArgs &p, int page, int head) {
        if ((unsigned)page >= (unsigned)p.pages) return {0, 0};
        return {p.k_exp[(int64_t)page * p.Hk + head], p.v_exp[(int64_t)page * p.Hk + head]};
    }
    template <int D>
    static __device__ __forceinline__ void copy(const Maps &m, Stage<D> &s, int part, int box, int row, int head, int page,
                                                uint32_t bar) {
        ptx::tma_load_4d(ptx::smem_u32(s.k) + part * box * D, &m.k, 0, row, head, page, bar);
        ptx::tma_load_4d(ptx::smem_u32(s.v) + part * box * D, &m.v, 0, row, head, page, bar);
    }
    // Exponents of the tile whose pages lanes `first` and on have looked up, `parts` of them.
    static __device__ __forceinline__ void put_beside(StageBeside &s, const Beside &b, int first, int parts) {
        const int lane = threadIdx.x & 31, src = first + ((lane & 3) * parts >> 2);
        const int ke = __shfl_sync(~0u, b.ke, src), ve = __shfl_sync(~0u, b.ve, src);
        if (lane < kWarps) s.e[lane] = make_int2(min(max(ke, kExpMin), kExpMax), min(max(ve, kExpMin), kExpMax));
    }

    // A lane's ldmatrix address in the slice, without the chunk: the swizzle only flips bits
    // of the chunk number, so chunk c is at (address ^ c << 4).
    template <int D>
    struct Lane {
        int warp;
        uint32_t off;
        __device__ __forceinline__ Lane(const AttentionArgs &, int w) : warp(w) {
            const int lane = threadIdx.x & 31, key = warp * 16 + ((lane >> 3) & 1) * 8 + (lane & 7);
            off = key * D + (((lane >> 4) ^ (D == 128 ? key & 7 : (key >> 1) & 3)) << 4);
        }
    };

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

    template <int D, int ROWS>
    struct Queries {};
    // Where a lane's sums o[k] stand: values value_of(k, g) and the next one.
    static __device__ __forceinline__ int value_of(int k, int g) { return 16 * k + 2 * g; }

    // Query fragments of an item's rows: fp16, each row times a power of two.
    template <int D, int ROWS>
    static __device__ __forceinline__ void queries(const AttentionArgs &p, State<D, ROWS> &a, const Seq &s, int h, int row0,
                                                   Queries<D, ROWS> &) {
        constexpr int KS = D / 16, N = ROWS / 8;
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, nrows = s.n * p.G, first = s.len - s.n;
                #pragma unroll
                for (int n = 0; n < N; ++n) {
                    const int r = row0 + 8 * n + g;
                    const bool live = r < nrows;
                    const int i = live ? r / p.G : 0, hq = h * p.G + (live ? r - i * p.G : 0);
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
    }

    // One slice of 16 keys.  EDGE: some row does not see some key of it.
    template <int D, int ROWS, bool EDGE>
    static __device__ __forceinline__ void slice(const AttentionArgs &p, State<D, ROWS> &st, const Lane<D> &at, const Stage<D> &stage,
                                                 const StageBeside &beside, int key0, int len) {
        constexpr int KS = D / 16, N = ROWS / 8;
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const uint32_t kat = ptx::smem_u32(stage.k) + at.off, vat = ptx::smem_u32(stage.v) + at.off;
        const int2 e = beside.e[at.warp];
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
            grown |= fmaxf(x[n][0], x[n][2]) - st.m[n][0] > kPeak || fmaxf(x[n][1], x[n][3]) - st.m[n][1] > kPeak;
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

    template <int D>
    static bool make_maps(const AttentionArgs &p, Maps *m) {
        const uint32_t box_rows = (uint32_t)std::min(p.P, kTile);
        const uint64_t dims[4] = {(uint64_t)D, (uint64_t)p.P, (uint64_t)p.Hk, (uint64_t)p.pages};
        const uint64_t strides[3] = {(uint64_t)D, (uint64_t)p.head_stride, (uint64_t)p.page_stride};
        const uint32_t box[4] = {(uint32_t)D, box_rows, 1, 1};
        const CUtensorMapSwizzle sw = D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
        return encode_tiled(&m->k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, p.k_cache, dims, strides, box, sw) &&
               encode_tiled(&m->v, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, p.v_cache, dims, strides, box, sw);
    }
};

// Which kernels a call needs: sequences are sorted by their number of query rows (new
// tokens times heads of a group), on the device when the host does not know it.  Where the two
// cross depends on how much else there is: for 16, 32, 48, 64, 96 and 128 rows a sequence this kernel
// and the prompt kernel (from 32 on) take, in us,
//   8 x 6000 keys of 128 values: 29, 45, 61, 75, 106, 136 and 56, 57, 57, 58, 59;
//   8 x 6000 keys of 64:         18, 25, 34, 43, 59, 75 and 53, 53, 53, 54, 55;
//   1 x 8000 keys of 128:        14, 17, 20, 22, 26, 31 and 32, 33, 33, 35, 35;
//   1 x 300 keys of 128:         10, 11, 11, 11, 12, 12 and 13, 13, 13, 13, 13.
// 64 lies between: full batches of 128 values would cross at 45, of 64 values at 90, single
// sequences at 150.  Over a 4-bit cache, for 16, 32, 48, 64, 96 and 128 rows:
//   8 x 6000 keys of 128 values: 26, 39, 52, 67, 94, 121 and 53, 54, 55, 56, 58, 59;
//   8 x 6000 keys of 64:         19, 27, 36, 44, 60, 77 and 49, 50, 51, 51, 52, 52;
//   1 x 8000 keys of 128:        14, 17, 20, 21, 25, 29 and 30, 32, 33, 34, 35, 36;
//   1 x 300 keys of 128:         9, 10, 10, 10, 10, 11 and 12, 13, 13, 13, 13, 13;
// so that full batches (of sequences times kv heads) of 128 values take 48.  Between one and eight sequences, and for
// full batches of short ones, nothing was measured: single sequences behind long caches would cross past 128.
constexpr int kFewRows = 64, kFewRowsFull4 = 48, kFullBatch = 64;
struct Kernels { bool few, many; int few_rows; };
Kernels kernels_for(int max_q, bool uniform, int B, int Hq, int Hk, int D, bool four) {
    const int few_rows = four && D == 128 && (int64_t)B * Hk >= kFullBatch ? kFewRowsFull4 : kFewRows;
    if ((int64_t)max_q * (Hq / Hk) <= few_rows) return {true, false, few_rows};
    return {!uniform, true, uniform ? 0 : few_rows};
}

size_t few_workspace_bytes(int max_q, int G, int D, bool four) {
    return four ? attention4_workspace_bytes(max_q, G, D) : few_rows_workspace<Eight>(max_q, G, D);
}

}  // namespace

uint32_t attention_timeouts(bool reset) {
    const uint32_t prompt = prompt_timeouts(reset);
    return few_rows_timeouts(reset) + attention4_timeouts(reset) + prompt;
}

size_t attention_workspace_bytes(int64_t T, int B, int max_q, bool uniform, int Hq, int Hk, int D, int64_t max_len, bool four) {
    const Kernels k = kernels_for(max_q, uniform, B, Hq, Hk, D, four);
    size_t bytes = k.few ? few_workspace_bytes(max_q, Hq / Hk, D, four) : 0;
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
    const Kernels k = kernels_for(p.max_q, uniform, p.B, p.Hq, p.Hk, p.D, p.k_scale != nullptr);
    p.few_rows = k.few_rows;
    // A number that no other call's flags hold, and no other content of the workspace is likely to.
    static std::atomic<u64> calls{(u64)std::chrono::steady_clock::now().time_since_epoch().count() * 0x9E3779B97F4A7C15ull};
    p.call = calls.fetch_add(1, std::memory_order_relaxed) | 1ull << 63;
    if (k.many) {
        PromptGrid g = prompt_grid(p.T, p.B, p.max_q, uniform, p.Hq, p.Hk, (int64_t)p.width * p.P);
        g.workspace = k.few ? (int64_t)(few_workspace_bytes(p.max_q, p.G, p.D, p.k_scale != nullptr) / sizeof(float)) : 0;
        const cudaError_t e = launch_prompt(p, g, stream);
        if (e != cudaSuccess || !k.few) return e;
    }
    return p.k_scale != nullptr ? launch_attention4(p, stream) : launch_few_rows<Eight>(p, stream);
}

}  // namespace lowbit
