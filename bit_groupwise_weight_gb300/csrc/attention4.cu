// attention4.cu -- attention over the 4-bit paged cache for few query rows a sequence: what
// attention_few.cuh needs to know of the format (int4.cuh).
//
// Mathematics, beside attention.cu's.  A key's value is (c - 8) s, s the scale of its group of 32
// values, so
//     q . k = sum over groups of s (q . c - 8 sum q),
// and the products run on the codes c alone, groups apart: masking two nibbles out of a word of
// eight leaves a pair of fp16 subnormals c 2^-24 (c 2^-20 for the second nibble of a byte, whose q
// is held 2^4 smaller instead), exact, one instruction for two codes.  Scales are applied to the groups'
// sums in fp32.  The offsets, s times -8 sum q, are a product of their own for all groups at once: scales are
// fp16 numbers, and a sum is three of them (33 bits).
// In the product with V the groups run along the rows of the result and the scales along the sum:
// there codes become values first.  A nibble in the mantissa of 1.0 is 1 + c / 64, and
//     (1 + c / 64) s - 1.125 s = (c - 8) s / 64,
// one fused operation for two codes, exact in fp16 (3 + 3 bits) for every scale.  The result is
// multiplied by 64 at the end.
//
// Operands: the four bytes that a lane gets from ldmatrix are eight codes of one key (K), or, transposed,
// four codes of two neighbouring keys (V): the order of the values within a group is the codes' own,
// q is laid out to match, and a lane's four rows of the result are four neighbouring values.
//
// A stage is 128 keys, a warp's share 32 of them in two halves: softmax bookkeeping and the loop's own cost are
// paid once for both.
// Bound: no unit is full.  One sequence of 131001 keys takes 38 us, 3.8 TB/s, 0.56 of a copy's rate (21.3 us would be the
// bytes'), with 0.57 instructions issued a cycle and scheduler and the ALU (masks, shifts) at 0.52: each of the three consumer
// warps of a scheduler goes through one chain of dependent steps a slice (stage, K's products, scales, maximum, weights,
// transposition, V's products), and begins none of the next slice before.  The number of stages does not matter (2: the
// same), registers do: what only the list needs is in shared memory while a warp goes through its tiles (40.3 us without).
// q's fragments there too, and four CTAs an SM with 96 registers, were no faster (with 16 rows the first is).  64 sequences of
// up to 16001 keys 35.8 us; 96 windows of 1000 keys of 64 values in pages of 16 19.7; 8 sequences of 5 tokens, 28 heads over 4,
// 18.6: what an item costs beside its tiles, as for the 8-bit cache.  One sequence of 257 keys 6.3 us.
#include <type_traits>

#include "attention_few.cuh"
#include "int4.cuh"

namespace lowbit {
namespace {

__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// The values / 64 of nibble I of both halves of w; s, t: the halves' scales, and -1.125 of them.
template <int I>
__device__ __forceinline__ uint32_t values4(uint32_t w, uint32_t s, uint32_t t) {
    const uint32_t in = I == 0 ? w << 4 : w >> (4 * I - 4);
    return hfma2(ptx::lop3_and_or(in, 0x00F000F0u, 0x3C003C00u), s, t);
}
// D = A B.
__device__ __forceinline__ void mma_new(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// An infinite factor (of a row of values near 2^127) would make NaN of sums that are 0.
__device__ __forceinline__ float within(float x) { return fminf(fmaxf(x, -3.4028234663852886e38f), 3.4028234663852886e38f); }
// Bytes that hold an infinite or no number (e5m2), as 0xFF each.
__device__ __forceinline__ uint32_t bad_scales(uint32_t v) {
    return ((((v & 0x7C7C7C7Cu) + 0x04040404u) & 0x80808080u) >> 7) * 0xFFu;
}

// The 4-bit cache.
struct Four {
    static constexpr int kTile = 128, kTileBits = 7, kWarpKeys = 32;
    // As for the 8-bit cache (attention.cu), in tiles twice as long (before 16 rows had q in shared memory, which takes the
    // 20.9 below to 18.6): an item's cost of 2 and 4 instead of 3 gives
    // 37.7 and 36.4 us for 64 sequences of up to 16001 keys (34.4), 36.7 and 37.8 for one of 131001 (37.6); a
    // least range of 4 and 6 instead of 3 7.2 and 6.1 us for 257 keys (6.2), 8.4 and 10.4 for 1000 (7.9), 20.9
    // and 22.3 for 8 sequences of 5 tokens (20.9), 9.4 and 10.4 for 4000 (9.9).
    static constexpr int kItemCost = 3;
    static constexpr int kMinChunk = 3;
    static constexpr int per_sm(int D, int ROWS) { return ROWS == 16 ? (D == 128 ? 2 : 3) : (D == 128 ? 3 : 4); }
    static constexpr int stages(int D, int ROWS) { return D == 64 ? (ROWS == 16 ? 6 : 4) : (ROWS == 16 ? 5 : 3); }
    static constexpr int kCtas = kSms * 4;                                // at most
    static constexpr bool kHold = true;                                   // the list in shared memory during tiles
    static constexpr float kUnit = 64.f;
    // m of a row that has seen nothing: any score outgrows it, and, unlike with -inf, scores less m are no NaN.
    static constexpr float kNone = -3.4028234663852886e38f;
    static __device__ __forceinline__ bool is_far(float m) { return fabsf(m) >= kFar && m != kNone; }
    template <int D>
    static constexpr int kKeyBytes = D + D / 16;                          // codes and scales of K and V

    struct Maps { CUtensorMap k, v, k_scale, v_scale; };
    template <int D>
    struct Stage {
        alignas(1024) uint8_t k[kTile * D / 2];
        alignas(1024) uint8_t v[kTile * D / 2];
        alignas(128) uint8_t k_scale[kTile / 16 * 128];                   // up to eight pages' slots
        alignas(128) uint8_t v_scale[kTile / 16 * 128];
    };
    // A copy's place in shared memory is a multiple of 128 bytes: so far apart are the scales of pages in a stage.
    template <int D>
    static __device__ __forceinline__ int slot_of_box(int box) { return max(box * (D / kGroup4), 128); }

    struct StageBeside {};
    struct Beside {};

    static __device__ __forceinline__ void prefetch(const Maps &m) {
        ptx::prefetch_tensormap(&m.k);
        ptx::prefetch_tensormap(&m.v);
        ptx::prefetch_tensormap(&m.k_scale);
        ptx::prefetch_tensormap(&m.v_scale);
    }
    static __device__ __forceinline__ Beside beside(const AttentionArgs &, int, int) { return {}; }
    template <int D>
    static __device__ __forceinline__ void copy(const Maps &m, Stage<D> &s, int part, int box, int row, int head, int page,
                                                uint32_t bar) {
        constexpr int kCodes = D / 2;
        const int x = row * (D / kGroup4) / 4, slot = part * slot_of_box<D>(box);
        ptx::tma_load_4d(ptx::smem_u32(s.k) + part * box * kCodes, &m.k, 0, row * kCodes / 128, head, page, bar);
        ptx::tma_load_4d(ptx::smem_u32(s.k_scale) + slot, &m.k_scale, x, head, page, 0, bar);
        ptx::tma_load_4d(ptx::smem_u32(s.v) + part * box * kCodes, &m.v, 0, row * kCodes / 128, head, page, bar);
        ptx::tma_load_4d(ptx::smem_u32(s.v_scale) + slot, &m.v_scale, x, head, page, 0, bar);
    }
    static __device__ __forceinline__ void put_beside(StageBeside &, const Beside &, int, int) {}

    // A stage's codes are lines of 128 bytes, two keys (of 128 values) or four (lines of 64 bytes took 40.5 us
    // for 131001 keys where these took 40.3: copies were not the bound).  A lane's ldmatrix address in the first 16 keys of its warp's 32,
    // without the chunk of 16 bytes (32 codes, a group): the swizzle flips bits of a chunk's number in its line by the
    // line's, so chunk c is at (address ^ c << 4); the second 16 keys are 8 lines on, or 4.
    template <int D>
    struct Lane {
        uint32_t off, scales[2];                     // scales: of the first key of each 16
        __device__ __forceinline__ Lane(const AttentionArgs &p, int warp) {
            const int box = min(p.P, kTile), slot = slot_of_box<D>(box);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int first = warp * kWarpKeys + 16 * i;
                scales[i] = first / box * slot + first % box * (D / kGroup4);
            }
            const int lane = threadIdx.x & 31, key = warp * kWarpKeys + ((lane >> 3) & 1) * 8 + (lane & 7);
            const uint32_t in = key * (D / 2) + ((lane >> 4) << 4);
            off = in ^ (in >> 7 & 7) << 4;
        }
    };

    // Of the first 16 keys (half 0) or the second.
    template <int D>
    static __device__ __forceinline__ uint32_t second(uint32_t at, int half) {
        return half == 0 ? at : (D == 128 ? at : at ^ 64u) + 8 * D;
    }

    // A consumer warp's state of an item.  Lane (g, t) = (lane / 4, lane % 4); column pair
    // n: query rows 8n + 2t and 8n + 2t + 1.
    template <int D, int ROWS>
    struct State {
        static constexpr int KS = D / 16, N = ROWS / 8, G = D / kGroup4;
        // B fragments of q^T: values 8t + (0, 4), (1, 5); (2, 6), (3, 7) of a group.  Of 16 rows the warps
        // of a CTA share them in shared memory: the registers are worth more (8 sequences of 5 tokens 20.9 -> 18.1 us, 4 of 16
        // 33.1 -> 26.2; 8 rows gain nothing).
        static constexpr bool kShared = N == 2;
        uint32_t q[kShared ? 1 : KS][N][2];
        uint32_t shared;
        __device__ __forceinline__ void fragments(int j, uint32_t (&f)[N][4]) const {
            if constexpr (kShared) {
                #pragma unroll
                for (int n = 0; n < N; ++n) ptx::lds_v4<0>(shared + (n * G + j) * 512, f[n][0], f[n][1], f[n][2], f[n][3]);
            } else {
#pragma unroll
                for (int n = 0; n < N; ++n) f[n][0] = q[2 * j][n][0], f[n][1] = q[2 * j][n][1], f[n][2] = q[2 * j + 1][n][0], f[n][3] = q[2 * j + 1][n][1];
            }
        }
        uint32_t offset[N][2];                       // B fragment of -8 sum q of the groups, in three parts
        float qs[N][2];                              // factor of the row's scores
        int pos[N][2];
        float o[KS][N][4];                           // O^T
        float m[N][2], l[N][2];
        float limit;                                 // of scores over m: kPeak, or all are looked at (some |m| past kFar)
    };
    template <int D, int ROWS>
    struct Queries { uint4 q[State<D, ROWS>::kShared ? ROWS / 8 * (D / kGroup4) : 1][State<D, ROWS>::kShared ? 32 : 1]; };
    static __device__ __forceinline__ int value_of(int k, int g) { return 32 * (k >> 1) + 4 * g + 2 * (k & 1); }

    // Query fragments: fp16, each row times a power of two, 2^4 more than for the 8-bit cache where the
    // codes are 2^-24 of themselves.
    template <int D, int ROWS>
    static __device__ __forceinline__ void queries(const AttentionArgs &p, State<D, ROWS> &a, const Seq &s, int h, int row0,
                                                   Queries<D, ROWS> &queries) {
        constexpr int KS = D / 16, N = ROWS / 8, G = D / kGroup4;
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, nrows = s.n * p.G, first = s.len - s.n;
        a.limit = kPeak;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int r = row0 + 8 * n + g;
            const bool live = r < nrows;
            const int i = live ? r / p.G : 0, hq = h * p.G + (live ? r - i * p.G : 0);
            const uint16_t *q = p.q + (int64_t)(s.start + i) * p.q_token + hq * p.q_head + 8 * t;
            uint2 v[G][2];
            float amax = 0.f;
#pragma unroll
            for (int j = 0; j < G; ++j)
#pragma unroll
                for (int c = 0; c < 2; ++c) v[j][c] = live ? *reinterpret_cast<const uint2 *>(q + 32 * j + 4 * c) : make_uint2(0u, 0u);
#pragma unroll
            for (int j = 0; j < G; ++j)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float x[4] = {bf16_lo(v[j][c].x), bf16_hi(v[j][c].x), bf16_lo(v[j][c].y), bf16_hi(v[j][c].y)};
#pragma unroll
                    for (int k = 0; k < 4; ++k) amax = fabsf(x[k]) < INFINITY ? fmaxf(amax, fabsf(x[k])) : amax;
                }
            amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 2));
            const int up = query_shift(amax);
            const float odd = exp2_int(up), even = exp2_int(up + 4), scale = within(exp2_int(4 - up) * p.scale_log2);
            float sum[G];
#pragma unroll
            for (int j = 0; j < G; ++j) {
                const uint2 lo = v[j][0], hi = v[j][1];                     // values 0 .. 3 and 4 .. 7 of the lane's eight
                const uint32_t q[4] = {f32x2_to_f16x2(bf16_lo(lo.x) * even, bf16_lo(hi.x) * even), f32x2_to_f16x2(bf16_hi(lo.x) * odd, bf16_hi(hi.x) * odd),
                                       f32x2_to_f16x2(bf16_lo(lo.y) * even, bf16_lo(hi.y) * even), f32x2_to_f16x2(bf16_hi(lo.y) * odd, bf16_hi(hi.y) * odd)};
                if constexpr (State<D, ROWS>::kShared) {
                    if (threadIdx.x < 32) queries.q[n * G + j][lane] = make_uint4(q[0], q[1], q[2], q[3]);
                } else {
                    a.q[2 * j][n][0] = q[0], a.q[2 * j][n][1] = q[1], a.q[2 * j + 1][n][0] = q[2], a.q[2 * j + 1][n][1] = q[3];
                }
                float half[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&q[c]));
                    const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&q[2 + c]));
                    half[c] = (x.x + x.y) + (y.x + y.y);
                }
                sum[j] = fmaf(half[1], 16.f, half[0]) * (-8.f * 0x1p-8f);          // below 2^15
                sum[j] += __shfl_xor_sync(~0u, sum[j], 1);
                sum[j] += __shfl_xor_sync(~0u, sum[j], 2);
            }
            // Rows of the fragment: lanes t = 0 and 1 the groups' upper 11 bits, 2 and 3 the next 11; then, 0 and 1, the last.
            float rest[2] = {G == 4 && (t & 1) ? sum[G - 2] : sum[0], G == 4 && (t & 1) ? sum[G - 1] : sum[1]};
            uint32_t parts[3];
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                parts[k] = f32x2_to_f16x2(rest[0], rest[1]);
                const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&parts[k]));
                rest[0] -= x.x, rest[1] -= x.y;
            }
            const bool counts = G == 4 || (t & 1) == 0;                        // two groups fill half of the lanes
            a.offset[n][0] = counts ? (t < 2 ? parts[0] : parts[1]) : 0u;
            a.offset[n][1] = counts && t < 2 ? parts[2] : 0u;
            // This lane's columns are rows 2t and 2t + 1.
            const int position = live ? first + i : -1;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                a.qs[n][c] = __shfl_sync(~0u, scale, 8 * t + 4 * c);
                a.pos[n][c] = __shfl_sync(~0u, position, 8 * t + 4 * c);
                a.m[n][c] = kNone, a.l[n][c] = 0.f;
            }
#pragma unroll
            for (int c = 0; c < KS; ++c) a.o[c][n][0] = a.o[c][n][1] = a.o[c][n][2] = a.o[c][n][3] = 0.f;
        }
        if constexpr (State<D, ROWS>::kShared) {     // (the last item's are no longer read: its warps have been joined)
            a.shared = ptx::smem_u32(&queries.q[0][lane]);
            ptx::named_sync(1, kWarps * 32);
        }
    }

    // The scales of a key's groups, a byte each.
    template <int D>
    static __device__ __forceinline__ uint32_t key_scales(uint32_t at) { return D == 128 ? ptx::lds_u32(at) : (uint32_t)ptx::lds_u16(at); }
    // Those of groups c and c + 1 as fp32, times 2^16: what the codes are 2^-24 (2^-20) and q 2^4 (1) times themselves, and the
    // offsets 2^-8 and the 2^4 of q, leave 2^-4 for the row's factor, a number for every row of q (2^20 was none from 2^121 on).
    static __device__ __forceinline__ float2 scale_pair(uint32_t u, int c) {
        const uint32_t h = ptx::prmt(u, 0u, c == 0 ? 0x1404u : 0x3424u);
        return ptx::fmul2(__half22float2(*reinterpret_cast<const __half2 *>(&h)), make_float2(0x1p16f, 0x1p16f));
    }

    // A warp's 32 keys of a stage, in two halves of 16.  EDGE: some row does not see some key of them.
    template <int D, int ROWS, bool EDGE>
    static __device__ __forceinline__ void slice(const AttentionArgs &p, State<D, ROWS> &st, const Lane<D> &at, const Stage<D> &stage,
                                                 const StageBeside &, int key0, int len) {
        constexpr int N = ROWS / 8, G = D / kGroup4;
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const uint32_t kat = ptx::smem_u32(stage.k) + at.off, vat = ptx::smem_u32(stage.v) + at.off;
        const uint32_t kst = ptx::smem_u32(stage.k_scale) + g * G, vst = ptx::smem_u32(stage.v_scale) + 2 * t * G;
        const uint32_t mine = D == 128 && (t & 1) ? 0x3424u : 0x1404u;           // this lane's two groups as an fp16 pair
        float x[2][N][4];
        uint32_t seen[2][N];                         // bit i: value i of the pair is seen
        uint32_t u[2][2];                            // the scales of keys g and g + 8 of both halves
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            u[half][0] = key_scales<D>(kst + at.scales[half]), u[half][1] = key_scales<D>(kst + at.scales[half] + 8 * G);
            // The groups' offsets: scales times -8 sum q.
            const uint32_t f0 = ptx::prmt(u[half][0], 0u, mine), f1 = ptx::prmt(u[half][1], 0u, mine);
#pragma unroll
            for (int n = 0; n < N; ++n) {
                mma_new(x[half][n], f0, f1, f0, f1, st.offset[n][0], st.offset[n][1]);
                seen[half][n] = 0xFu;
                if constexpr (EDGE) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {    // (key g, row 2t), (g, 2t+1), (g+8, 2t), (g+8, 2t+1)
                        const int key = key0 + half * 16 + g + 8 * (i >> 1), pos = st.pos[n][i & 1];
                        if (!(key <= pos && (p.window == 0 || key > pos - p.window))) seen[half][n] &= ~(1u << i);
                    }
                }
            }
        }
#pragma unroll
        for (int c = 0; c < G; c += 2) {
            uint32_t r[2][4];
            ldsm_x4(second<D>(kat, 0) ^ (c << 4), r[0]);         // (keys 0-7, chunk c), (8-15, c), (0-7, c+1), (8-15, c+1)
            ldsm_x4(second<D>(kat, 1) ^ (c << 4), r[1]);
            const float2 s[2][2] = {{scale_pair(u[0][0], c), scale_pair(u[0][1], c)}, {scale_pair(u[1][0], c), scale_pair(u[1][1], c)}};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int j = c + i;
                uint32_t q[N][4];
                st.fragments(j, q);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const uint32_t a = r[half][2 * i], b = r[half][2 * i + 1], a8 = a >> 8, b8 = b >> 8;
                    const float s0 = i == 0 ? s[half][0].x : s[half][0].y, s1 = i == 0 ? s[half][1].x : s[half][1].y;
#pragma unroll
                    for (int n = 0; n < N; ++n) {
                        float acc[4];
                        mma_new(acc, a & 0x000F000Fu, b & 0x000F000Fu, a & 0x00F000F0u, b & 0x00F000F0u, q[n][0], q[n][1]);
                        ptx::mma_16816_f16(acc, a8 & 0x000F000Fu, b8 & 0x000F000Fu, a8 & 0x00F000F0u, b8 & 0x00F000F0u, q[n][2], q[n][3]);
#pragma unroll
                        for (int k = 0; k < 4; ++k) x[half][n][k] = fmaf(acc[k], k < 2 ? s0 : s1, x[half][n][k]);
                    }
                }
            }
        }
        // Exponents of the weights: scores over m.
        float y[2][N][4];
        auto exponents = [&](auto moved) {
            float top = -INFINITY;
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int half = 0; half < 2; ++half)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float by = st.qs[n][i & 1], m = st.m[n][i & 1];
                        y[half][n][i] = moved && is_far(m) ? __fsub_rn(__fmul_rn(x[half][n][i], by), m) : fmaf(x[half][n][i], by, -m);
                        if (EDGE && !(seen[half][n] >> i & 1u)) y[half][n][i] = -INFINITY;
                        top = fmaxf(top, y[half][n][i]);
                    }
            return top;
        };
        if (__any_sync(~0u, exponents(std::false_type{}) > st.limit)) {   // rows whose maximum has outgrown m (the first keys seen: from kNone)
            bool any = false;
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float mx = -INFINITY;
#pragma unroll
                    for (int half = 0; half < 2; ++half)
#pragma unroll
                        for (int i = c; i < 4; i += 2)
                            if (!EDGE || (seen[half][n] >> i & 1u)) mx = fmaxf(mx, x[half][n][i] * st.qs[n][c]);
                    mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 8));
                    mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 16));
                    const float to = mx - st.m[n][c] > kPeak ? mx - kStart : st.m[n][c];    // of this row alone
                    const Rescale by(st.m[n][c] - to);
                    const float f = by.of_o();
                    st.m[n][c] = to;
                    st.l[n][c] = by.of_l(st.l[n][c]);
                    any |= is_far(to);
#pragma unroll
                    for (int k = 0; k < 2 * G; ++k) st.o[k][n][c] *= f, st.o[k][n][c + 2] *= f;
                }
            st.limit = __any_sync(~0u, any) ? -INFINITY : kPeak;
            exponents(std::true_type{});
        }
        uint32_t pb[2][N][2];                        // P^T: B fragments
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int n = 0; n < N; ++n) {
                float (&w)[4] = y[half][n];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = ex2(w[i]);
                st.l[n][0] += w[0] + w[2];
                st.l[n][1] += w[1] + w[3];
                pb[half][n][0] = transpose8(f32x2_to_f16x2(w[0], w[1]));
                pb[half][n][1] = transpose8(f32x2_to_f16x2(w[2], w[3]));
            }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            // Scales of keys 2t, 2t + 1 and 2t + 8, 2t + 9; zero past the sequence's end.
            uint32_t w[4];
            if constexpr (D == 128) {
                ptx::lds_v2<0>(vst + at.scales[half], w[0], w[1]);
                ptx::lds_v2<8 * G>(vst + at.scales[half], w[2], w[3]);
            } else {
                w[0] = w[1] = ptx::lds_u32(vst + at.scales[half]);
                w[2] = w[3] = ptx::lds_u32_off<8 * G>(vst + at.scales[half]);
            }
            uint32_t bad[4];
            bool apart = false;                      // a scale that is no number, at a key that not all rows see
            if constexpr (EDGE) {
                const int key = key0 + half * 16 + 2 * t;
                const bool in[4] = {key < len, key + 1 < len, key + 8 < len, key + 9 < len};
                uint32_t any = 0u;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (D == 128) {
                        if (!in[i]) w[i] = 0u;
                    } else {
                        w[i] &= (in[i & 2] ? 0xFFFFu : 0u) | (in[(i & 2) + 1] ? 0xFFFF0000u : 0u);
                    }
                    bad[i] = bad_scales(w[i]);
                    any |= bad[i];
                    w[i] &= ~bad[i];
                }
                apart = __any_sync(~0u, any != 0u);
            }
#pragma unroll
            for (int c = 0; c < G; c += 2) {
                uint32_t r[4];
                ldsm_x4_trans(second<D>(vat, half) ^ (c << 4), r);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int j = c + i, k = D == 128 ? 4 + j : 2 + j;
                    // The upper bytes of an fp16 pair; the lower ones take the scale's sign bits, 0.
                    const uint32_t pick = (uint32_t)((8 | j) | j << 4 | (8 | k) << 8 | k << 12);
                    const uint32_t s0 = ptx::prmt(w[0], w[1], pick), s1 = ptx::prmt(w[2], w[3], pick);
                    const uint32_t t0 = hmul2(s0, 0xBC80BC80u), t1 = hmul2(s1, 0xBC80BC80u);       // times -1.125
                    const uint32_t a = r[2 * i], b = r[2 * i + 1];
                    const uint32_t lo[4] = {values4<0>(a, s0, t0), values4<1>(a, s0, t0), values4<0>(b, s1, t1), values4<1>(b, s1, t1)};
                    const uint32_t hi[4] = {values4<2>(a, s0, t0), values4<3>(a, s0, t0), values4<2>(b, s1, t1), values4<3>(b, s1, t1)};
#pragma unroll
                    for (int n = 0; n < N; ++n) {
                        ptx::mma_16816_f16(st.o[2 * j][n], lo[0], lo[1], lo[2], lo[3], pb[half][n][0], pb[half][n][1]);
                        ptx::mma_16816_f16(st.o[2 * j + 1][n], hi[0], hi[1], hi[2], hi[3], pb[half][n][0], pb[half][n][1]);
                    }
                    if constexpr (EDGE) {
                        if (apart) {                 // rows that see such a key take NaN in its group
                            const uint32_t both = (uint32_t)(j | j << 4 | k << 8 | k << 12);
                            const uint32_t b0 = ptx::prmt(bad[0], bad[1], both), b1 = ptx::prmt(bad[2], bad[3], both);
#pragma unroll
                            for (int n = 0; n < N; ++n) {
                                const uint32_t see = seen[half][n];
                                const uint32_t f0 = (see & 1u ? 0xFFFFu : 0u) | (see & 2u ? 0xFFFF0000u : 0u);
                                const uint32_t f1 = (see & 4u ? 0xFFFFu : 0u) | (see & 8u ? 0xFFFF0000u : 0u);
                                uint32_t hit = (transpose8(f0) & b0) | (transpose8(f1) & b1);          // of row g
                                hit |= __shfl_xor_sync(~0u, hit, 1);
                                hit |= __shfl_xor_sync(~0u, hit, 2);
#pragma unroll
                                for (int q = 0; q < 2; ++q) {
                                    if (__shfl_sync(~0u, hit, 8 * t + 4 * q) == 0u) continue;
#pragma unroll
                                    for (int e = q; e < 4; e += 2)
                                        st.o[2 * j][n][e] = st.o[2 * j + 1][n][e] = __int_as_float(0x7FFFFFFF);
                                }
                            }
                        }
                    }
                }
            }
        }
    }

    template <int D>
    static bool make_maps(const AttentionArgs &p, Maps *m) {
        const uint32_t rows = (uint32_t)std::min(p.P, kTile);
        const uint64_t dims[4] = {128, (uint64_t)p.P * D / 2 / 128, (uint64_t)p.Hk, (uint64_t)p.pages};
        const uint64_t strides[3] = {128, (uint64_t)p.head_stride, (uint64_t)p.page_stride};
        const uint32_t box[4] = {128, rows * D / 2 / 128, 1, 1};
        // A page's scales of a head are one run of bytes, copied as words (a box has 256 elements at most).
        const uint64_t sdims[4] = {(uint64_t)p.P * D / kGroup4 / 4, (uint64_t)p.Hk, (uint64_t)p.pages, 1};
        const uint64_t sstrides[3] = {(uint64_t)p.scale_head_stride, (uint64_t)p.scale_page_stride, (uint64_t)p.scale_page_stride};
        const uint32_t sbox[4] = {rows * D / kGroup4 / 4, 1, 1, 1};
        const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
        return encode_tiled(&m->k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, p.k_cache, dims, strides, box, sw) &&
               encode_tiled(&m->v, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, p.v_cache, dims, strides, box, sw) &&
               encode_tiled(&m->k_scale, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, p.k_scale, sdims, sstrides, sbox, CU_TENSOR_MAP_SWIZZLE_NONE) &&
               encode_tiled(&m->v_scale, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, p.v_scale, sdims, sstrides, sbox, CU_TENSOR_MAP_SWIZZLE_NONE);
    }
};

}  // namespace

cudaError_t launch_attention4(const AttentionArgs &p, cudaStream_t stream) { return launch_few_rows<Four>(p, stream); }
size_t attention4_workspace_bytes(int max_q, int G, int D) { return few_rows_workspace<Four>(max_q, G, D); }
uint32_t attention4_timeouts(bool reset) { return few_rows_timeouts(reset); }

}  // namespace lowbit
