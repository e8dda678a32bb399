// attention.cu -- softmax attention of the new tokens' queries over the 8-bit
// paged cache (lowbit_attention), on the warp-level tensor cores.
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
//     w_t = 2^(s_t + ve(t) - m),  m = running max of s_t + ve(t),
//     O += fp16(w_t) Vc_t,  l += w_t 2^-ve(t),  out = O / l,  lse = ln2 (m + log2 l).
// w <= 1, so fp16 holds it to 2^-11 of itself down to 2^-14 and to 2^-25 below;
// m, l, O are fp32.  q is multiplied by a power of two per row that puts its
// largest value into [2^10, 2^11): its 8 significant bits fit fp16's 11.
//
// A row that sees nothing has l = 0: out = 0, lse = -inf.  Masked scores are
// replaced, not added to, and V codes past a sequence's end are zeroed, so what
// a page holds there (NaN codes among it) does not reach the sums; a NaN in V that
// some rows of a tile see and others do not is handled apart (poison).
//
// Work split.  An item is (sequence, kv head, tile of 8 or 16 rows), the rows being
// the new tokens times the heads of the group; its keys come in tiles of 64.  All
// items' tiles form one list, cut into equal ranges, one per CTA: sequences of any
// lengths fill the machine evenly.  An item that a cut divides leaves its parts'
// (m, l, O) in the workspace, and a second launch joins them.
//
// A CTA: one producer warp (TMA: K and V tile of 64 keys per stage, 128- or 64-byte
// swizzle; pages smaller than a tile take one copy each) and four consumer warps of
// 16 keys each with their own running (m, l, O), joined at the item's end.
// Bound: HBM, 2 D bytes per key and kv head.
#include <algorithm>

#include "attention.cuh"

namespace lowbit {
namespace {

using namespace attn;

constexpr int kTile = 64;                        // keys of a stage
constexpr int kWarps = 4;                        // consumer warps, 16 keys each
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kMinTiles = 4;                     // of a CTA's range

// Stages and CTAs per SM: together about 150 KB of loads in flight on an SM.
template <int D, int ROWS>
struct Shape {
    static constexpr int kStages = D == 128 ? (ROWS == 8 ? 5 : 4) : 6;
    static constexpr int kPerSm = D == 128 ? 2 : 3;
    static constexpr int kCtas = kSms * kPerSm;
};
// Sequences with more query rows (new tokens times heads of a group) than this go to
// the prompt kernel.
constexpr int kFewRows = 64;

__device__ unsigned int g_attn_timeouts;

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// ---------------------------------------------------------------------------
// The list of tiles.

struct Seq : Span {
    int lo, nt;             // first key tile and number of tiles
    int rt;                 // row tiles; none for a sequence of the prompt kernel
};

__device__ __forceinline__ Seq sequence(const AttentionArgs &p, int b, int rows) {
    Seq s;
    static_cast<Span &>(s) = span(p, b);
    const int first = s.len - s.n, n = s.n * (p.Hq / p.Hk);
    s.lo = p.window > 0 ? max(first - p.window + 1, 0) / kTile : 0;
    s.nt = max((s.len + kTile - 1) / kTile - s.lo, 1);           // an empty sequence still writes its rows
    s.rt = n > p.few_rows ? 0 : (n + rows - 1) / rows;
    return s;
}

// A place in the list: item (b, h, rt) and tile t of it.
struct Place { int b, h, rt, t; long long before; };             // before: tiles of earlier sequences

// Moves pl.b (with pl.before) forward to the sequence that holds `idx`; fills the rest.
__device__ __forceinline__ Seq locate(const AttentionArgs &p, int rows, long long idx, Place &pl) {
    Seq s = sequence(p, pl.b, rows);
    long long w = (long long)s.nt * s.rt * p.Hk;
    while (idx >= pl.before + w && pl.b + 1 < p.B) {
        pl.before += w;
        s = sequence(p, ++pl.b, rows);
        w = (long long)s.nt * s.rt * p.Hk;
    }
    const long long in = idx - pl.before;
    const int item = (int)(in / s.nt);
    pl.t = (int)(in - (long long)item * s.nt);
    pl.h = item / max(s.rt, 1);
    pl.rt = item - pl.h * max(s.rt, 1);
    return s;
}

// Total number of tiles, and the sequence (with the tiles before it) that holds
// place c * chunk.  All threads of the CTA take part; result in shared memory.
struct Plan { long long total, chunk, begin, end, before; int b; };

__device__ __forceinline__ void make_plan(const AttentionArgs &p, int rows, int cta, int ctas, Plan *out,
                                          long long *scratch) {
    const int tid = threadIdx.x, nthr = blockDim.x, warp = tid >> 5, lane = tid & 31;
    long long sum = 0;
    for (int b = tid; b < p.B; b += nthr) {
        const Seq s = sequence(p, b, rows);
        sum += (long long)s.nt * s.rt * p.Hk;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    if (lane == 0) scratch[warp] = sum;
    __syncthreads();
    long long total = 0;
    for (int i = 0; i < nthr / 32; ++i) total += scratch[i];
    const long long chunk = max((total + ctas - 1) / ctas, (long long)kMinTiles);
    const long long begin = min((long long)cta * chunk, total);
    if (warp == 0) {
        // Warp 0 walks the sequences 32 at a time until the one that holds `begin`.
        long long before = 0;
        int found = -1;
        for (int b0 = 0; b0 < p.B && found < 0; b0 += 32) {
            long long w = 0;
            if (b0 + lane < p.B) {
                const Seq s = sequence(p, b0 + lane, rows);
                w = (long long)s.nt * s.rt * p.Hk;
            }
            long long inc = w;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long v = __shfl_up_sync(~0u, inc, o);
                if (lane >= o) inc += v;
            }
            const unsigned hit = __ballot_sync(~0u, begin < before + inc);
            if (hit) {
                const int l = __ffs(hit) - 1;
                found = b0 + l;
                before += __shfl_sync(~0u, inc - w, l);
            } else {
                before += __shfl_sync(~0u, inc, 31);
            }
        }
        if (lane == 0) {
            out->total = total;
            out->chunk = chunk;
            out->begin = begin;
            out->end = min(begin + chunk, total);
            out->b = max(found, 0);
            out->before = found < 0 ? 0 : before;
        }
    }
    __syncthreads();
}

// ---------------------------------------------------------------------------
// Shared memory of a CTA.

template <int D, int ROWS>
struct Smem {
    static constexpr int kStages = Shape<D, ROWS>::kStages;
    alignas(1024) uint8_t k[kStages][kTile * D];
    alignas(1024) uint8_t v[kStages][kTile * D];
    float o[kWarps][ROWS][D];                    // the warps' sums at an item's end
    float m[kWarps][ROWS], l[kWarps][ROWS];
    int2 exps[kStages][kWarps];                  // (ke, ve) of each 16 keys
    alignas(8) uint64_t full[kStages], empty[kStages];
    Plan plan;
    long long scratch[kThreads / 32];
};

// Partial results: slot 2c is the item that CTA c continues, slot 2c + 1 the one
// that it leaves unfinished.  A slot: ROWS x D sums, then ROWS (m, l) pairs.
template <int D, int ROWS>
__device__ __forceinline__ float *slot_of(const AttentionArgs &p, long long slot) {
    return p.workspace + slot * (ROWS * (D + 2));
}

// Writes a row's result.
template <int D>
__device__ __forceinline__ void write_row(const AttentionArgs &p, int token, int head, int d, float4 o, float m, float l) {
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);          // NaN stays
    uint16_t *at = p.out + token * p.o_token + head * p.o_head + d;
    const uint32_t a = f32x2_to_bf16x2(o.x * inv, o.y * inv), c = f32x2_to_bf16x2(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2 *>(at) = make_uint2(a, c);
    if (d == 0 && p.lse != nullptr) p.lse[token * p.lse_token + head] = l == 0.f ? -INFINITY : kLn2 * (m + log2f(l));
}

template <int D, int ROWS>
__global__ void __launch_bounds__(kThreads, Shape<D, ROWS>::kPerSm)
    attention_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                     const AttentionArgs p) {
    constexpr int kStages = Shape<D, ROWS>::kStages;
    extern __shared__ uint8_t raw[];
    Smem<D, ROWS> &sm = *reinterpret_cast<Smem<D, ROWS> *>(raw + ((1024 - (ptx::smem_u32(raw) & 1023)) & 1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            ptx::mbar_init(ptx::smem_u32(&sm.full[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&sm.empty[i]), kWarps);
        }
        ptx::fence_mbar_init();
    }
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();
    make_plan(p, ROWS, blockIdx.x, gridDim.x, &sm.plan, sm.scratch);
    const long long begin = sm.plan.begin, end = sm.plan.end;
    if (begin >= end) return;
    const int G = p.Hq / p.Hk, P = p.P;
    Place pl{sm.plan.b, 0, 0, 0, sm.plan.before};

    if (warp == kWarps) {
        // ------------- producer.  Lanes look up the pages of the next tiles (one
        // page, or one part of a large page, a lane) a window ahead of their use.
        const int parts = P < kTile ? kTile / P : 1;             // pages of a tile
        const int ahead = 32 / parts;                            // tiles of a window
        const int box = min(P, kTile);
        int page = -1, row = 0, head = 0, n_page = -1, n_row = 0, n_head = 0, ke = 0, ve = 0, n_ke = 0, n_ve = 0;
        auto look_up = [&](long long w0) {                       // window that starts at tile w0 of the list
            const long long idx = w0 + lane / parts;
            n_page = -1;                                         // nothing to fetch
            if (idx < end) {
                const Seq s = locate(p, ROWS, idx, pl);
                const int key = (s.lo + pl.t) * kTile + (lane % parts) * box;
                n_head = pl.h;
                n_row = key % P;
                if (key < s.len) {
                    n_page = p.page_table[(int64_t)pl.b * p.table_stride + key / P];
                    if (n_page < 0) n_page = p.pages;            // outside the cache: read as zeros
                }
            }
        };
        auto look_up_exps = [&] {
            n_ke = n_ve = 0;
            if ((unsigned)n_page < (unsigned)p.pages) {
                n_ke = min(max((int)p.k_exp[(int64_t)n_page * p.Hk + n_head], kExpMin), kExpMax);
                n_ve = min(max((int)p.v_exp[(int64_t)n_page * p.Hk + n_head], kExpMin), kExpMax);
            }
        };
        look_up(begin);
        look_up_exps();
        bool ok = true;
        int issued = 0;
        for (long long w0 = begin; w0 < end && ok; w0 += ahead) {
            page = n_page, row = n_row, head = n_head, ke = n_ke, ve = n_ve;
            look_up(w0 + ahead);
            const int cnt = (int)min((long long)ahead, end - w0);
            for (int i = 0; i < cnt; ++i, ++issued) {
                if (i == cnt / 2) look_up_exps();
                const int st = issued % kStages;
                if (issued >= kStages)
                    ok = __all_sync(~0u, ptx::mbar_wait(ptx::smem_u32(&sm.empty[st]), (issued / kStages - 1) & 1,
                                                        &g_attn_timeouts));
                if (!ok) break;
                // The exponents of the tile's four 16-key slices, then the copies.
                const int src = i * parts + (lane & 3) * parts / kWarps;
                const int ske = __shfl_sync(~0u, ke, src), sve = __shfl_sync(~0u, ve, src);
                if (lane < kWarps) sm.exps[st][lane] = make_int2(ske, sve);
                const bool mine = lane / parts == i && page >= 0;
                const uint32_t bytes = __popc(__ballot_sync(~0u, mine)) * 2u * box * D;
                const uint32_t bar = ptx::smem_u32(&sm.full[st]);
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_expect_tx(bar, bytes);
                __syncwarp();
                if (mine) {
                    const uint32_t off = (lane % parts) * box * D;
                    ptx::tma_load_4d(ptx::smem_u32(sm.k[st]) + off, &kmap, 0, row, head, page, bar);
                    ptx::tma_load_4d(ptx::smem_u32(sm.v[st]) + off, &vmap, 0, row, head, page, bar);
                }
                __syncwarp();
            }
        }
        for (int i = max(0, issued - kStages); i < issued; ++i)
            if (!ptx::mbar_wait(ptx::smem_u32(&sm.full[i % kStages]), (i / kStages) & 1, &g_attn_timeouts)) break;
        return;
    }

    // ---------------- consumers.  Lane (g, t): rows g and g + 8, columns 2t, 2t+1.
    const int g = lane >> 2, t = lane & 3;
    constexpr int KS = D / 16;                                   // 16-byte chunks of a cache row
    constexpr int HALVES = ROWS / 8;
    auto chunk_addr = [&](uint32_t base, int key, int c) {       // swizzled 16-byte chunk c of a key's row
        const int sw = D == 128 ? key & 7 : (key >> 1) & 3;
        return base + key * D + ((c ^ sw) << 4);
    };
    // ldmatrix addresses.  K: matrices (keys 0-7, chunk c), (keys 8-15, c), (0-7, c+1), (8-15, c+1).
    const int mkey = warp * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), mchunk = lane >> 4;
    bool ok = true;
    int used = 0;                                                // stages consumed
    for (long long idx = begin; idx < end;) {
        const Seq s = locate(p, ROWS, idx, pl);
        const int cnt = (int)min((long long)(s.nt - pl.t), end - idx);
        const int nrows = s.n * G, row0 = pl.rt * ROWS;
        const int first = s.len - s.n;

        // Query fragments: fp16, each row times a power of two.
        uint32_t qf[KS][2 * HALVES];
        float qs[HALVES];                                        // scale of the row's scores
        int pos[HALVES];
#pragma unroll
        for (int hf = 0; hf < HALVES; ++hf) {
            const int r = row0 + g + 8 * hf;
            const bool live = r < nrows;
            const int i = live ? r / G : 0, hq = pl.h * G + (live ? r - i * G : 0);
            pos[hf] = live ? first + i : -1;
            const uint16_t *q = p.q + (int64_t)(s.start + i) * p.q_token + hq * p.q_head;
            float x[KS][4], amax = 0.f;
#pragma unroll
            for (int c = 0; c < KS; ++c) {
                const uint2 v = live ? *reinterpret_cast<const uint2 *>(q + 16 * c + 4 * t) : make_uint2(0u, 0u);
                x[c][0] = bf16_lo(v.x), x[c][1] = bf16_hi(v.x), x[c][2] = bf16_lo(v.y), x[c][3] = bf16_hi(v.y);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float a = fabsf(x[c][k]);
                    amax = a < INFINITY ? fmaxf(amax, a) : amax;
                }
            }
            amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 2));
            const int up = query_shift(amax);
            const float f = exp2_int(up);
            qs[hf] = exp2_int(-up) * p.scale_log2;
#pragma unroll
            for (int c = 0; c < KS; ++c) {
                qf[c][hf] = f32x2_to_f16x2(x[c][0] * f, x[c][1] * f);
                qf[c][HALVES + hf] = f32x2_to_f16x2(x[c][2] * f, x[c][3] * f);
            }
        }
        const int pos_lo = first + row0 / G, pos_hi = first + (min(row0 + ROWS, nrows) - 1) / G;

        float o[2 * KS][4], m[HALVES], l[HALVES];
#pragma unroll
        for (int j = 0; j < 2 * KS; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
#pragma unroll
        for (int hf = 0; hf < HALVES; ++hf) m[hf] = -INFINITY, l[hf] = 0.f;

        for (int tile = 0; tile < cnt; ++tile, ++used) {
            const int st = used % kStages;
            if (ok) ok = ptx::mbar_wait(ptx::smem_u32(&sm.full[st]), (used / kStages) & 1, &g_attn_timeouts);
            const int key0 = (s.lo + pl.t + tile) * kTile + warp * 16;
            // Keys that some row sees: up to pos_hi, from pos_lo - window + 1 on.
            if (key0 <= pos_hi && (p.window == 0 || key0 + 15 > pos_lo - p.window)) {
                const int2 e = sm.exps[st][warp];
                const uint32_t kb = ptx::smem_u32(sm.k[st]), vb = ptx::smem_u32(sm.v[st]);
                float sc[2][4];
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
#pragma unroll
                for (int c = 0; c < KS; c += 2) {
                    uint32_t r[4];
                    ldsm_x4(chunk_addr(kb, mkey, c + mchunk), r);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t b0, b1;
                        e4m3x4_to_f16x2(r[i], b0, b1);
                        const int cc = c + (i >> 1);
                        if constexpr (HALVES == 2)
                            ptx::mma_16816_f16(sc[i & 1], qf[cc][0], qf[cc][1], qf[cc][2], qf[cc][3], b0, b1);
                        else
                            ptx::mma_16816_f16(sc[i & 1], qf[cc][0], 0u, qf[cc][1], 0u, b0, b1);
                    }
                }
                const bool whole = key0 + 15 <= pos_lo && (p.window == 0 || key0 > pos_hi - p.window);
                uint32_t seen[HALVES];                           // bit 2 nt + c: the row sees key 8 nt + 2t + c
                uint32_t pf[HALVES][2];                          // weights, fp16 pairs
#pragma unroll
                for (int hf = 0; hf < HALVES; ++hf) {
                    const float f = qs[hf] * exp2_int(e.x), ve = (float)e.y;
                    float x[4] = {sc[0][2 * hf], sc[0][2 * hf + 1], sc[1][2 * hf], sc[1][2 * hf + 1]};
                    seen[hf] = 0xFu;
                    if (!whole) {
                        seen[hf] = 0u;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int key = key0 + 8 * (k >> 1) + 2 * t + (k & 1);
                            if (key <= pos[hf] && (p.window == 0 || key > pos[hf] - p.window)) seen[hf] |= 1u << k;
                        }
                    }
                    float mx = m[hf];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        x[k] = (seen[hf] >> k & 1u) ? fmaf(x[k], f, ve) : -INFINITY;
                        mx = fmaxf(mx, x[k]);
                    }
                    mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 2));
                    const float ref = mx == -INFINITY ? 0.f : mx;
                    if (__any_sync(~0u, mx != m[hf])) {
                        const float a = ex2(m[hf] - ref);        // 0 at the first keys seen
                        l[hf] *= a;
#pragma unroll
                        for (int j = 0; j < 2 * KS; ++j) o[j][2 * hf] *= a, o[j][2 * hf + 1] *= a;
                    }
                    m[hf] = mx;
#pragma unroll
                    for (int k = 0; k < 4; ++k) x[k] = ex2(x[k] - ref);
                    l[hf] = fmaf((x[0] + x[1]) + (x[2] + x[3]), exp2_int(-e.y), l[hf]);
                    pf[hf][0] = f32x2_to_f16x2(x[0], x[1]);
                    pf[hf][1] = f32x2_to_f16x2(x[2], x[3]);
                }
                // Codes past the sequence's end are cleared (keys 2t, 2t+1 and 2t+8, 2t+9 of the slice).
                uint32_t keep[2] = {~0u, ~0u};
                bool apart = false;                              // a NaN that not all rows see
                if (!whole) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int key = key0 + 8 * i + 2 * t;
                        keep[i] = (key < s.len ? 0xFFFFu : 0u) | (key + 1 < s.len ? 0xFFFF0000u : 0u);
                    }
                    uint32_t nan = 0u;
#pragma unroll
                    for (int c = 0; c < KS; c += 2) {
                        uint32_t r[4];
                        ldsm_x4_trans(chunk_addr(vb, mkey, c + mchunk), r);
#pragma unroll
                        for (int i = 0; i < 4; ++i) nan |= (((r[i] & keep[i & 1]) & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                    }
                    apart = __any_sync(~0u, nan != 0u);
                }
#pragma unroll
                for (int c = 0; c < KS; c += 2) {
                    uint32_t r[4];
                    ldsm_x4_trans(chunk_addr(vb, mkey, c + mchunk), r);
#pragma unroll
                    for (int i = 0; i < 4; ++i) r[i] &= keep[i & 1];
#pragma unroll
                    for (int i = 0; i < 4; i += 2) {
                        uint32_t b[2][2], bad[2] = {0u, 0u};
                        const int j = 2 * (c + (i >> 1));
                        if (apart) {                             // NaN codes out, and a flag (1.0) in their place
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const uint32_t hit = (((r[i + k] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7;
                                r[i + k] &= ~(hit * 0xFFu);
                                bad[k] = hit * 0x38u;            // e4m3 1.0
                            }
                        }
                        // Bytes (key, d), (key, d+1), (key+1, d), (key+1, d+1) -> key pairs of d and of d+1.
                        e4m3x4_to_f16x2(ptx::prmt(r[i], 0u, 0x3120u), b[0][0], b[1][0]);
                        e4m3x4_to_f16x2(ptx::prmt(r[i + 1], 0u, 0x3120u), b[0][1], b[1][1]);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            if constexpr (HALVES == 2)
                                ptx::mma_16816_f16(o[j + k], pf[0][0], pf[1][0], pf[0][1], pf[1][1], b[k][0], b[k][1]);
                            else
                                ptx::mma_16816_f16(o[j + k], pf[0][0], 0u, pf[0][1], 0u, b[k][0], b[k][1]);
                        }
                        if (apart) {
                            // Rows that see a flagged key take NaN: seen (1.0 or 0) times flags > 0.
                            uint32_t f[2][2], sf[HALVES][2];
                            e4m3x4_to_f16x2(ptx::prmt(bad[0], 0u, 0x3120u), f[0][0], f[1][0]);
                            e4m3x4_to_f16x2(ptx::prmt(bad[1], 0u, 0x3120u), f[0][1], f[1][1]);
#pragma unroll
                            for (int hf = 0; hf < HALVES; ++hf)
#pragma unroll
                                for (int n = 0; n < 2; ++n)
                                    sf[hf][n] = ((seen[hf] >> (2 * n) & 1u) ? 0x3C00u : 0u) |
                                                ((seen[hf] >> (2 * n + 1) & 1u) ? 0x3C000000u : 0u);
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                float hits[4] = {0.f, 0.f, 0.f, 0.f};
                                if constexpr (HALVES == 2)
                                    ptx::mma_16816_f16(hits, sf[0][0], sf[1][0], sf[0][1], sf[1][1], f[k][0], f[k][1]);
                                else
                                    ptx::mma_16816_f16(hits, sf[0][0], 0u, sf[0][1], 0u, f[k][0], f[k][1]);
#pragma unroll
                                for (int x = 0; x < 2 * HALVES; ++x)
                                    if (hits[x] > 0.f) o[j + k][x] = __int_as_float(0x7FFFFFFF);
                            }
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sm.empty[st]));
        }

        // The warps' parts of the item are joined in shared memory.
#pragma unroll
        for (int hf = 0; hf < HALVES; ++hf) {
            l[hf] += __shfl_xor_sync(~0u, l[hf], 1);
            l[hf] += __shfl_xor_sync(~0u, l[hf], 2);
            if (t == 0) sm.m[warp][g + 8 * hf] = m[hf], sm.l[warp][g + 8 * hf] = l[hf];
#pragma unroll
            for (int c = 0; c < KS; ++c)                          // tiles 2c, 2c+1: four consecutive d
                *reinterpret_cast<float4 *>(&sm.o[warp][g + 8 * hf][16 * c + 4 * t]) =
                    make_float4(o[2 * c][2 * hf], o[2 * c + 1][2 * hf], o[2 * c][2 * hf + 1], o[2 * c + 1][2 * hf + 1]);
        }
        ptx::named_sync(1, kWarps * 32);
        const bool head_part = pl.t > 0, tail_part = pl.t + cnt < s.nt;
        float *slot = slot_of<D, ROWS>(p, 2 * (long long)blockIdx.x + (head_part ? 0 : 1));
        for (int i = tid; i < ROWS * (D / 4); i += kWarps * 32) {
            const int r = i / (D / 4), d = (i % (D / 4)) * 4, row = row0 + r;
            if (row >= nrows) break;
            float mm = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sm.m[w][r]);
            const float ref = mm == -INFINITY ? 0.f : mm;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            float ll = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float a = ex2(sm.m[w][r] - ref);
                const float4 v = *reinterpret_cast<const float4 *>(&sm.o[w][r][d]);
                acc.x = fmaf(a, v.x, acc.x), acc.y = fmaf(a, v.y, acc.y);
                acc.z = fmaf(a, v.z, acc.z), acc.w = fmaf(a, v.w, acc.w);
                ll = fmaf(a, sm.l[w][r], ll);
            }
            if (head_part || tail_part) {
                *reinterpret_cast<float4 *>(slot + r * D + d) = acc;
                if (d == 0) *reinterpret_cast<float2 *>(slot + ROWS * D + 2 * r) = make_float2(mm, ll);
            } else {
                const int ii = row / G;
                write_row<D>(p, s.start + ii, pl.h * G + row - ii * G, d, acc, mm, ll);
            }
        }
        ptx::named_sync(1, kWarps * 32);
        idx += cnt;
    }
}

// Joins the parts of the items that cuts divide: block (c, r) takes row r of the
// item whose first cut is at CTA c's start.
template <int D, int ROWS>
__global__ void __launch_bounds__(128) attention_join_kernel(const AttentionArgs p, int ctas) {
    constexpr int kGroups = 128 / (D / 4);                       // parts read at a time
    __shared__ Plan plan;
    __shared__ long long scratch[4];
    __shared__ float4 so[kGroups][D / 4];
    __shared__ float2 sml[kGroups];
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();
    const int c = blockIdx.x + 1, r = blockIdx.y;
    make_plan(p, ROWS, c, ctas, &plan, scratch);
    const long long idx = plan.begin, chunk = plan.chunk;
    if (idx >= plan.total) return;
    Place pl{plan.b, 0, 0, 0, plan.before};
    const Seq s = locate(p, ROWS, idx, pl);
    if (pl.t == 0 || idx - pl.t < (long long)(c - 1) * chunk) return;    // no cut here, or not the item's first
    const int G = p.Hq / p.Hk, row = pl.rt * ROWS + r;
    if (row >= s.n * G) return;
    const int last = (int)((idx - pl.t + s.nt - 1) / chunk);             // last CTA of the item
    const int parts = last - (c - 1) + 1;
    const int grp = threadIdx.x / (D / 4), d = (threadIdx.x % (D / 4)) * 4;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float pm, float pL, float4 po) {
        const float mx = fmaxf(m, pm), ref = mx == -INFINITY ? 0.f : mx;
        const float a = ex2(m - ref), b = ex2(pm - ref);
        o.x = o.x * a + po.x * b, o.y = o.y * a + po.y * b, o.z = o.z * a + po.z * b, o.w = o.w * a + po.w * b;
        l = l * a + pL * b;
        m = mx;
    };
#pragma unroll 4
    for (int i = grp; i < parts; i += kGroups) {
        const float *slot = slot_of<D, ROWS>(p, i == 0 ? 2 * (long long)(c - 1) + 1 : 2 * (long long)(c - 1 + i));
        const float2 ml = *reinterpret_cast<const float2 *>(slot + ROWS * D + 2 * r);
        add(ml.x, ml.y, *reinterpret_cast<const float4 *>(slot + r * D + d));
    }
    so[grp][d / 4] = o;
    if (d == 0) sml[grp] = make_float2(m, l);
    __syncthreads();
    if (grp == 0) {
#pragma unroll
        for (int k = 1; k < kGroups; ++k) add(sml[k].x, sml[k].y, so[k][d / 4]);
        const int i = row / G;
        write_row<D>(p, s.start + i, pl.h * G + row - i * G, d, o, m, l);
    }
}

template <int D, int ROWS>
cudaError_t launch(const AttentionArgs &p, cudaStream_t stream) {
    const uint32_t box_rows = (uint32_t)std::min(p.P, kTile);
    const uint64_t dims[4] = {(uint64_t)D, (uint64_t)p.P, (uint64_t)p.Hk, (uint64_t)p.pages};
    const uint64_t strides[3] = {(uint64_t)D, (uint64_t)p.head_stride, (uint64_t)p.page_stride};
    const uint32_t box[4] = {(uint32_t)D, box_rows, 1, 1};
    const CUtensorMapSwizzle sw = D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    CUtensorMap kmap, vmap;
    if (!encode_tiled(&kmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, p.k_cache, dims, strides, box, sw) ||
        !encode_tiled(&vmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, p.v_cache, dims, strides, box, sw))
        return cudaErrorInvalidValue;
    const int dev = current_device();
    const void *fn = (const void *)attention_kernel<D, ROWS>;
    const int smem = (int)sizeof(Smem<D, ROWS>) + 1024;
    cudaError_t e = raise_smem_limit(fn, dev, smem);
    if (e != cudaSuccess) return e;
    // No more CTAs than ranges of kMinTiles that the page table allows.
    const int rows_max = (int)std::min<int64_t>((int64_t)p.max_q * (p.Hq / p.Hk), p.few_rows);
    const int64_t items = (int64_t)p.B * p.Hk * ((rows_max + ROWS - 1) / ROWS);
    const int64_t tiles = ((int64_t)p.width * p.P + kTile - 1) / kTile;
    const int ctas = (int)std::min<int64_t>(Shape<D, ROWS>::kCtas, std::max<int64_t>(1, (items * tiles + kMinTiles - 1) / kMinTiles));
    e = launch_pdl(attention_kernel<D, ROWS>, dim3(ctas), dim3(kThreads), smem, stream, kmap, vmap, p);
    if (e != cudaSuccess || ctas == 1) return e;
    return launch_pdl(attention_join_kernel<D, ROWS>, dim3(ctas - 1, ROWS), dim3(128), 0, stream, p, ctas);
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

// Which kernels a call needs: sequences are sorted by their number of query rows, on
// the device when the host does not know it.
struct Split { bool few, many; int few_rows; };
static Split split_of(int max_q, bool uniform, int G) {
    if ((int64_t)max_q * G <= kFewRows) return {true, false, kFewRows};
    return {!uniform, true, uniform ? 0 : kFewRows};
}

static size_t few_workspace_bytes(int max_q, int G, int D) {
    const int rows = (int64_t)max_q * G <= 8 ? 8 : 16;
    return (size_t)(kSms * 3) * 2 * rows * (D + 2) * sizeof(float);
}

size_t attention_workspace_bytes(int64_t T, int B, int max_q, bool uniform, int Hq, int Hk, int D) {
    const Split s = split_of(max_q, uniform, Hq / Hk);
    size_t bytes = s.few ? few_workspace_bytes(max_q, Hq / Hk, D) : 0;
    if (s.many) bytes += prompt_workspace_bytes(prompt_grid(T, B, max_q, uniform, Hq, Hk, D), Hk, D);
    return std::max<size_t>(bytes, 16);
}

cudaError_t launch_attention(const AttentionArgs &args, cudaStream_t stream) {
    AttentionArgs p = args;
    const bool uniform = p.cu_q == nullptr;
    if (uniform) p.max_q = p.T / p.B;
    const int G = p.Hq / p.Hk;
    const Split s = split_of(p.max_q, uniform, G);
    p.few_rows = s.few_rows;
    if (s.many) {
        PromptGrid g = prompt_grid(p.T, p.B, p.max_q, uniform, p.Hq, p.Hk, p.D);
        g.workspace = s.few ? (int64_t)(few_workspace_bytes(p.max_q, G, p.D) / sizeof(float)) : 0;
        const cudaError_t e = launch_prompt(p, g, stream);
        if (e != cudaSuccess || !s.few) return e;
    }
    const bool half = (int64_t)p.max_q * G <= 8;
    if (p.D == 128) return half ? launch<128, 8>(p, stream) : launch<128, 16>(p, stream);
    return half ? launch<64, 8>(p, stream) : launch<64, 16>(p, stream);
}

}  // namespace lowbit
