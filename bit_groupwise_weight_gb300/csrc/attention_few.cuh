// attention_few.cuh -- softmax attention over a paged cache for few query rows a sequence:
// the list of tiles and how it is cut, the kernel's frame, and the join of parts.  What
// depends on how a cache holds its values is a format's own (attention.cu: 8 bits,
// attention4.cu: 4 bits): stages, copies, query fragments, and the products over a
// warp's slice of a stage.  attention.cu describes the work's split.
#pragma once

#include <algorithm>

#include "attention.cuh"

namespace lowbit {
namespace {

using namespace attn;

typedef unsigned long long u64;
constexpr int kWarps = 4;                        // consumer warps, each with a quarter of a stage's keys
constexpr int kThreads = 32 * (kWarps + 1);

__device__ unsigned int g_attn_timeouts;

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
// ---------------------------------------------------------------------------
// The list of tiles.

struct Seq : Span {
    int lo, nt;             // first key tile and number of tiles
    int rt;                 // row tiles; none for a sequence of the prompt kernel
    template <class F>
    __device__ long long units(const AttentionArgs &p) const { return (long long)(F::kItemCost + nt) * (rt * p.Hk); }
};

template <class F, int ROWS>
__device__ __forceinline__ Seq sequence(const AttentionArgs &p, int b) {
    Seq s;
    static_cast<Span &>(s) = span(p, b);
    const int n = s.n * p.G;
    s.lo = p.window > 0 ? max(s.len - s.n - p.window + 1, 0) / F::kTile : 0;
    s.nt = max((s.len + F::kTile - 1) / F::kTile - s.lo, 1);           // an empty sequence still writes its rows
    s.rt = n > p.few_rows ? 0 : (n + ROWS - 1) / ROWS;
    return s;
}

// A place in the list: sequence b, item (h, rt) and tile t of it (below 0: before its
// first tile); `before`: units of earlier sequences.
struct Place { int b, h, rt, t; long long before; };

// Moves pl forward to the place `idx`.
template <class F, int ROWS>
__device__ __forceinline__ Seq locate(const AttentionArgs &p, long long idx, Place &pl) {
    Seq s = sequence<F, ROWS>(p, pl.b);
    while (idx - pl.before >= s.template units<F>(p) && pl.b + 1 < p.B) {
        pl.before += s.template units<F>(p);
        s = sequence<F, ROWS>(p, ++pl.b);
    }
    const uint32_t in = (uint32_t)(idx - pl.before), each = (uint32_t)(F::kItemCost + s.nt), item = in / each;
    pl.t = (int)(in - item * each) - F::kItemCost;
    pl.h = s.rt > 1 ? (int)item / s.rt : (int)item;
    pl.rt = (int)item - pl.h * s.rt;
    return s;
}

// A CTA's range of the list and the sequence in which it begins.  Each warp works it
// out by itself.
struct Plan { long long begin, end, chunk; Place pl; };

template <class F, int ROWS>
__device__ __forceinline__ Plan make_plan(const AttentionArgs &p, int cta, int ctas) {
    const int lane = threadIdx.x & 31;
    auto weight = [&](int b) { return b < p.B ? sequence<F, ROWS>(p, b).template units<F>(p) : 0ll; };
    const long long w0 = weight(lane);
    long long total = w0;
    for (int b = lane + 32; b < p.B; b += 32) total += weight(b);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(~0u, total, o);
    Plan r;
    r.chunk = total <= (long long)ctas * F::kMinChunk ? F::kMinChunk : (total + ctas - 1) / ctas;
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

// What the second launch needs to know of an item: written by the CTA that ends it, from
// CTA `begun` on (below 0: none).
struct Join { int begun, start, nrows, row0, h, pad; };
// What a consumer warp keeps of the list while it goes through tiles.
struct Held {
    Plan plan;
    Place pl;
    Seq s;
    long long idx, first_tile;
    Join join;
    int t0, cnt, nrows, row0;
};

template <class F, int D, int ROWS>
struct Smem {
    typename F::template Stage<D> stage[F::stages(D, ROWS)];
    float o[kWarps][8][D + 4];                   // the warps' sums at an item's end, 8 rows at a time
    float m[kWarps][8], l[kWarps][8];
    Held held[F::kHold ? kWarps : 1];
    typename F::template Queries<D, ROWS> queries;
    typename F::StageBeside beside[F::stages(D, ROWS)];
    alignas(8) uint64_t full[F::stages(D, ROWS)], empty[F::stages(D, ROWS)];
};

// More CTAs than this for each item that the page table allows: a second launch joins the parts.
// (By the last CTA always, 131001 keys take 55.6 us instead of 49.6; with 4 or 48 instead of 12 no
// measured case changes by more than 1.2 us.  The lengths may be far below the table's width, and
// the second launch is then for little: 66 keys take 5.6 us with a table of 2 pages, 9.6 with 2048.)
constexpr int kManyParts = 12;

// Workspace: a flag and a Join per CTA, then two slots per CTA: for the part of an item that it leaves
// to a later CTA (it leaves one at most), and for the part of the item that it joins
// itself.  A slot: ROWS x D sums, then ROWS (m, l) pairs.
__device__ __forceinline__ u64 *flag_of(const AttentionArgs &p, int cta) { return reinterpret_cast<u64 *>(p.workspace) + cta; }
template <class F>
__device__ __forceinline__ Join *join_of(const AttentionArgs &p, int cta) { return reinterpret_cast<Join *>(p.workspace + F::kCtas * 2) + cta; }
template <class F, int D, int ROWS>
__device__ __forceinline__ float *slot_of(const AttentionArgs &p, int slot) {
    return p.workspace + F::kCtas * (2 + (int)sizeof(Join) / 4) + (int64_t)slot * (ROWS * (D + 2));
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
template <class F>
__device__ __forceinline__ void write_row(const AttentionArgs &p, int start, int h, int row, int d, float4 o, float m, float l) {
    const int i = row / p.G, token = start + i, head = h * p.G + row - i * p.G;
    const float inv = (l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l)) * F::kUnit;          // NaN stays
    const uint32_t a = f32x2_to_bf16x2(o.x * inv, o.y * inv), c = f32x2_to_bf16x2(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2 *>(p.out + token * p.o_token + head * p.o_head + d) = make_uint2(a, c);
    if (d == 0 && p.lse != nullptr) p.lse[token * p.lse_token + head] = l == 0.f ? -INFINITY : kLn2 * (m + log2f(l));
}

template <class F, int D, int ROWS>
__global__ void __launch_bounds__(kThreads, F::per_sm(D, ROWS))
    attention_kernel(const __grid_constant__ typename F::Maps maps, const AttentionArgs p) {
    constexpr int S = F::stages(D, ROWS), KS = D / 16, N = ROWS / 8;
    extern __shared__ uint8_t raw[];
    Smem<F, D, ROWS> &sm = *reinterpret_cast<Smem<F, D, ROWS> *>(raw + ((1024 - (ptx::smem_u32(raw) & 1023)) & 1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            ptx::mbar_init(ptx::smem_u32(&sm.full[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&sm.empty[i]), kWarps);
        }
        ptx::fence_mbar_init();
        F::prefetch(maps);
    }
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();
    Plan plan = make_plan<F, ROWS>(p, blockIdx.x, gridDim.x);
    if (plan.begin >= plan.end) {
        if (p.defer && tid == 0) join_of<F>(p, blockIdx.x)->begun = -1;
        return;
    }
    __syncthreads();
    Place pl = plan.pl;

    if (warp == kWarps) {
        // ------------- producer.  Lanes look up the pages of the next tiles (one
        // page, or one part of a large page, a lane) a window ahead of their use.
        const int pshift = p.pshift, page_keys = 1 << pshift;
        const int parts = page_keys < F::kTile ? F::kTile >> pshift : 1;       // pages of a tile
        const int pbits = page_keys < F::kTile ? F::kTileBits - pshift : 0, part = lane & (parts - 1);
        const int box = min(page_keys, F::kTile);
        int n_page = -1, n_row = 0, n_head = 0, n_tiles = 0;
        typename F::Beside n_beside{};
        long long next = plan.begin;                                     // unit from which the next window's tiles are counted
        auto look_up = [&] {
            long long u = next;
            int i = lane >> pbits;                                       // this lane's tile of the window
            bool found = false;
            n_page = -1;                                                 // nothing to fetch
            while (u < plan.end) {
                const Seq s = locate<F, ROWS>(p, u, pl);
                const int t = max(pl.t, 0), left = (int)min((long long)(s.nt - t), plan.end - u - (t - pl.t));
                u += t - pl.t;
                if (i < left) {
                    u += i;
                    found = true;
                    const int key = (s.lo + t + i) * F::kTile + part * box;
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
        look_up();
        n_beside = F::beside(p, n_page, n_head);
        bool ok = true;
        int issued = 0, st = 0;
        uint32_t round = 1;                                              // parity of the stage's last release
        while (n_tiles > 0 && ok) {
            const int page = n_page, row = n_row, head = n_head, cnt = n_tiles;
            const typename F::Beside beside = n_beside;
            n_tiles = 0;
            if (cnt == 32 >> pbits && next < plan.end) look_up();
            for (int i = 0; i < cnt; ++i) {
                if (i == cnt / 2 && n_tiles > 0) n_beside = F::beside(p, n_page, n_head);
                if (issued >= S)
                    ok = __all_sync(~0u, ptx::mbar_wait(ptx::smem_u32(&sm.empty[st]), round, &g_attn_timeouts));
                if (!ok) break;
                // The copies, then what goes beside them.
                const bool mine = (lane >> pbits) == i && page >= 0;
                const uint32_t bytes = __popc(__ballot_sync(~0u, mine)) * (uint32_t)(box * F::template kKeyBytes<D>);
                const uint32_t bar = ptx::smem_u32(&sm.full[st]);
                if (mine) F::template copy<D>(maps, sm.stage[st], part, box, row, head, page, bar);
                F::put_beside(sm.beside[st], beside, i << pbits, parts);
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
    const typename F::template Lane<D> at(p, warp);
    bool ok = true;
    int st = 0;
    uint32_t round = 0;
    Join join{-1, 0, 0, 0, 0, 0};                                        // the item that this CTA ends and others began
    typename F::template State<D, ROWS> a;
    for (long long idx = plan.begin; idx < plan.end;) {
        Seq s = locate<F, ROWS>(p, idx, pl);
        const int units = (int)min((long long)(s.nt - pl.t), plan.end - idx);
        int t0 = max(pl.t, 0), cnt = pl.t + units - t0;                  // this CTA's tiles of the item
        long long first_tile = idx - pl.t;                               // place of the item's first tile
        idx += units;
        if (cnt <= 0) continue;
        int nrows = s.n * p.G, row0 = pl.rt * ROWS;
        const int first = s.len - s.n;

        F::template queries<D, ROWS>(p, a, s, pl.h, row0, sm.queries);
        const int pos_lo = first + row0 / p.G, pos_hi = first + (min(row0 + ROWS, nrows) - 1) / p.G;

        // The tiles' loop needs its registers: what only the items need waits in shared memory.
        if constexpr (F::kHold) {
            if (lane == 0) sm.held[warp] = Held{plan, pl, s, idx, first_tile, join, t0, cnt, nrows, row0};
            __syncwarp();
        }
        const int len = s.len;
        int key0 = (s.lo + t0) * F::kTile + warp * F::kWarpKeys;
        for (int tile = cnt; tile > 0; --tile, key0 += F::kTile) {
            if (ok) ok = ptx::mbar_wait(ptx::smem_u32(&sm.full[st]), round, &g_attn_timeouts);
            const int last = key0 + F::kWarpKeys - 1;
            if (last <= pos_lo && (p.window == 0 || key0 > pos_hi - p.window))
                F::template slice<D, ROWS, false>(p, a, at, sm.stage[st], sm.beside[st], key0, len);
            else if (key0 <= pos_hi && (p.window == 0 || last > pos_lo - p.window))
                F::template slice<D, ROWS, true>(p, a, at, sm.stage[st], sm.beside[st], key0, len);
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sm.empty[st]));
            if (++st == S) st = 0, round ^= 1;
        }
        if constexpr (F::kHold) {
            asm volatile("" ::: "memory");
            const Held &w = sm.held[warp];
            plan = w.plan, pl = w.pl, s = w.s, idx = w.idx, first_tile = w.first_tile, join = w.join;
            t0 = w.t0, cnt = w.cnt, nrows = w.nrows, row0 = w.row0;
            __syncwarp();
        }

        // The warps' parts of the item are joined in shared memory, 8 rows at a time.
        const bool continued = t0 > 0, unfinished = t0 + cnt < s.nt;
        float *slot = slot_of<F, D, ROWS>(p, 2 * (int)blockIdx.x + (unfinished ? 0 : 1));
        if (continued && !unfinished) join = Join{(int)(first_tile / plan.chunk), s.start, nrows, row0, pl.h, 0};
#pragma unroll
        for (int n = 0; n < N; ++n) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) a.l[n][c] += __shfl_xor_sync(~0u, a.l[n][c], o);
                if (g == 0) sm.m[warp][2 * t + c] = a.m[n][c], sm.l[warp][2 * t + c] = a.l[n][c];
#pragma unroll
                for (int k = 0; k < KS; ++k)
                    *reinterpret_cast<float2 *>(&sm.o[warp][2 * t + c][F::value_of(k, g)]) = make_float2(a.o[k][n][c], a.o[k][n][c + 2]);
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
                    write_row<F>(p, s.start, pl.h, row, d, acc, mm, ll);
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
    if (p.defer && tid == 0) *join_of<F>(p, blockIdx.x) = join;
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
        const float *part = slot_of<F, D, ROWS>(p, 2 * c + (c == (int)blockIdx.x));
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
        if (join.row0 + r[q] < join.nrows) write_row<F>(p, join.start, join.h, join.row0 + r[q], d, o[q], m[q], l[q]);
}

// The second launch: block (c, r) takes row r of the item that CTA c ends.
template <class F, int D, int ROWS>
__global__ void __launch_bounds__(128) attention_join_kernel(const AttentionArgs p) {
    constexpr int kGroups = 128 / (D / 4);                       // parts read at a time
    __shared__ float4 so[kGroups][D / 4];
    __shared__ float2 sml[kGroups];
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();
    const int c = blockIdx.x, r = blockIdx.y;
    const Join join = *join_of<F>(p, c);
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
        const float *slot = slot_of<F, D, ROWS>(p, 2 * i + (i == c));
        const float2 ml = *reinterpret_cast<const float2 *>(slot + ROWS * D + 2 * r);
        add(ml.x, ml.y, *reinterpret_cast<const float4 *>(slot + r * D + d));
    }
    so[grp][d / 4] = o;
    if (d == 0) sml[grp] = make_float2(m, l);
    __syncthreads();
    if (grp == 0) {
#pragma unroll
        for (int k = 1; k < kGroups; ++k) add(sml[k].x, sml[k].y, so[k][d / 4]);
        write_row<F>(p, join.start, join.h, join.row0 + r, d, o, m, l);
    }
}

template <class F, int D, int ROWS>
cudaError_t launch_few(const AttentionArgs &args, cudaStream_t stream) {
    AttentionArgs p = args;
    typename F::Maps maps;
    if (!F::template make_maps<D>(p, &maps)) return cudaErrorInvalidValue;
    const int smem = (int)sizeof(Smem<F, D, ROWS>) + 1024;
    cudaError_t e = raise_smem_limit((const void *)attention_kernel<F, D, ROWS>, current_device(), smem);
    if (e != cudaSuccess) return e;
    // No more CTAs than ranges of kMinChunk that the page table allows.
    const int rows_max = (int)std::min<int64_t>((int64_t)p.max_q * p.G, p.few_rows);
    const int64_t items = (int64_t)p.B * p.Hk * ((rows_max + ROWS - 1) / ROWS);
    const int64_t tiles = ((int64_t)p.width * p.P + F::kTile - 1) / F::kTile;
    const int ctas = (int)std::min<int64_t>(kSms * F::per_sm(D, ROWS), std::max<int64_t>(1, (items * (F::kItemCost + tiles) + F::kMinChunk - 1) / F::kMinChunk));
    p.defer = ctas > kManyParts * items;
    e = launch_pdl(attention_kernel<F, D, ROWS>, dim3(ctas), dim3(kThreads), smem, stream, maps, (const AttentionArgs)p);
    if (e != cudaSuccess || !p.defer) return e;
    return launch_pdl(attention_join_kernel<F, D, ROWS>, dim3(ctas, ROWS), dim3(128), 0, stream, (const AttentionArgs)p);
}


template <class F>
cudaError_t launch_few_rows(const AttentionArgs &p, cudaStream_t stream) {
    const bool half = (int64_t)p.max_q * p.G <= 8;
    if (p.D == 128) return half ? launch_few<F, 128, 8>(p, stream) : launch_few<F, 128, 16>(p, stream);
    return half ? launch_few<F, 64, 8>(p, stream) : launch_few<F, 64, 16>(p, stream);
}

template <class F>
size_t few_rows_workspace(int max_q, int G, int D) {
    const int rows = (int64_t)max_q * G <= 8 ? 8 : 16;
    return (size_t)F::kCtas * (sizeof(u64) + sizeof(Join) + 2 * rows * (D + 2) * sizeof(float));
}

inline uint32_t few_rows_timeouts(bool reset) {
    unsigned int v = 0;
    cudaMemcpyFromSymbol(&v, g_attn_timeouts, sizeof(v));
    if (reset) {
        const unsigned int zero = 0;
        cudaMemcpyToSymbol(g_attn_timeouts, &zero, sizeof(zero));
    }
    return v;
}

}  // namespace
}  // namespace lowbit
