// sample.cu -- one token for each row of logits, from a given uniform number
// (lowbit_sample): temperature, min-p, top-k, top-p, then the draw.
//
// Mathematics.  With m the row's maximum and T its temperature,
//     s_i = (x_i - m) / T,  w_i = e^s_i,  W_i = rint(2^30 w_i)  (64-bit sums).
// The weights are whole numbers from here on, so that every sum is exact and the
// result does not depend on the order in which threads or CTAs add: the same
// inputs give the same token on any split.  In the order (x falling, index
// rising) the kept tokens are a prefix:
//     min-p   w_i >= min_p (a falling function of the order),
//     top-k   the first k of those,
//     top-p   of those, the ones before which less than ceil(p Z) has been summed,
//             Z their total.
// The token is the first index whose running total (index order, kept tokens)
// passes floor(u Z'), Z' the kept total.  T <= 0: the first largest logit.  Tokens
// with W_i = 0 (s < -21.5) can never be drawn and count for nothing.
//
// Most tokens cannot be among the kept, and a bound on x that says so costs little:
//     top-k   a value that at least k threads' largest logits reach (bisected with
//             the CTA's counting barrier),
//     top-p   tokens under (1 - p) Z / V together hold less than (1 - p) Z; the mass of
//             those above, in 256 bins of s, says in which bin p Z is reached.
// The tokens above the bound (usually some hundreds) go to one CTA, which sorts them
// and does the rest by itself.  When they are more than its list holds, that of top-p
// takes the tokens of the last bin only and finds the threshold among them (the last
// kept logit, and how many equal ones are kept, in index order); the draw then runs
// over all tokens above it.  Where even that does not fit (flat logits, very large k)
// the threshold is found by counting: bins of s, then ranges of the bits of x, until
// one value is left.
//
// Work split: a cluster of up to 8 CTAs takes a row and holds it in shared memory (each
// logit is read from memory once, and each thread reads back its own vectors; held in
// registers, every pass had to be unrolled over them, and the code no longer fit the
// instruction cache); what CTAs need of each other goes through distributed shared
// memory.  Bound: the chain of cluster-wide steps (three for top-k,
// five to seven for top-p) for few rows, the exponentials of all tokens for many.
#include <algorithm>

#include "common.cuh"
#include "ptx.cuh"

namespace lowbit {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;                        // of the counting path
constexpr int kCoarse = 256;                       // of the top-p bound
constexpr int kList = 2048;                        // tokens that one CTA sorts
constexpr int kMaxCluster = 8;
constexpr int kHeld = 8;                           // 16-byte vectors that a thread holds
constexpr int kMaxVecs = 64;                       // that it may have (the others are read again)
constexpr int kMaxTokens = 131071;                 // of a CTA: sums of 15-bit parts of W stay inside 32 bits
constexpr int kShort = 256;                        // a list that is ordered by counting
constexpr int kWanted = 152;                       // CTAs of a launch, where small batches are split
constexpr int64_t kShare = 128 * 1024;             // bytes of a row that one CTA is left with (see launch_sample)
constexpr int64_t kSmallShare = 8 * 1024;
constexpr float kUnit = 1073741824.0f;             // 2^30
constexpr float kSpan = 21.6f;                     // rint(2^30 e^-s) is 0 beyond
typedef unsigned long long u64;

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ u64 ld_cluster_u64(uint32_t addr) {
    u64 v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void st_cluster_u64(uint32_t addr, u64 v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// Order-preserving map of floats to unsigned integers (-0 like 0), and back.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }

struct alignas(16) Shared {
    union {
        struct {                                   // the list, and the bins of the top-p bound
            u64 list[kList];
            uint32_t coarse_lo[kCoarse], coarse_hi[kCoarse];
        };
        struct {                                   // the counting path: W = lo + 2^15 hi, summed apart in 32 bits
            uint32_t count[kBins], lo[kBins], hi[kBins];
        };
    };
    u64 above[kMaxVecs * kWarps];                  // mass above the cut of each run of a warp's vectors, in index order
    uint32_t equal[kMaxVecs * kWarps];             // tokens equal to it
    u64 pub[2][4];                                 // what this CTA tells the others, in two buffers
    u64 peer[kMaxCluster][4];                      // what each CTA told
    u64 red[kWarps][2];
    u64 found[4];
    uint32_t kmin, kmax;
};

// A row's part in this CTA: vectors (16 bytes) first, first + kThreads, ... of the row's
// aligned memory; `lead` values of the first vector are before the row.
template <int DTYPE>
struct Row {
    static constexpr int kVec = DTYPE == LOWBIT_DTYPE_F32 ? 4 : 8;
    const uint4 *base;
    int lead, V, first, end, nvec;                 // vectors [first, end) are this CTA's, nvec of a thread at most
    bool infinite;                                 // the maximum is +infinity: those count as 0, the others as -infinity
    uint4 *held;                                   // this thread's vectors, kThreads apart (shared memory)

    __device__ __forceinline__ static float get(const uint4 &w, int v) {
        const uint32_t a[4] = {w.x, w.y, w.z, w.w};
        if constexpr (DTYPE == LOWBIT_DTYPE_F32) return __uint_as_float(a[v]);
        const uint16_t h = (uint16_t)(a[v >> 1] >> (v & 1 ? 16 : 0));
        if constexpr (DTYPE == LOWBIT_DTYPE_BF16) return __uint_as_float((uint32_t)h << 16);
        return half_bits_to_float(h);
    }
    __device__ __forceinline__ int vec_of(int it) const { return first + it * kThreads + (int)threadIdx.x; }
    __device__ __forceinline__ int index_of(int it, int v) const { return vec_of(it) * kVec + v - lead; }
    // Vector `it` of this thread; what is not of the row is -infinity.
    __device__ __forceinline__ uint4 load(int it) const {
        constexpr uint32_t kNone = DTYPE == LOWBIT_DTYPE_F32 ? 0xFF800000u : DTYPE == LOWBIT_DTYPE_BF16 ? 0xFF80FF80u : 0xFC00FC00u;
        uint32_t a[4] = {kNone, kNone, kNone, kNone};
        const int vec = vec_of(it);
        if (vec < end) {
            const uint4 w = __ldg(base + vec);
            a[0] = w.x, a[1] = w.y, a[2] = w.z, a[3] = w.w;
            const int i0 = vec * kVec - lead;
            if (i0 < 0 || i0 + kVec > V || infinite) {
#pragma unroll
                for (int v = 0; v < kVec; ++v) {
                    const bool in = i0 + v >= 0 && i0 + v < V;
                    bool none = !in, zero = false;
                    if (infinite) zero = in && get(w, v) == INFINITY, none = !zero;
                    if constexpr (DTYPE == LOWBIT_DTYPE_F32) {
                        if (none || zero) a[v] = none ? kNone : 0u;
                    } else {
                        const uint32_t m = v & 1 ? 0xFFFF0000u : 0xFFFFu;
                        if (none || zero) a[v >> 1] = (a[v >> 1] & ~m) | ((none ? kNone : 0u) & m);
                    }
                }
            }
        }
        return make_uint4(a[0], a[1], a[2], a[3]);
    }
    // Fills `held`.
    __device__ __forceinline__ void hold() {
#pragma unroll 4
        for (int it = 0; it < min(nvec, kHeld); ++it) held[it * kThreads] = load(it);
    }
    template <typename F>
    __device__ __forceinline__ void each(const F &f) const {          // f(x, it, v)
#pragma unroll 1
        for (int it = 0; it < nvec; ++it) {
            const uint4 w = it < kHeld ? held[it * kThreads] : load(it);
#pragma unroll
            for (int v = 0; v < kVec; ++v) f(get(w, v), it, v);
        }
    }
};

// A row's settings, and its cluster.
struct Draw {
    float m, inv_t, T, min_p;
    int rank, ranks, round;                        // in the cluster; exchanges so far
};

struct Token { float s, w; uint32_t W; bool in; };

__device__ __forceinline__ Token weigh(const Draw &r, float x) {
    Token t;
    t.s = __fmul_rn(__fsub_rn(x, r.m), r.inv_t);
    t.w = expf(t.s);
    t.W = __float2uint_rn(__fmul_rn(t.w, kUnit));  // NaN gives 0
    t.in = t.W > 0u && t.w >= r.min_p;
    return t;
}
__device__ __forceinline__ int bin_of(float s) { return min((int)(-s * (kBins / kSpan)), kBins - 1); }

// Cluster-wide exchange: sm.peer[rank] holds every CTA's words (given by its thread
// 0), for all threads.  A CTA overwrites a buffer only after the next exchange's
// barrier, which every reader of it has passed.
__device__ __forceinline__ void exchange(Shared &sm, Draw &r, u64 a, u64 b = 0, u64 c = 0, u64 d = 0) {
    u64 *pub = sm.pub[r.round & 1];
    if (r.ranks == 1) {
        __syncthreads();
        if (threadIdx.x == 0) sm.peer[0][0] = a, sm.peer[0][1] = b, sm.peer[0][2] = c, sm.peer[0][3] = d;
    } else {
        if (threadIdx.x == 0) pub[0] = a, pub[1] = b, pub[2] = c, pub[3] = d;
        ptx::cluster_sync();
        if ((int)threadIdx.x < 4 * r.ranks) {
            const uint32_t rank = threadIdx.x >> 2, w = threadIdx.x & 3;
            sm.peer[rank][w] = ld_cluster_u64(ptx::mapa_shared(ptx::smem_u32(pub + w), rank));
        }
    }
    __syncthreads();
    ++r.round;
}
__device__ __forceinline__ void cluster_barrier(const Draw &r) {
    if (r.ranks == 1) __syncthreads();
    else ptx::cluster_sync();
}

// Exclusive prefix of (a, b) over the CTA's threads in order; the totals in ta, tb.
__device__ __forceinline__ void block_scan(Shared &sm, u64 &a, u64 &b, u64 &ta, u64 &tb) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    u64 ia = a, ib = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 va = __shfl_up_sync(~0u, ia, o), vb = __shfl_up_sync(~0u, ib, o);
        if (lane >= o) ia += va, ib += vb;
    }
    __syncthreads();
    if (lane == 31) sm.red[warp][0] = ia, sm.red[warp][1] = ib;
    __syncthreads();
    a = ia - a, b = ib - b, ta = tb = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        if (i < warp) a += sm.red[i][0], b += sm.red[i][1];
        ta += sm.red[i][0], tb += sm.red[i][1];
    }
}

// a + W in one instruction.
__device__ __forceinline__ void accumulate(u64 &a, uint32_t W) { asm("mad.wide.u32 %0, %1, 1, %0;" : "+l"(a) : "r"(W)); }
// Sum over the warp of values below 2^57.
__device__ __forceinline__ u64 warp_sum(u64 a) {
    return __reduce_add_sync(~0u, (uint32_t)a & 0x3FFFFFFu) + ((u64)__reduce_add_sync(~0u, (uint32_t)(a >> 26) & 0x3FFFFFFu) << 26) +
           ((u64)__reduce_add_sync(~0u, (uint32_t)(a >> 52)) << 52);
}

// floor(u * total), below total.
__device__ __forceinline__ u64 target_of(float u, u64 total) {
    const u64 t = u > 0.f ? (u64)floor((double)u * (double)total) : 0ull;
    return t < total ? t : total - 1;
}

// The mass that a prefix has to reach for top-p: ceil(p total), at least 1.
__device__ __forceinline__ u64 limit_of(float top_p, u64 total) {
    const double want = ceil((double)top_p * (double)total);
    return want > 1.0 ? (u64)want : 1ull;
}

// Sorts the first n entries of the list (n a power of two), rising.  Steps over fewer
// than 32 entries stay in registers.
__device__ __forceinline__ void sort_list(Shared &sm, int n) {
    const int tid = threadIdx.x;
    for (int k = 2; k <= n; k <<= 1) {
        for (int j = k >> 1; j >= 32; j >>= 1) {
            for (int p = tid; p < n / 2; p += kThreads) {
                const int i = ((p & ~(j - 1)) << 1) | (p & (j - 1)), o = i | j;
                const u64 a = sm.list[i], b = sm.list[o];
                if ((a > b) == ((i & k) == 0)) sm.list[i] = b, sm.list[o] = a;
            }
            __syncthreads();
        }
        for (int i0 = 0; i0 < n; i0 += kThreads) {
            const int i = i0 + tid;
            if ((i & ~31) < n) {                   // whole warps
                u64 v = i < n ? sm.list[i] : ~0ull;
                const bool up = (i & k) == 0;
                for (int j = min(k >> 1, 16); j > 0; j >>= 1) {
                    const u64 o = __shfl_xor_sync(~0u, v, j);
                    v = ((i & j) == 0) == up ? (v < o ? v : o) : (v > o ? v : o);
                }
                if (i < n) sm.list[i] = v;
            }
        }
        __syncthreads();
    }
}
__device__ __forceinline__ int power_of_two(int n) { return n <= 2 ? 2 : 1 << (32 - __clz(n - 1)); }

// The kept prefix: tokens whose key is above `key`, and of those equal to it the
// first `quota` in index order (W each).
struct Cut { uint32_t key, W; u64 quota; };

// The counting path.  Narrows the prefix to the tokens before which less than `target`
// tokens (by_mass: units of W) come; the present prefix reaches the target.
template <int DTYPE>
__device__ __noinline__ void narrow(Shared &sm, const Row<DTYPE> &row, Draw &r, bool by_mass, u64 target, Cut &cut) {
    const int tid = threadIdx.x, lane = tid & 31;
    const int slice = kBins / r.ranks, per = max(slice / kThreads, 1);    // bins of a CTA, of a thread
    u64 n_above = 0, m_above = 0;                  // tokens and mass above the range under search
    uint32_t klo = 0u, khi = ~0u;                  // its keys
    int bin = 0, shift = 0;
    for (int level = 0;; ++level) {
        // Of the tokens above the present cut's key, those in the range.
        auto inside = [&](uint32_t k, float x, Token &t) {
            if (k <= cut.key || (level > 1 && (k < klo || k > khi))) return false;
            t = weigh(r, x);
            return t.in && (level != 1 || bin_of(t.s) == bin);
        };
        if (level > 0) {
            // The keys that the range really holds; one: that is the threshold.
            if (tid == 0) sm.kmin = ~0u, sm.kmax = 0u;
            __syncthreads();
            uint32_t lo = ~0u, hi = 0u;
            row.each([&](float x, int, int) {
                const uint32_t k = ordered(x);
                Token t;
                if (inside(k, x, t)) lo = min(lo, k), hi = max(hi, k);
            });
            lo = __reduce_min_sync(~0u, lo);
            hi = __reduce_max_sync(~0u, hi);
            if (lane == 0) atomicMin(&sm.kmin, lo), atomicMax(&sm.kmax, hi);
            __syncthreads();
            exchange(sm, r, sm.kmin, sm.kmax);
            klo = ~0u, khi = 0u;
            for (int i = 0; i < r.ranks; ++i)
                klo = min(klo, (uint32_t)sm.peer[i][0]), khi = max(khi, (uint32_t)sm.peer[i][1]);
            if (klo >= khi) break;
            shift = max(0, 21 - __clz(khi - klo));                       // ranges of keys: at most 2048
        }
        for (int i = tid; i < kBins; i += kThreads) sm.count[i] = sm.lo[i] = sm.hi[i] = 0u;
        __syncthreads();
        row.each([&](float x, int, int) {
            const uint32_t k = ordered(x);
            Token t;
            if (!inside(k, x, t)) return;
            const int at = level == 0 ? bin_of(t.s) : (int)((khi - k) >> shift);
            atomicAdd(&sm.count[at], 1u);
            atomicAdd(&sm.lo[at], t.W & 0x7FFFu);
            atomicAdd(&sm.hi[at], t.W >> 15);
        });
        cluster_barrier(r);
        // This CTA's slice of the bins, summed over the cluster.
        u64 cn[kBins / kThreads], cm[kBins / kThreads], en = 0, em = 0, tn, tm;
#pragma unroll
        for (int q = 0; q < kBins / kThreads; ++q) {
            cn[q] = cm[q] = 0;
            if (q < per && tid * per + q < slice) {
                const uint32_t at = (uint32_t)(r.rank * slice + tid * per + q);
                for (int i = 0; i < r.ranks; ++i) {
                    cn[q] += ld_cluster_u32(ptx::mapa_shared(ptx::smem_u32(&sm.count[at]), i));
                    cm[q] += ld_cluster_u32(ptx::mapa_shared(ptx::smem_u32(&sm.lo[at]), i)) +
                             ((u64)ld_cluster_u32(ptx::mapa_shared(ptx::smem_u32(&sm.hi[at]), i)) << 15);
                }
            }
            en += cn[q], em += cm[q];
        }
        block_scan(sm, en, em, tn, tm);
        if (tid == 0) sm.found[0] = 0;
        exchange(sm, r, tn, tm);                   // also the barrier before the bins are cleared again
        en += n_above, em += m_above;
        for (int i = 0; i < r.rank; ++i) en += sm.peer[i][0], em += sm.peer[i][1];
#pragma unroll
        for (int q = 0; q < kBins / kThreads; ++q) {
            const u64 before = by_mass ? em : en, add = by_mass ? cm[q] : cn[q];
            if (before < target && before + add >= target) {
                sm.found[0] = (u64)(r.rank * slice + tid * per + q + 1);
                sm.found[1] = en;
                sm.found[2] = em;
            }
            en += cn[q], em += cm[q];
        }
        // If no bin reaches the target, it falls among the tokens of the present cut's key.
        u64 all_n = n_above, all_m = m_above;
        for (int i = 0; i < r.ranks; ++i) all_n += sm.peer[i][0], all_m += sm.peer[i][1];
        __syncthreads();
        exchange(sm, r, sm.found[0], sm.found[1], sm.found[2]);
        int hit = -1;
        for (int i = 0; i < r.ranks; ++i)
            if (sm.peer[i][0] != 0) hit = i;
        if (hit < 0) {
            const u64 need = by_mass ? (target - all_m + cut.W - 1) / cut.W : target - all_n;
            cut.quota = need < cut.quota ? need : cut.quota;
            return;
        }
        const int at = (int)sm.peer[hit][0] - 1;
        n_above = sm.peer[hit][1], m_above = sm.peer[hit][2];
        if (level == 0) {
            bin = at;
        } else {
            khi -= (uint32_t)at << shift;
            klo = max(klo, khi - min(khi, (1u << shift) - 1u));
        }
        __syncthreads();
    }
    // klo == khi: every token of the range has this key.
    cut.key = khi;
    cut.W = weigh(r, unordered(khi)).W;
    cut.quota = by_mass ? (target - m_above + cut.W - 1) / cut.W : target - n_above;
}

// Mass above the cut and tokens equal to it, for each run of a warp's vectors (in index
// order: vector number, then warp) in sm.above and sm.equal, and of every CTA in sm.peer.
// upto: tokens above it are in sm.above already (a key; ~0: none are).
template <int DTYPE>
__device__ __forceinline__ void tally(Shared &sm, const Row<DTYPE> &row, Draw &r, const Cut &cut, uint32_t upto) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float from = cut.key == 0 ? -INFINITY : unordered(cut.key), to = upto == ~0u ? INFINITY : unordered(upto);
    u64 above = 0, all_above = 0;
    uint32_t equal = 0, all_equal = 0;
    row.each([&](float x, int it, int v) {
        if (x >= from && x <= to) {
            const Token t = weigh(r, x);
            if (t.in) {
                if (x > from) accumulate(above, t.W);
                else ++equal;
            }
        }
        if (v == Row<DTYPE>::kVec - 1) {
            above = warp_sum(above);
            equal = __reduce_add_sync(~0u, equal);
            if (lane == 0) {
                if (upto != ~0u) above += sm.above[it * kWarps + warp];
                sm.above[it * kWarps + warp] = above, sm.equal[it * kWarps + warp] = equal;
                all_above += above, all_equal += equal;
            }
            above = 0, equal = 0;
        }
    });
    u64 a = lane == 0 ? all_above : 0, b = lane == 0 ? all_equal : 0, ta, tb;
    block_scan(sm, a, b, ta, tb);
    exchange(sm, r, ta, tb);
}

// The draw from all of the row's tokens above the cut, after tally.
template <int DTYPE>
__device__ __forceinline__ void draw_all(Shared &sm, const Row<DTYPE> &row, const Draw &r, const Cut &cut, const SampleArgs &p, int b) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto kept = [&](u64 above, u64 equal, u64 before) {       // of a run with `before` equal tokens before it
        const u64 left = cut.quota > before ? cut.quota - before : 0;
        return above + (equal < left ? equal : left) * cut.W;
    };
    u64 total = 0, start = 0, mine = 0, eq = 0, eq0 = 0;      // start, eq0: before this CTA
    for (int i = 0; i < r.ranks; ++i) {
        const u64 k = kept(sm.peer[i][0], sm.peer[i][1], eq);
        if (i == r.rank) start = total, eq0 = eq, mine = k;
        total += k;
        eq += sm.peer[i][1];
    }
    const u64 target = target_of(p.u[b], total);
    if (target < start || target >= start + mine) return;     // the same for the whole CTA
    // The run in which it falls: two runs a thread at most.
    const int runs = row.nvec * kWarps, per = (runs + kThreads - 1) / kThreads;
    u64 e = 0, k = 0, te, tk, zero = 0, tz;
    for (int q = 0; q < per; ++q)
        if (tid * per + q < runs) e += sm.equal[tid * per + q];
    block_scan(sm, e, zero, te, tz);
    e += eq0;
    u64 run = e;
    for (int q = 0; q < per; ++q)
        if (tid * per + q < runs) {
            k += kept(sm.above[tid * per + q], sm.equal[tid * per + q], run);
            run += sm.equal[tid * per + q];
        }
    u64 z2 = 0;
    block_scan(sm, k, z2, tk, tz);
    k += start;
    for (int q = 0; q < per; ++q)
        if (tid * per + q < runs) {
            const int at = tid * per + q;
            const u64 add = kept(sm.above[at], sm.equal[at], e);
            if (target >= k && target < k + add) sm.found[0] = (u64)at, sm.found[1] = k, sm.found[2] = e;
            k += add;
            e += sm.equal[at];
        }
    __syncthreads();
    const int at = (int)sm.found[0];
    if (at % kWarps != warp) return;
    // The lane, then the token.
    const uint4 w = row.load(at / kWarps);
    u64 above = 0;
    uint32_t equal = 0;
#pragma unroll
    for (int v = 0; v < Row<DTYPE>::kVec; ++v) {
        const float x = Row<DTYPE>::get(w, v);
        const uint32_t key = ordered(x);
        const Token t = weigh(r, x);
        if (t.in && key > cut.key) above += t.W;
        if (t.in && key == cut.key) ++equal;
    }
    u64 ie = equal;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 v = __shfl_up_sync(~0u, ie, o);
        if (lane >= o) ie += v;
    }
    u64 seen = sm.found[2] + ie - equal, ik = kept(above, equal, seen);
    const u64 own = ik;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 v = __shfl_up_sync(~0u, ik, o);
        if (lane >= o) ik += v;
    }
    u64 sum = sm.found[1] + ik - own;
    if (target < sum || target >= sum + own) return;
#pragma unroll
    for (int v = 0; v < Row<DTYPE>::kVec; ++v) {
        const float x = Row<DTYPE>::get(w, v);
        const uint32_t key = ordered(x);
        const Token t = weigh(r, x);
        const bool tie = t.in && key == cut.key;
        const u64 add = (t.in && key > cut.key) || (tie && seen < cut.quota) ? t.W : 0;
        seen += tie;
        if (target >= sum && target < sum + add) {
            p.token[b] = row.index_of(at / kWarps, v);
            if (p.logprob != nullptr) p.logprob[b] = t.s - logf((float)total * (1.f / kUnit));
        }
        sum += add;
    }
}

// The cut of the list's n tokens, before which `before` units of mass come: the last kept
// key and how many of it are kept (this CTA's alone).
__device__ __forceinline__ Cut cut_listed(Shared &sm, const Draw &r, int n, u64 before, u64 limit) {
    constexpr int kPer = kList / kThreads;
    const int tid = threadIdx.x, size = power_of_two(n);
    for (int i = n + tid; i < size; i += kThreads) sm.list[i] = ~0ull;
    if (tid == 0) sm.found[0] = 0;
    __syncthreads();
    sort_list(sm, size);
    u64 W[kPer], sum = 0, z = 0, ts, tz;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
        const int i = tid * kPer + q;
        W[q] = i < n ? weigh(r, unordered(~(uint32_t)(sm.list[i] >> 32))).W : 0;
        sum += W[q];
    }
    block_scan(sm, sum, z, ts, tz);
    sum += before;
    u64 kept = 0;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
        kept += tid * kPer + q < n && sum < limit;
        sum += W[q];
    }
    z = 0;
    block_scan(sm, kept, z, ts, tz);               // ts: kept in all
    const uint32_t key = ~(uint32_t)(sm.list[ts - 1] >> 32);
    u64 same = 0;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
        const int i = tid * kPer + q;
        same += i < (int)ts && ~(uint32_t)(sm.list[i] >> 32) == key;
    }
    z = 0;
    u64 quota;
    block_scan(sm, same, z, quota, tz);
    return Cut{key, weigh(r, unordered(key)).W, quota};
}

// Writes the drawn token.
template <int DTYPE>
__device__ __forceinline__ void write_token(const Row<DTYPE> &row, const Draw &r, int i, u64 mass, const SampleArgs &p, int b) {
    p.token[b] = i;
    if (p.logprob == nullptr) return;
    float x = r.m;
    if (!row.infinite) {
        const int at = i + row.lead;
        const uint4 w = __ldg(row.base + at / Row<DTYPE>::kVec);
#pragma unroll
        for (int v = 0; v < Row<DTYPE>::kVec; ++v)
            if (v == at % Row<DTYPE>::kVec) x = Row<DTYPE>::get(w, v);
    }
    p.logprob[b] = weigh(r, x).s - logf((float)mass * (1.f / kUnit));
}

// The rest of the work on a short list, a token a thread: places and the mass before each
// by comparing with all others.
template <int DTYPE>
__device__ __forceinline__ void draw_short(Shared &sm, const Row<DTYPE> &row, const Draw &r, int n, int top_k, float top_p, u64 total,
                                           const SampleArgs &p, int b) {
    const int tid = threadIdx.x;
    u64 *weight = sm.list + kShort;                // W beside the entries
    const u64 me = tid < n ? sm.list[tid] : ~0ull;
    const Token t = weigh(r, unordered(~(uint32_t)(me >> 32)));
    const uint32_t W = tid < n && t.in ? t.W : 0u;
    if (tid < kShort) weight[tid] = W;
    __syncthreads();
    if (tid >= ((n + 31) & ~31)) return;           // whole warps
    int place = 0;
    u64 before = 0, all = 0;
    for (int j = 0; j < n; ++j) {
        const bool earlier = sm.list[j] < me;
        place += earlier;
        if (earlier) before += weight[j];
    }
    // Of the first top_k (all): the mass.
    if (total == 0) {
        // Places are a permutation: the mass before place top_k is the largest of before + W there.
        u64 upto = tid < n && (top_k <= 0 || place < top_k) ? before + W : 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const u64 v = __shfl_xor_sync(~0u, upto, o);
            upto = v > upto ? v : upto;
        }
        if ((tid & 31) == 0) sm.red[tid >> 5][0] = upto;
        ptx::named_sync(1, (uint32_t)((n + 31) & ~31));
        for (int i = 0; i < (n + 31) / 32; ++i) all = sm.red[i][0] > all ? sm.red[i][0] : all;
    } else {
        all = total;
    }
    const u64 limit = top_p < 1.f ? limit_of(top_p, all) : ~0ull;
    const bool kept = W != 0 && (top_k <= 0 || place < top_k) && before < limit;
    ptx::named_sync(1, (uint32_t)((n + 31) & ~31));
    if (tid < kShort) weight[tid] = kept ? W : 0;
    ptx::named_sync(1, (uint32_t)((n + 31) & ~31));
    // The running total in index order, and the whole.
    const uint32_t index = (uint32_t)me;
    u64 ahead = 0, mass = 0;
    for (int j = 0; j < n; ++j) {
        const u64 w = weight[j];
        mass += w;
        if ((uint32_t)sm.list[j] < index) ahead += w;
    }
    const u64 target = target_of(p.u[b], mass);
    if (kept && target >= ahead && target < ahead + W) write_token(row, r, (int)index, mass, p, b);
}

// The rest of the work on the list of n tokens (this CTA's alone): order, top-k, top-p,
// draw.  total: mass of all tokens within min-p (0: that of the first top_k of the list).
template <int DTYPE>
__device__ __forceinline__ void draw_listed(Shared &sm, const Row<DTYPE> &row, const Draw &r, int n, int top_k, float top_p, u64 total,
                                            const SampleArgs &p, int b) {
    constexpr int kPer = kList / kThreads;
    const int tid = threadIdx.x;
    int size = power_of_two(n);
    for (int i = n + tid; i < size; i += kThreads) sm.list[i] = ~0ull;
    __syncthreads();
    sort_list(sm, size);                           // ~key, index: x falling, index rising
    // Weights in that order, kPer neighbours a thread.
    u64 W[kPer], idx[kPer], sum = 0, z = 0, all, tz;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
        const int i = tid * kPer + q;
        W[q] = idx[q] = 0;
        if (i < n) {
            const Token t = weigh(r, unordered(~(uint32_t)(sm.list[i] >> 32)));
            if (t.in && (top_k <= 0 || i < top_k)) W[q] = t.W;
            idx[q] = sm.list[i] & 0xFFFFFFFFull;
        }
        sum += W[q];
    }
    block_scan(sm, sum, z, all, tz);
    if (total == 0) total = all;
    const u64 limit = top_p < 1.f ? limit_of(top_p, total) : ~0ull;
    u64 kept = 0, count = 0;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
        const u64 w = W[q];
        if (sum >= limit) W[q] = 0;
        sum += w;
        kept += W[q];
        count += W[q] != 0;
    }
    // The kept in index order.
    u64 before = kept, place = count, mass, left;
    block_scan(sm, before, place, mass, left);
    size = power_of_two((int)left);
    for (int i = (int)left + tid; i < size; i += kThreads) sm.list[i] = ~0ull;
#pragma unroll
    for (int q = 0; q < kPer; ++q)
        if (W[q] != 0) sm.list[place++] = idx[q] << 32 | W[q];
    __syncthreads();
    sort_list(sm, size);
    u64 own = 0;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
        const int i = tid * kPer + q;
        W[q] = i < (int)left ? sm.list[i] & 0xFFFFFFFFull : 0;
        own += W[q];
    }
    u64 zero = 0;
    block_scan(sm, own, zero, all, tz);
    const u64 target = target_of(p.u[b], mass);
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
        if (target >= own && target < own + W[q])
            write_token(row, r, (int)(sm.list[tid * kPer + q] >> 32), mass, p, b);
        own += W[q];
    }
}

template <int DTYPE>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs p) {
    constexpr int kVec = Row<DTYPE>::kVec;
    extern __shared__ __align__(16) uint8_t raw[];
    Shared &sm = *reinterpret_cast<Shared *>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();

    Draw r;
    uint32_t ranks;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ranks));
    r.ranks = (int)ranks, r.rank = (int)ptx::cluster_ctarank(), r.round = 0;
    const int b = (int)(blockIdx.x / ranks);
    Row<DTYPE> row;
    {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p.logits) + (int64_t)b * p.row_stride * (DTYPE == LOWBIT_DTYPE_F32 ? 4 : 2);
        row.base = reinterpret_cast<const uint4 *>(at & ~(uintptr_t)15);
        row.lead = (int)(at & 15) / (16 / kVec);
        row.V = p.V;
        row.infinite = false;
        const int all = (row.lead + p.V + kVec - 1) / kVec, part = (all + r.ranks - 1) / r.ranks;
        row.first = r.rank * part;
        row.end = min(row.first + part, all);
        row.nvec = (part + kThreads - 1) / kThreads;
    }
    row.held = reinterpret_cast<uint4 *>(raw + sizeof(Shared)) + tid;
    row.hold();
    r.T = p.temperature != nullptr ? p.temperature[b] : p.temperature_all;
    const float top_p = p.top_p != nullptr ? p.top_p[b] : p.top_p_all;
    const float min_p = p.min_p != nullptr ? p.min_p[b] : p.min_p_all;
    const int top_k = p.top_k != nullptr ? p.top_k[b] : p.top_k_all;
    const bool greedy = !(r.T > 0.f);

    // The largest logit of the thread, the CTA and the row.
    float own = -INFINITY;                         // fmaxf leaves NaN out
    row.each([&](float x, int, int) { own = fmaxf(own, x); });
    {
        const uint32_t k = __reduce_max_sync(~0u, ordered(own));
        if (lane == 0) sm.red[warp][0] = k;
    }
    __syncthreads();
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) top = max(top, (uint32_t)sm.red[i][0]);
    // A value that at least ceil(k / ranks) threads' logits reach, in every CTA: the k
    // first tokens are not below the least of these.
    const bool by_k = !greedy && top_k > 0 && top_k <= (kThreads - kThreads / 8) * r.ranks && top_k <= kList / 2;
    uint32_t reach = 0;
    if (by_k) {
        const int need = (top_k + r.ranks - 1) / r.ranks;
        float hi = unordered(top), lo = hi - 22.f * r.T;
        if (lo > -INFINITY && __syncthreads_count(own >= lo) >= need) {
            for (int i = 0; i < 12; ++i) {
                const float mid = 0.5f * (lo + hi);
                if (__syncthreads_count(own >= mid) >= need) lo = mid;
                else hi = mid;
            }
            reach = ordered(lo);
        }
    }
    exchange(sm, r, top, reach);
    reach = ~0u;
    for (int i = 0; i < r.ranks; ++i) top = max(top, (uint32_t)sm.peer[i][0]), reach = min(reach, (uint32_t)sm.peer[i][1]);
    r.m = unordered(top);
    if (r.m == -INFINITY) {                        // nothing can be drawn
        if (r.rank == 0 && tid == 0) {
            p.token[b] = -1;
            if (p.logprob != nullptr) p.logprob[b] = -INFINITY;
        }
        cluster_barrier(r);                        // others may still read this CTA's words
        return;
    }
    if (greedy) {
        int first = INT32_MAX;
        row.each([&](float x, int it, int v) {
            if (x == r.m) first = min(first, row.index_of(it, v));
        });
        first = __reduce_min_sync(~0u, first);
        __syncthreads();
        if (lane == 0) sm.red[warp][0] = (u64)first;
        __syncthreads();
        for (int i = 0; i < kWarps; ++i) first = min(first, (int)sm.red[i][0]);
        exchange(sm, r, (u64)first);
        for (int i = 0; i < r.ranks; ++i) first = min(first, (int)sm.peer[i][0]);
        if (r.rank == 0 && tid == 0) {
            p.token[b] = first;
            if (p.logprob != nullptr) p.logprob[b] = 0.f;
        }
        cluster_barrier(r);
        return;
    }
    if (r.m == INFINITY) {
        row.infinite = true;
        r.m = 0.f;
        row.hold();
    }
    r.inv_t = fminf(__fdiv_rn(1.f, r.T), 3.402823466e38f);
    r.min_p = fminf(min_p, 1.f);                   // the largest logit is always kept

    u64 total = 0, tokens = 0;                     // mass and number of the tokens within min-p
    const bool by_p = top_p < 1.f, counted = !by_k && (by_p || top_k > 0);
    float per = 0.f;                               // top-p: bins of a unit of s
    if (counted) {
        float floor_s = 0.f, above = INFINITY;     // tokens below are not binned
        if (by_p) {
            // The threads' largest tokens give a lower bound of Z.
            const Token t = weigh(r, row.infinite ? (own == INFINITY ? 0.f : -INFINITY) : own);
            u64 least = t.in ? t.W : 0, z = 0, tl, tz;
            block_scan(sm, least, z, tl, tz);
            for (int i = tid; i < kCoarse; i += kThreads) sm.coarse_lo[i] = sm.coarse_hi[i] = 0u;
            exchange(sm, r, tl);
            tl = 0;
            for (int i = 0; i < r.ranks; ++i) tl += sm.peer[i][0];
            const float share = (1.f - top_p) * (float)tl / (float)p.V * (1.f / kUnit);
            floor_s = fmaxf(share > 0.f ? logf(share) - 1e-3f : -kSpan, -kSpan);
            per = kCoarse / -floor_s;
            above = r.m + (floor_s - 1e-3f) * r.T - fabsf(r.m) * 1e-6f;
        }
        u64 mass = 0;
        uint32_t n = 0;
        row.each([&](float x, int, int) {
            const Token t = weigh(r, x);
            if (t.in) {
                accumulate(mass, t.W), ++n;
                if (x >= above) {
                    // In parts of 15 bits, large weights to the nearest 2^15: one addition mostly.
                    const int at = min((int)(-t.s * per), kCoarse - 1);
                    const uint32_t hi = t.W < 1u << 22 ? t.W >> 15 : (t.W + (1u << 14)) >> 15;
                    if (t.W < 1u << 22) atomicAdd(&sm.coarse_lo[at], t.W & 0x7FFFu);
                    if (hi != 0u) atomicAdd(&sm.coarse_hi[at], hi);
                }
            }
        });
        u64 nn = n, tm, tn;
        block_scan(sm, mass, nn, tm, tn);
        exchange(sm, r, tm, tn);
        for (int i = 0; i < r.ranks; ++i) total += sm.peer[i][0], tokens += sm.peer[i][1];
    }
    const bool cut_k = top_k > 0 && (by_k || (u64)top_k < tokens);
    Cut cut{0u, 1u, 0};
    if (cut_k || by_p) {
        // No token below `bound` is kept (margins for rounding only make it lower).
        float bound = r.m - 21.7f * r.T - fabsf(r.m) * 1e-6f, over = INFINITY;
        int last = -1;                             // top-p: the bin of s in which the limit is reached
        const u64 limit = by_p && counted ? limit_of(top_p, total) : 0;
        const bool listing = by_k || !cut_k;
        if (by_k) {
            if (!row.infinite) bound = fmaxf(bound, unordered(reach));
        } else if (listing) {
            // By the bins' rounded sums: what is found from them is checked exactly below.
            u64 sum = 0, z = 0, tm, tz;
            if (tid < kCoarse)
                for (int i = 0; i < r.ranks; ++i)
                    sum += ld_cluster_u32(ptx::mapa_shared(ptx::smem_u32(&sm.coarse_lo[tid]), i)) +
                           ((u64)ld_cluster_u32(ptx::mapa_shared(ptx::smem_u32(&sm.coarse_hi[tid]), i)) << 15);
            const u64 of_bin = sum;
            if (tid == 0) sm.found[0] = kCoarse;
            block_scan(sm, sum, z, tm, tz);
            if (tid < kCoarse && sum < limit && sum + of_bin >= limit) sm.found[0] = (u64)tid;
            __syncthreads();
            last = (int)sm.found[0];
            bound = fmaxf(bound, r.m - ((float)(last + 1) / per + 1e-3f) * r.T - fabsf(r.m) * 1e-6f);
            over = r.m - ((float)last / per - 1e-3f) * r.T + fabsf(r.m) * 1e-6f;      // above: an earlier bin
        }
        if (listing) {
            // How many tokens there are from the bound on, and between it and `over`; the mass
            // above `over` of each run, of the CTA, and that between.
            uint32_t n_mine = 0, n_between = 0;
            u64 run = 0, above = 0, between = 0;
            row.each([&](float x, int it, int v) {
                if (x >= bound) {
                    ++n_mine;
                    if (last >= 0) {
                        const Token t = weigh(r, x);
                        if (t.in) {
                            if (x > over) accumulate(run, t.W);
                            else accumulate(between, t.W), ++n_between;
                        }
                    }
                }
                if (v == kVec - 1 && last >= 0) {
                    run = warp_sum(run);
                    if (lane == 0) sm.above[it * kWarps + warp] = run, above += run;
                    run = 0;
                }
            });
            u64 mine = n_mine, mine_between = n_between, of_cta, of_between, cta_above = 0, cta_between = 0;
            block_scan(sm, mine, mine_between, of_cta, of_between);
            if (last >= 0) block_scan(sm, above, between, cta_above, cta_between);
            exchange(sm, r, of_cta, of_between, cta_above, cta_between);
            u64 n = 0, n_bin = 0, before = 0, of_bin = 0;
            for (int i = 0; i < r.ranks; ++i) {
                if (i == r.rank) mine += n, mine_between += n_bin;
                n += sm.peer[i][0], n_bin += sm.peer[i][1], before += sm.peer[i][2], of_bin += sm.peer[i][3];
            }
            // The list may hold all of them, or those of the last bin if the limit is indeed there.
            const bool whole = n <= (u64)kList && (last < 0 || before + of_bin >= limit);
            const bool bin_only = !whole && last >= 0 && n_bin > 0 && n_bin <= (u64)kList && before < limit && before + of_bin >= limit;
            if (whole || bin_only) {
                // They go to the first CTA's list, each CTA and thread at its place.
                uint32_t at = ptx::mapa_shared(ptx::smem_u32(sm.list), 0u) + (uint32_t)(whole ? mine : mine_between) * 8u;
                const float to = whole ? INFINITY : over;
                if ((whole ? n_mine : n_between) > 0)
                    row.each([&](float x, int it, int v) {
                        if (x >= bound && x <= to && (whole || weigh(r, x).in)) {
                            st_cluster_u64(at, (u64)(uint32_t)~ordered(x) << 32 | (uint32_t)row.index_of(it, v));
                            at += 8;
                        }
                    });
                cluster_barrier(r);
            }
            if (whole) {
                if (r.rank != 0) return;
                if (n <= (u64)kShort) draw_short(sm, row, r, (int)n, cut_k ? top_k : 0, top_p, counted ? total : 0, p, b);
                else draw_listed(sm, row, r, (int)n, cut_k ? top_k : 0, top_p, counted ? total : 0, p, b);
                return;                            // nobody reads another's shared memory any more
            }
            if (bin_only) {
                if (r.rank == 0) cut = cut_listed(sm, r, (int)n_bin, before, limit);
                exchange(sm, r, cut.key, cut.quota, cut.W);
                cut = Cut{(uint32_t)sm.peer[0][0], (uint32_t)sm.peer[0][2], sm.peer[0][1]};
                __syncthreads();
                tally(sm, row, r, cut, ordered(over));
                draw_all(sm, row, r, cut, p, b);
                cluster_barrier(r);
                return;
            }
        }
        // The counting path.
        if (!counted) {
            u64 mass = 0;
            uint32_t n = 0;
            row.each([&](float x, int, int) {
                const Token t = weigh(r, x);
                if (t.in) mass += t.W, ++n;
            });
            u64 nn = n, tm, tn;
            block_scan(sm, mass, nn, tm, tn);
            exchange(sm, r, tm, tn);
            total = tokens = 0;
            for (int i = 0; i < r.ranks; ++i) total += sm.peer[i][0], tokens += sm.peer[i][1];
        }
        if (top_k > 0 && (u64)top_k < tokens) {
            narrow(sm, row, r, false, (u64)top_k, cut);
            tally(sm, row, r, cut, ~0u);
            total = cut.quota * cut.W;
            for (int i = 0; i < r.ranks; ++i) total += sm.peer[i][0];
        }
        if (by_p) narrow(sm, row, r, true, limit_of(top_p, total), cut);
    }
    tally(sm, row, r, cut, ~0u);
    draw_all(sm, row, r, cut, p, b);
    cluster_barrier(r);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &args, cudaStream_t stream) {
    // CTAs of a row: as many as its tokens need, then more while each has over kShare bytes,
    // and for small batches while there are SMs for them and over kSmallShare bytes each.
    // (A step over the cluster costs the same for any share, and rows differ in their work,
    // so that more and smaller CTAs even out: 256 rows of 128256 floats take 244 us with one
    // CTA each, 180 with two, 169 with four and 193 with eight; 192 rows of 19439 floats 18.8
    // us with one and 24.8 with two.)
    const int64_t bytes = (int64_t)args.V * (args.dtype == LOWBIT_DTYPE_F32 ? 4 : 2);
    int ranks = 1;
    while (ranks < kMaxCluster && (bytes + 32 > (int64_t)ranks * kThreads * kMaxVecs * 16 || args.V > ranks * kMaxTokens - 16 ||
                                   bytes > ranks * kShare ||
                                   (bytes > ranks * kSmallShare && (int64_t)args.B * ranks < kWanted)))
        ranks *= 2;
    const auto kernel = args.dtype == LOWBIT_DTYPE_F32    ? sample_kernel<LOWBIT_DTYPE_F32>
                        : args.dtype == LOWBIT_DTYPE_BF16 ? sample_kernel<LOWBIT_DTYPE_BF16>
                                                          : sample_kernel<LOWBIT_DTYPE_F16>;
    const int64_t vecs = (bytes / 16 + 2 + ranks - 1) / ranks, held = std::min<int64_t>((vecs + kThreads - 1) / kThreads, kHeld);
    const int smem = (int)(sizeof(Shared) + held * kThreads * 16);
    const cudaError_t e = raise_smem_limit((const void *)kernel, current_device(), (int)sizeof(Shared) + kHeld * kThreads * 16);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ranks * (unsigned)args.B);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ranks;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, args);
}

}  // namespace lowbit
