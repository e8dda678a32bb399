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
//             those above, in 1024 bins of s, says in which bin p Z is reached.
// The tokens above the bound (usually some hundreds) go to one CTA, which does the rest by
// itself: each of top-k, top-p and the draw looks for one token of its list, by 512 bins
// of the range that may hold it (two or three passes over the list; ordering the list
// took twice as long).  When they are more than the list holds, that of top-p takes the
// tokens of the last bin only and finds the last kept one among them; the draw then runs
// over all tokens, by the sums of runs of them.  Where even that does not fit (flat
// logits, very large k) the threshold is found by counting: bins of s, then ranges of the
// bits of x, until one value is left.
//
// Work split: a cluster of up to 8 CTAs takes a row and holds it in shared memory (each
// logit is read from memory once, and each thread reads back its own vectors; held in
// registers, every pass had to be unrolled over them, and the code no longer fit the
// instruction cache); what CTAs need of each other goes through distributed shared
// memory.  Bound: for few rows the chain of some twenty barriers of the CTA and three
// (top-k) to six (top-p) of the cluster, for many the instructions of the pass that
// weighs all tokens (some 35 a token, of which two at a quarter of the rate or less).
// One row of 128256 in bfloat16 takes 16 us, 64 rows of them with top-p 54 us (0.3 TB/s),
// 256 rows in float32 of mixed settings 137 us (1.0 TB/s).
#include <algorithm>

#include "common.cuh"
#include "ptx.cuh"

namespace lowbit {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;                        // of the counting path
constexpr int kCoarse = 1024;                      // of the top-p bound
constexpr int kList = 2048;                        // tokens of the list, less one
constexpr int kMaxCluster = 8;
constexpr int kHeld = 8;                           // 16-byte vectors that a thread holds
constexpr int kMaxVecs = 64;                       // that it may have (the others are read again)
constexpr int kFew = 32;                           // of its tokens that are compared all with all
constexpr int kMaxTokens = 131071;                 // of a CTA: sums of 15-bit parts of W stay inside 32 bits
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

__device__ __forceinline__ void add_cluster_u64(uint32_t addr, u64 v) {
    asm volatile("red.relaxed.cluster.shared::cluster.add.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// Order-preserving map of floats to unsigned integers (-0 like 0), and back.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }

// A token's place among the others as one number: larger logits, then lower indexes,
// are larger.
constexpr int kIndexBits = 20;
constexpr u64 kIndexMask = (1u << kIndexBits) - 1;
__device__ __forceinline__ u64 place_of(float x, int index) { return (u64)ordered(x) << kIndexBits | (kIndexMask - (uint32_t)index); }
__device__ __forceinline__ int index_at(u64 place) { return (int)(kIndexMask - (place & kIndexMask)); }

struct alignas(16) Shared {
    union {
        struct {                                   // the list with its weights, and the bins of the top-p bound
            u64 list[kList];
            uint32_t weight[kList];
            uint32_t coarse[kCoarse];              // each at a scale of its own (scale_bits)
        };
        struct {                                   // the counting path: W = lo + 2^15 hi, summed apart in 32 bits
            uint32_t count[kBins], lo[kBins], hi[kBins];
        };
    };
    u64 runs[kMaxVecs * kWarps];                   // mass (or tokens) of each run of a warp's vectors, in index order
    u64 pub[2][4];                                 // what this CTA tells the others, in two buffers
    u64 peer[kMaxCluster][4];                      // what each CTA told
    u64 red[kWarps][2];
    u64 found[4];
    u64 few[kFew];                                 // of a search
    uint32_t few_weight[kFew];
    int fews;
    uint32_t kmin, kmax;
};

// A row's part in this CTA: vectors (16 bytes) first, first + kThreads, ... of the row's
// aligned memory; `lead` values of the first vector are before the row.
template <int DTYPE>
struct Row {
    static constexpr int kVec = DTYPE == LOWBIT_DTYPE_F32 ? 4 : 8;
    const uint4 *base;
    int lead, V, all, part, first, end, nvec;      // vectors [first, end) of `all` are this CTA's (part), nvec of a thread at most
    bool infinite;                                 // the maximum is +infinity: those count as 0, the others as -infinity
    uint4 *held;                                   // this thread's vectors, kThreads apart (shared memory)

    __device__ __forceinline__ static float get(const uint4 &w, int v) {
        const uint32_t a[4] = {w.x, w.y, w.z, w.w};
        if constexpr (DTYPE == LOWBIT_DTYPE_F32) return __uint_as_float(a[v]);
        const uint16_t h = (uint16_t)(a[v >> 1] >> (v & 1 ? 16 : 0));
        if constexpr (DTYPE == LOWBIT_DTYPE_BF16) return __uint_as_float((uint32_t)h << 16);
        return half_bits_to_float(h);
    }
    // The largest of a vector's values; NaN are left out.
    __device__ __forceinline__ static float largest(const uint4 &w) {
        if constexpr (DTYPE == LOWBIT_DTYPE_F32) {
            return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)), fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
        } else {
            const uint32_t a = larger2(larger2(w.x, w.y), larger2(w.z, w.w));
            return fmaxf(get(make_uint4(a, 0u, 0u, 0u), 0), get(make_uint4(a, 0u, 0u, 0u), 1));
        }
    }
    __device__ __forceinline__ static uint32_t larger2(uint32_t a, uint32_t b) {
        uint32_t d;
        if constexpr (DTYPE == LOWBIT_DTYPE_BF16) asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        else asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
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
    // Fills `held`; the thread's largest value.
    __device__ __forceinline__ float hold() {
        float top = -INFINITY;
#pragma unroll 4
        for (int it = 0; it < nvec; ++it) {
            const uint4 w = load(it);
            if (it < kHeld) held[it * kThreads] = w;
            top = fmaxf(top, largest(w));
        }
        return top;
    }
    // f(x, it, v) for each token; after a vector the whole warp comes to done(it).
    template <typename F, typename G>
    __device__ __forceinline__ void each(const F &f, const G &done) const {
#pragma unroll 1
        for (int it = 0; it < nvec; ++it) {
            const uint4 w = it < kHeld ? held[it * kThreads] : load(it);
#pragma unroll
            for (int v = 0; v < kVec; ++v) f(get(w, v), it, v);
            done(it);
        }
    }
    template <typename F>
    __device__ __forceinline__ void each(const F &f) const {
        each(f, [](int) {});
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

// The whole part of f * total for 0 <= f < 1, and whether there is a rest: in whole numbers
// (double precision is slow on this device).
struct Product { u64 whole; bool rest; };
__device__ __forceinline__ Product times(float f, u64 total) {
    const uint32_t bits = __float_as_uint(f), e = max(bits >> 23, 1u);
    const u64 m = (bits & 0x7FFFFFu) | (bits >> 23 != 0 ? 0x800000u : 0u), lo = m * total, hi = __umul64hi(m, total);
    const uint32_t shift = 150u - e;               // f = m / 2^shift, shift >= 24
    if (shift >= 128) return {0ull, (lo | hi) != 0};
    if (shift >= 64) return {hi >> (shift - 64), (lo | (hi & ((1ull << (shift - 64)) - 1))) != 0};
    return {hi << (64 - shift) | lo >> shift, (lo & ((1ull << shift) - 1)) != 0};
}
// floor(u * total), below total.
__device__ __forceinline__ u64 target_of(float u, u64 total) {
    return !(u > 0.f) ? 0ull : u >= 1.f ? total - 1 : times(u, total).whole;
}
// The mass that a prefix has to reach for top-p (below 1): ceil(p total), at least 1.
__device__ __forceinline__ u64 limit_of(float top_p, u64 total) {
    const Product p = times(top_p, total);
    return max(p.whole + p.rest, 1ull);
}

// The least v in (lo, hi] for which the entries of the list with (entry & mask) > v hold
// less than `need`, in mass or in number: hi is one, lo is not, and v is an entry (they
// differ).  512 bins of the range, one of which is the next range, until few are left.
__device__ __noinline__ u64 search(Shared &sm, int n, u64 mask, bool by_mass, u64 need, u64 lo, u64 hi) {
    const int tid = threadIdx.x, lane = tid & 31;
    uint32_t *const number = sm.coarse, *const high = sm.coarse + kThreads;      // number << 21 | low 10 bits of W; the others
    u64 above = 0;                                 // of the entries over hi
    int left = n;
    __syncthreads();
    while (left > kFew) {
        const int shift = max(55 - __clzll((long long)(hi - lo - 1)), 0);
        number[tid] = high[tid] = 0u;
        if (tid == 0) sm.found[3] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += kThreads) {
            const u64 v = sm.list[i] & mask;
            if (v <= lo || v > hi) continue;
            const uint32_t W = by_mass ? sm.weight[i] : 1u, at = kThreads - 1 - (uint32_t)((v - lo - 1) >> shift);
            atomicAdd(number + at, 1u << 21 | (W & 0x3FFu));
            if (W >> 10 != 0) atomicAdd(high + at, W >> 10);
        }
        __syncthreads();
        const uint32_t word = number[tid];
        const u64 mine = (word & 0x1FFFFFu) + ((u64)high[tid] << 10);
        u64 before = mine, z = 0, t, tz;
        block_scan(sm, before, z, t, tz);
        before += above;
        if (before < need && before + mine >= need) sm.found[3] = (u64)(word >> 21) << 32 | (uint32_t)(tid + 1), sm.found[2] = before;
        __syncthreads();
        if (sm.found[3] == 0) return hi;
        left = (int)(sm.found[3] >> 32), above = sm.found[2];
        const u64 at = (u64)(kThreads - (int)(uint32_t)sm.found[3]);
        hi = min(lo + ((at + 1) << shift), hi), lo += at << shift;
        __syncthreads();
    }
    if (tid == 0) sm.fews = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
        const u64 v = sm.list[i] & mask;
        if (v <= lo || v > hi) continue;
        const int at = atomicAdd(&sm.fews, 1) & (kFew - 1);
        sm.few[at] = v, sm.few_weight[at] = by_mass ? sm.weight[i] : 1u;
    }
    __syncthreads();
    // Every warp compares all of them with all.
    const int few = min(sm.fews, kFew);
    const u64 v = lane < few ? sm.few[lane] : 0ull;
    u64 before = above;
    for (int j = 0; j < few; ++j) accumulate(before, sm.few[j] > v ? sm.few_weight[j] : 0u);
    const uint32_t is = __ballot_sync(~0u, lane < few && before < need && before + sm.few_weight[lane] >= need);
    return is != 0 ? __shfl_sync(~0u, v, __ffs(is) - 1) : hi;
}
// Weights of the list's entries, of those at `cut` and above; their sum.
__device__ __noinline__ u64 weigh_list(Shared &sm, const Draw r, int n, u64 cut) {
    const int tid = threadIdx.x;
    u64 sum = 0, z = 0, all, tz;
    for (int i = tid; i < n; i += kThreads) {
        const u64 place = sm.list[i];
        const Token t = weigh(r, unordered((uint32_t)(place >> kIndexBits)));
        const uint32_t W = t.in && place >= cut ? t.W : 0u;
        sm.weight[i] = W;
        sum += W;
    }
    block_scan(sm, sum, z, all, tz);
    return all;
}

// The kept prefix: tokens whose key is above `key`, and of those equal to it (W each) the
// first `quota` in index order, which are those up to index `last`.
struct Cut { uint32_t key, W; u64 quota; int last; };

// The counting path.  Narrows the prefix to the tokens before which less than `target`
// tokens (by_mass: units of W) come; the present prefix reaches the target.  `mass` is that
// of the prefix (by number only), `round` the exchanges so far.
struct Narrowed { Cut cut; u64 mass; int round; };
template <int DTYPE>
__device__ __noinline__ Narrowed narrow(Shared &sm, const Row<DTYPE> row, Draw r, bool by_mass, u64 target, Cut cut) {
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
            return Narrowed{cut, 0, r.round};
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
    return Narrowed{cut, m_above + cut.quota * cut.W, r.round};
}

// What counts of a token: its weight if it is kept, or (equals) one if its key is the cut's.
struct Count {
    float from;
    int last;
    bool equals;
    __device__ __forceinline__ Count(const Cut &cut, bool equals)
        : from(cut.key == 0 ? -INFINITY : unordered(cut.key)), last(cut.last), equals(equals) {}
    __device__ __forceinline__ uint32_t of(const Draw &r, float x, int index) const {
        if (!(x >= from) || (x == from ? !equals && index > last : equals)) return 0u;
        const Token t = weigh(r, x);
        return !t.in ? 0u : equals ? 1u : t.W;
    }
};

// The sum of each run of a warp's vectors (in index order: vector number, then warp).
template <int DTYPE>
__device__ __noinline__ void tally(Shared &sm, const Row<DTYPE> row, const Draw r, const Count count) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    u64 sum = 0;
    row.each([&](float x, int it, int v) { accumulate(sum, count.of(r, x, row.index_of(it, v))); },
             [&](int it) {
                 __syncwarp();
                 sum = warp_sum(sum);
                 if (lane == 0) sm.runs[it * kWarps + warp] = sum;
                 sum = 0;
             });
}

// The token in which the running total in index order passes a target: that of the given
// uniform number, or (count.equals) of the cut's quota.  One thread of the cluster gets
// its index, the others -1; `total` is the sum.  Begins with a barrier of the CTA; counts as
// one exchange.
struct Found { int index; u64 total; };
template <int DTYPE>
__device__ __noinline__ Found locate(Shared &sm, const Row<DTYPE> row, Draw r, const Count count, u64 quota, float u) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // Two runs a thread at most.
    const int runs = row.nvec * kWarps, per = (runs + kThreads - 1) / kThreads;
    __syncthreads();
    u64 mine = 0, z = 0, of_cta, tz;
    for (int q = 0; q < per; ++q)
        if (tid * per + q < runs) mine += sm.runs[tid * per + q];
    block_scan(sm, mine, z, of_cta, tz);
    exchange(sm, r, of_cta);
    u64 total = 0;
    for (int i = 0; i < r.ranks; ++i) {
        if (i == r.rank) mine += total;
        total += sm.peer[i][0];
    }
    const u64 target = count.equals ? quota - 1 : target_of(u, total);
    if (tid == 0) sm.found[0] = 0;
    __syncthreads();
    for (int q = 0; q < per; ++q)
        if (tid * per + q < runs) {
            const u64 add = sm.runs[tid * per + q];
            if (target >= mine && target < mine + add) sm.found[0] = (u64)(tid * per + q + 1), sm.found[1] = mine;
            mine += add;
        }
    __syncthreads();
    const int at = (int)sm.found[0] - 1;
    if (at < 0 || at % kWarps != warp) return Found{-1, total};
    // The lane, then the token.
    const uint4 w = row.load(at / kWarps);
    u64 own = 0;
#pragma unroll
    for (int v = 0; v < Row<DTYPE>::kVec; ++v) own += count.of(r, Row<DTYPE>::get(w, v), row.index_of(at / kWarps, v));
    u64 sum = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 v = __shfl_up_sync(~0u, sum, o);
        if (lane >= o) sum += v;
    }
    sum += sm.found[1] - own;
    if (target < sum || target >= sum + own) return Found{-1, total};
    int index = -1;
#pragma unroll
    for (int v = 0; v < Row<DTYPE>::kVec; ++v) {
        const int i = row.index_of(at / kWarps, v);
        const u64 add = count.of(r, Row<DTYPE>::get(w, v), i);
        if (target >= sum && target < sum + add) index = i;
        sum += add;
    }
    return Found{index, total};
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
    p.logprob[b] = __fmul_rn(__fsub_rn(x, r.m), r.inv_t) - logf((float)mass * (1.f / kUnit));
}

// What a token of a warp has before it: how many of the others' places & mask are larger,
// and their mass.
struct Before { int number; u64 mass; };
__device__ __forceinline__ Before before_of(int n, u64 place, uint32_t W, u64 mask) {
    Before b{0, 0ull};
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
        const bool is = (__shfl_sync(~0u, place, j) & mask) > (place & mask);
        const uint32_t w = __shfl_sync(~0u, W, j);
        b.number += is;
        accumulate(b.mass, is ? w : 0u);
    }
    return b;
}
// draw_listed (below) for up to 32 tokens, a token a lane.
template <int DTYPE>
__device__ __noinline__ void draw_few(Shared &sm, const Row<DTYPE> row, const Draw r, int n, int top_k, float top_p, u64 total,
                                      const SampleArgs &p, int b) {
    const int lane = threadIdx.x & 31;
    if (threadIdx.x >= 32) return;
    const u64 place = lane < n ? sm.list[lane] : 0ull;
    const Token t = weigh(r, unordered((uint32_t)(place >> kIndexBits)));
    const uint32_t W = lane < n && t.in ? t.W : 0u;
    const float u = p.u[b];
    const Before of = before_of(n, place, W, ~0ull);
    bool kept = W != 0 && (top_k <= 0 || of.number < top_k);
    const u64 all = warp_sum(kept ? W : 0u);
    if (top_p < 1.f) kept = kept && of.mass < limit_of(top_p, total != 0 ? total : all);
    const u64 mass = warp_sum(kept ? W : 0u), target = target_of(u, mass);
    const Before ahead = before_of(n, place, kept ? W : 0u, kIndexMask);
    if (kept && target >= ahead.mass && target < ahead.mass + W) write_token(row, r, index_at(place), mass, p, b);
}

// The rest of the work on the list of n tokens (this CTA's alone; places in (lo, hi]):
// top-k, top-p, draw.  total: mass of all tokens within min-p (0: that of the first top_k
// of the list).
template <int DTYPE>
__device__ __noinline__ void draw_listed(Shared &sm, const Row<DTYPE> row, const Draw r, int n, u64 lo, u64 hi, int top_k, float top_p,
                                         u64 total, const SampleArgs &p, int b) {
    u64 cut = 0;
    if (top_k > 0 && top_k < n) cut = search(sm, n, ~0ull, false, (u64)top_k, lo, hi);
    u64 mass = weigh_list(sm, r, n, cut);
    if (top_p < 1.f) {
        const u64 limit = limit_of(top_p, total == 0 ? mass : total);
        if (mass >= limit) {
            cut = search(sm, n, ~0ull, true, limit, cut == 0 ? lo : cut - 1, hi);
            mass = weigh_list(sm, r, n, cut);
        }
    }
    const u64 at = search(sm, n, kIndexMask, true, target_of(p.u[b], mass) + 1, 0ull, kIndexMask);
    if (threadIdx.x == 0) write_token(row, r, index_at(at), mass, p, b);
}

// 2^15 to 2^46, a power of two by which the weights of bin `at` of the top-p bound are
// multiplied: at most 2^15 of them.  drop: 2^23 / (bins of a halving).
__device__ __forceinline__ uint32_t scale_bits(int at, int drop) { return (uint32_t)(at * drop + (142 << 23)) & 0x7F800000u; }

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
        row.all = (row.lead + p.V + kVec - 1) / kVec;
        row.part = (row.all + r.ranks - 1) / r.ranks;
        row.first = r.rank * row.part;
        row.end = min(row.first + row.part, row.all);
        row.nvec = (row.part + kThreads - 1) / kThreads;
    }
    row.held = reinterpret_cast<uint4 *>(raw + sizeof(Shared)) + tid;
    const float own = row.hold();                  // NaN left out
    r.T = p.temperature != nullptr ? p.temperature[b] : p.temperature_all;
    const float top_p = fmaxf(p.top_p != nullptr ? p.top_p[b] : p.top_p_all, 0.f);
    const float min_p = p.min_p != nullptr ? p.min_p[b] : p.min_p_all;
    const int top_k = p.top_k != nullptr ? p.top_k[b] : p.top_k_all;
    const bool greedy = !(r.T > 0.f);

    // The largest logit of the CTA and the row.
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
    int drop = 0;
    if (counted) {
        float floor_s = 0.f, above = INFINITY;     // tokens below are not binned
        if (by_p) {
            // The threads' largest tokens give a lower bound of Z.
            const Token t = weigh(r, row.infinite ? (own == INFINITY ? 0.f : -INFINITY) : own);
            u64 least = t.in ? t.W : 0, z = 0, tl, tz;
            block_scan(sm, least, z, tl, tz);
            for (int i = tid; i < kCoarse; i += kThreads) sm.coarse[i] = 0u;
            exchange(sm, r, tl);
            tl = 0;
            for (int i = 0; i < r.ranks; ++i) tl += sm.peer[i][0];
            const float share = (1.f - top_p) * (float)tl / (float)p.V * (1.f / kUnit);
            floor_s = fmaxf(share > 0.f ? logf(share) - 1e-3f : -kSpan, -kSpan);
            per = kCoarse / -floor_s;
            drop = (int)(8388608.f * 1.442695f / per);
            above = r.m + (floor_s - 1e-3f) * r.T - fabsf(r.m) * 1e-6f;
        }
        u64 mass = 0;
        uint32_t n = 0;
        row.each([&](float x, int, int) {
            const Token t = weigh(r, x);
            accumulate(mass, t.in ? t.W : 0u);
            n += t.in;
            // The bin, floor(-s per), by adding 1.5 2^23 (a conversion would take eight times as
            // long); the weight at the bin's scale, by adding 2^23.
            const int at = (int)min(__float_as_uint(__fadd_rn(fmaf(-t.s, per, -0.5f), 12582912.f)) - 0x4B400000u, (uint32_t)kCoarse - 1u);
            const uint32_t add = __float_as_uint(fmaf(t.w, __uint_as_float(scale_bits(at, drop)), 8388608.f)) - 0x4B000000u;
            if (t.in && x >= above) atomicAdd(&sm.coarse[at], add);
        });
        u64 nn = n, tm, tn;
        block_scan(sm, mass, nn, tm, tn);
        exchange(sm, r, tm, tn);
        for (int i = 0; i < r.ranks; ++i) total += sm.peer[i][0], tokens += sm.peer[i][1];
    }
    const bool cut_k = top_k > 0 && (by_k || (u64)top_k < tokens);
    Cut cut{0u, 1u, 0, INT32_MAX};
    bool tallied = false;                          // the runs' sums are there
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
            u64 of_bin[kCoarse / kThreads], sum = 0, z = 0, tm, tz;
#pragma unroll
            for (int q = 0; q < kCoarse / kThreads; ++q) {
                const int at = tid * (kCoarse / kThreads) + q;
                of_bin[q] = 0;
                for (int i = 0; i < r.ranks; ++i)
                    of_bin[q] += ld_cluster_u32(ptx::mapa_shared(ptx::smem_u32(&sm.coarse[at]), i));
                of_bin[q] = of_bin[q] << 30 >> ((scale_bits(at, drop) >> 23) - 127);
                sum += of_bin[q];
            }
            if (tid == 0) sm.found[0] = sm.found[1] = kCoarse;
            block_scan(sm, sum, z, tm, tz);
            // The bins in which the limit may lie for what rounding may have moved it: one and the
            // same for all but one row in some hundreds, which took the counting path otherwise.
            const u64 from = limit - (limit >> 15), to = max(min(limit + (limit >> 15), tm), limit);
#pragma unroll
            for (int q = 0; q < kCoarse / kThreads; ++q) {
                const u64 upto = sum + of_bin[q];
                if (sum < from && upto >= from) sm.found[0] = (u64)(tid * (kCoarse / kThreads) + q);
                if (sum < to && upto >= to) sm.found[1] = (u64)(tid * (kCoarse / kThreads) + q);
                sum = upto;
            }
            __syncthreads();
            last = (int)sm.found[1];
            bound = fmaxf(bound, r.m - ((float)(last + 1) / per + 1e-3f) * r.T - fabsf(r.m) * 1e-6f);
            over = r.m - ((float)(int)sm.found[0] / per - 1e-3f) * r.T + fabsf(r.m) * 1e-6f;      // above: an earlier bin
        }
        if (listing) {
            // How many tokens there are from the bound on, and between it and `over`; the mass
            // above `over` of each run, of the CTA, and that between.
            uint32_t n_mine = 0, n_between = 0;
            u64 run = 0, above = 0, between = 0;
            if (last < 0) {
                row.each([&](float x, int, int) { n_mine += x >= bound; });
            } else {
                row.each(
                    [&](float x, int, int) {
                        if (x >= bound) {
                            ++n_mine;
                            const Token t = weigh(r, x);
                            const uint32_t W = t.in ? t.W : 0u;
                            accumulate(run, x > over ? W : 0u);
                            accumulate(between, x > over ? 0u : W);
                            n_between += t.in && !(x > over);
                        }
                    },
                    [&](int it) {
                        __syncwarp();
                        if (__any_sync(~0u, run != 0)) run = warp_sum(run);
                        if (lane == 0) sm.runs[it * kWarps + warp] = run, above += run;
                        run = 0;
                    });
            }
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
            const bool there = last >= 0 && before < limit && before + of_bin >= limit;
            const bool whole = n < (u64)kList && (last < 0 || there);
            const bool bin_only = !whole && there && n_bin < (u64)kList;
            if (whole || bin_only) {
                // They go to the first CTA's list, each CTA and thread at its place.
                uint32_t at = ptx::mapa_shared(ptx::smem_u32(sm.list), 0u) + (uint32_t)(whole ? mine : mine_between) * 8u;
                if ((whole ? n_mine : n_between) > 0)
                    row.each([&](float x, int it, int v) {
                        if (x >= bound && (whole || (!(x > over) && weigh(r, x).in))) {
                            st_cluster_u64(at, place_of(x, row.index_of(it, v)));
                            at += 8;
                        }
                    });
                cluster_barrier(r);
            }
            const u64 lo = place_of(bound, 0) - kIndexMask - 1, hi = place_of(whole ? r.m : fminf(over, r.m), 0);
            if (whole) {
                if (r.rank != 0) return;
                if (n <= 32) draw_few(sm, row, r, (int)n, cut_k ? top_k : 0, top_p, counted ? total : 0, p, b);
                else draw_listed(sm, row, r, (int)n, lo, hi, cut_k ? top_k : 0, top_p, counted ? total : 0, p, b);
                return;                            // nobody reads another's shared memory any more
            }
            if (bin_only) {
                u64 place = 0;
                if (r.rank == 0) {
                    weigh_list(sm, r, (int)n_bin, 0ull);
                    place = search(sm, (int)n_bin, ~0ull, true, limit - before, lo, hi);
                    // The kept ones join the runs that they are of.
                    for (int i = tid; i < (int)n_bin; i += kThreads) {
                        if (sm.list[i] < place) continue;
                        const int vec = (index_at(sm.list[i]) + row.lead) / kVec, of = vec / row.part;
                        add_cluster_u64(ptx::mapa_shared(ptx::smem_u32(&sm.runs[(vec - of * row.part) / 32]), (uint32_t)of), sm.weight[i]);
                    }
                }
                exchange(sm, r, place);
                place = sm.peer[0][0];
                cut.key = (uint32_t)(place >> kIndexBits), cut.last = index_at(place);
                tallied = true;
            }
        }
        if (!tallied) {
            // The counting path.
            if (!counted) {
                u64 mass = 0;
                uint32_t n = 0;
                row.each([&](float x, int, int) {
                    const Token t = weigh(r, x);
                    if (t.in) accumulate(mass, t.W), ++n;
                });
                u64 nn = n, tm, tn;
                block_scan(sm, mass, nn, tm, tn);
                exchange(sm, r, tm, tn);
                total = tokens = 0;
                for (int i = 0; i < r.ranks; ++i) total += sm.peer[i][0], tokens += sm.peer[i][1];
            }
            if (top_k > 0 && (u64)top_k < tokens) {
                const Narrowed to = narrow(sm, row, r, false, (u64)top_k, cut);
                cut = to.cut, total = to.mass, r.round = to.round;
            }
            if (by_p) {
                const Narrowed to = narrow(sm, row, r, true, limit_of(top_p, total), cut);
                cut = to.cut, r.round = to.round;
            }
        }
    }
    if (!tallied) {
        if (cut.key != 0) {                        // the last kept token of the cut's key
            const Count equals(cut, true);
            if (tid == 0) sm.found[2] = 0;
            tally(sm, row, r, equals);
            const Found last = locate(sm, row, r, equals, cut.quota, 0.f);
            ++r.round;
            if (last.index >= 0) sm.found[2] = (u64)last.index + 1;
            __syncthreads();
            exchange(sm, r, sm.found[2]);
            for (int i = 0; i < r.ranks; ++i)
                if (sm.peer[i][0] != 0) cut.last = (int)sm.peer[i][0] - 1;
        }
        tally(sm, row, r, Count(cut, false));
    }
    const Found drawn = locate(sm, row, r, Count(cut, false), 0, p.u[b]);
    if (drawn.index >= 0) write_token(row, r, drawn.index, drawn.total, p, b);
    cluster_barrier(r);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &args, cudaStream_t stream) {
    // CTAs of a row: as many as its tokens need, then more while each has over kShare bytes,
    // and for small batches while there are SMs for them and over kSmallShare bytes each.
    // (A step over the cluster costs the same for any share, and rows differ in their work,
    // so that some more CTAs than there is room for even out: 256 rows of 128256 floats take
    // 178 us with one CTA each, 137 with two, 136 with four and 164 with eight; 192 rows of
    // 19439 floats 18.3 us with one and 23.4 with two; 64 rows of 128256 bfloat16 53 us with
    // four and 77 with eight.)
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
