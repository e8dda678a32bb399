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
// passes floor(u Z'), Z' the kept total.  T <= 0: the first largest logit.
//
// The prefix is found without sorting.  Level 1 counts tokens (and sums W) in
// 2048 bins of s; the bin in which the k-th token or the p-th mass falls is then
// split by the bits of x, over the range that it really holds, until one value
// is left: the threshold.  Equal logits are taken in index order up to a quota.
// Tokens with W_i = 0 (s < -21.5) can never be drawn and are left out, which
// bounds the bins.
//
// Work split: a cluster of up to 8 CTAs takes a row, each keeps its part of the
// logits in shared memory (read from HBM once), and counts are exchanged through
// distributed shared memory.  Bound: the chain of cluster-wide steps for few
// rows, HBM and the shared-memory atomics for many.
#include "common.cuh"
#include "ptx.cuh"

namespace lowbit {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kHeld = 32768;                       // logits a CTA keeps; more are read again
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

// A logit as fp32; NaN counts as -infinity, -0 as 0.
__device__ __forceinline__ float clean(float x) { return x != x ? -INFINITY : x + 0.0f; }

__device__ __forceinline__ float load_logit(const void *row, int dtype, int64_t i) {
    if (dtype == LOWBIT_DTYPE_F32) return clean(static_cast<const float *>(row)[i]);
    const uint16_t h = static_cast<const uint16_t *>(row)[i];
    return clean(dtype == LOWBIT_DTYPE_BF16 ? __uint_as_float((uint32_t)h << 16) : half_bits_to_float(h));
}

// Order-preserving map of floats to unsigned integers.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

struct Shared {
    float x[kHeld];
    uint32_t count[kBins], lo[kBins], hi[kBins];   // W = lo + 2^16 hi, summed apart in 32 bits
    u64 pub[2][3];                                 // what this CTA tells the others, in two buffers
    u64 peer[kMaxCluster][3];                      // what each CTA told
    u64 red[kWarps][2];
    u64 found[3];
    uint32_t kmin, kmax;
};

// A row's part in this CTA.
struct Part {
    const void *logits;
    int dtype, n;                                  // its tokens
    int64_t first;                                 // index of the first
    float m, inv_t, min_p;
    int rank, ranks, round;                        // in the cluster; exchanges so far
};

struct Token { float s; uint32_t W; bool in; };

__device__ __forceinline__ float value(const Shared &sm, const Part &r, int i) {
    return i < kHeld ? sm.x[i] : load_logit(r.logits, r.dtype, r.first + i);
}
__device__ __forceinline__ Token weigh(const Part &r, float x) {
    Token t;
    t.s = x == r.m ? 0.f : __fmul_rn(__fsub_rn(x, r.m), r.inv_t);
    const float w = expf(t.s);
    t.W = __float2uint_rn(__fmul_rn(w, kUnit));
    t.in = t.W > 0u && !(w < r.min_p);
    return t;
}
__device__ __forceinline__ int bin_of(float s) { return min((int)(-s * (kBins / kSpan)), kBins - 1); }

// Cluster-wide exchange: sm.peer[rank] holds every CTA's words (given by its thread
// 0), for all threads.  A CTA overwrites a buffer only after the next exchange's
// barrier, which every reader of it has passed.
__device__ __forceinline__ void exchange(Shared &sm, Part &r, u64 a, u64 b = 0, u64 c = 0) {
    u64 *pub = sm.pub[r.round & 1];
    if (threadIdx.x == 0) pub[0] = a, pub[1] = b, pub[2] = c;
    ptx::cluster_sync();
    if ((int)threadIdx.x < 3 * r.ranks) {
        const uint32_t rank = threadIdx.x / 3, w = threadIdx.x % 3;
        sm.peer[rank][w] = ld_cluster_u64(ptx::mapa_shared(ptx::smem_u32(pub + w), rank));
    }
    __syncthreads();
    ++r.round;
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
    for (int i = 0; i < kWarps; ++i) {
        if (i < warp) a += sm.red[i][0], b += sm.red[i][1];
        ta += sm.red[i][0], tb += sm.red[i][1];
    }
}

// The kept prefix: tokens whose key is above `key`, and of those equal to it the
// first `quota` in index order (W each).
struct Cut { uint32_t key, W; u64 quota; };

// Narrows the prefix to the tokens before which less than `target` tokens (by_mass:
// units of W) come; the present prefix reaches the target.
__device__ void narrow(Shared &sm, Part &r, bool by_mass, u64 target, Cut &cut) {
    const int tid = threadIdx.x, lane = tid & 31;
    const int slice = kBins / r.ranks, per = max(slice / kThreads, 1);    // bins of a CTA, of a thread
    u64 n_above = 0, m_above = 0;                  // tokens and mass above the range under search
    uint32_t klo = 0u, khi = ~0u;                  // its keys
    int bin = 0, shift = 0;
    for (int level = 0;; ++level) {
        // Of the tokens above the present cut's key, those in the range.
        auto inside = [&](uint32_t k, const Token &t) {
            if (!t.in || k <= cut.key) return false;
            return level == 0 || (level == 1 ? bin_of(t.s) == bin : (k >= klo && k <= khi));
        };
        if (level > 0) {
            // The keys that the range really holds; one: that is the threshold.
            if (tid == 0) sm.kmin = ~0u, sm.kmax = 0u;
            __syncthreads();
            uint32_t lo = ~0u, hi = 0u;
            for (int i = tid; i < r.n; i += kThreads) {
                const float x = value(sm, r, i);
                const uint32_t k = ordered(x);
                if (inside(k, weigh(r, x))) lo = min(lo, k), hi = max(hi, k);
            }
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
        for (int i = tid; i < r.n; i += kThreads) {
            const float x = value(sm, r, i);
            const uint32_t k = ordered(x);
            const Token t = weigh(r, x);
            if (!inside(k, t)) continue;
            const int at = level == 0 ? bin_of(t.s) : (int)((khi - k) >> shift);
            atomicAdd(&sm.count[at], 1u);
            atomicAdd(&sm.lo[at], t.W & 0xFFFFu);
            atomicAdd(&sm.hi[at], t.W >> 16);
        }
        ptx::cluster_sync();
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
                             ((u64)ld_cluster_u32(ptx::mapa_shared(ptx::smem_u32(&sm.hi[at]), i)) << 16);
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
    cut.W = weigh(r, __uint_as_float(khi & 0x80000000u ? khi ^ 0x80000000u : ~khi)).W;
    cut.quota = by_mass ? (target - m_above + cut.W - 1) / cut.W : target - n_above;
}

__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleArgs p) {
    extern __shared__ __align__(16) uint8_t raw[];
    Shared &sm = *reinterpret_cast<Shared *>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();

    Part r;
    uint32_t ranks;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ranks));
    r.ranks = (int)ranks, r.rank = (int)ptx::cluster_ctarank(), r.round = 0;
    const int b = (int)(blockIdx.x / ranks);
    const int part = (p.V + r.ranks - 1) / r.ranks;
    r.first = (int64_t)r.rank * part;
    r.n = (int)max((int64_t)0, min((int64_t)part, p.V - r.first));
    r.dtype = p.dtype;
    r.logits = static_cast<const uint8_t *>(p.logits) + b * p.row_stride * (p.dtype == LOWBIT_DTYPE_F32 ? 4 : 2);
    const float T = p.temperature != nullptr ? p.temperature[b] : p.temperature_all;
    const float top_p = p.top_p != nullptr ? p.top_p[b] : p.top_p_all;
    const float min_p = p.min_p != nullptr ? p.min_p[b] : p.min_p_all;
    const int top_k = p.top_k != nullptr ? p.top_k[b] : p.top_k_all;

    // The row's part into shared memory; its largest logit, lowest index first.
    u64 best = 0;
    for (int i = tid; i < r.n; i += kThreads) {
        const float x = load_logit(r.logits, r.dtype, r.first + i);
        if (i < kHeld) sm.x[i] = x;
        const u64 v = (u64)ordered(x) << 32 | (uint32_t)~(uint32_t)(r.first + i);
        best = v > best ? v : best;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const u64 v = __shfl_xor_sync(~0u, best, o);
        best = v > best ? v : best;
    }
    if (lane == 0) sm.red[warp][0] = best;
    __syncthreads();
    for (int i = 0; i < kWarps; ++i) best = sm.red[i][0] > best ? sm.red[i][0] : best;
    exchange(sm, r, best);
    for (int i = 0; i < r.ranks; ++i) best = sm.peer[i][0] > best ? sm.peer[i][0] : best;
    const uint32_t top = (uint32_t)(best >> 32);
    r.m = __uint_as_float(top & 0x80000000u ? top ^ 0x80000000u : ~top);
    const bool empty = r.m == -INFINITY;           // nothing can be drawn
    if (empty || !(T > 0.f)) {
        if (r.rank == 0 && tid == 0) {
            p.token[b] = empty ? -1 : (int64_t)(uint32_t)~(uint32_t)best;
            if (p.logprob != nullptr) p.logprob[b] = empty ? -INFINITY : 0.f;
        }
        ptx::cluster_sync();                       // others may still read this CTA's words
        return;
    }
    r.inv_t = __fdiv_rn(1.f, T);
    r.min_p = fminf(min_p, 1.f);                   // the largest logit is always kept

    // Tokens within min-p that can be drawn at all, and their mass.
    Cut cut{0u, 1u, 0};
    u64 n = 0, mass = 0, tn, tm;
    for (int i = tid; i < r.n; i += kThreads) {
        const Token t = weigh(r, value(sm, r, i));
        if (t.in) ++n, mass += t.W;
    }
    block_scan(sm, n, mass, tn, tm);
    exchange(sm, r, tn, tm);
    n = mass = 0;
    for (int i = 0; i < r.ranks; ++i) n += sm.peer[i][0], mass += sm.peer[i][1];

    const int seg = (r.n + 32 * kWarps - 1) / (32 * kWarps) * 32;        // a warp's tokens, in index order
    const int s0 = min(warp * seg, r.n), s1 = min(s0 + seg, r.n);
    // Mass above the cut and tokens equal to it: this thread's CTA, warp by warp, in sm.red.
    auto tally = [&] {
        u64 above = 0, equal = 0;
        for (int i = s0 + lane; i < s1; i += 32) {
            const float x = value(sm, r, i);
            const uint32_t k = ordered(x);
            if (k < cut.key) continue;
            const Token t = weigh(r, x);
            if (t.in) {
                if (k > cut.key) above += t.W;
                else ++equal;
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            above += __shfl_xor_sync(~0u, above, o);
            equal += __shfl_xor_sync(~0u, equal, o);
        }
        __syncthreads();
        if (lane == 0) sm.red[warp][0] = above, sm.red[warp][1] = equal;
        __syncthreads();
        above = equal = 0;
        for (int i = 0; i < kWarps; ++i) above += sm.red[i][0], equal += sm.red[i][1];
        exchange(sm, r, above, equal);
    };
    if (top_k > 0 && (u64)top_k < n) {
        narrow(sm, r, false, (u64)top_k, cut);
        tally();
        mass = cut.quota * cut.W;
        for (int i = 0; i < r.ranks; ++i) mass += sm.peer[i][0];
    }
    if (top_p < 1.f) {
        const double want = ceil((double)top_p * (double)mass);
        narrow(sm, r, true, want > 1.0 ? (u64)want : 1ull, cut);
    }
    tally();

    // The draw: CTA, warp and token in which the target falls.
    u64 total = 0, start = 0, equal = 0, mine = 0;                       // start, equal: before this CTA
    for (int i = 0, eq = 0; i < r.ranks; ++i) {
        const u64 e = sm.peer[i][1], left = cut.quota > (u64)eq ? cut.quota - eq : 0;
        const u64 kept = sm.peer[i][0] + (e < left ? e : left) * cut.W;
        if (i == r.rank) start = total, equal = eq, mine = kept;
        total += kept;
        eq += (int)e;
    }
    const float u = p.u[b];
    u64 target = u > 0.f ? (u64)floor((double)u * (double)total) : 0ull;
    target = target < total ? target : total - 1;
    if (target >= start && target < start + mine) {
        for (int i = 0; i < kWarps; ++i) {
            const u64 e = sm.red[i][1], left = cut.quota > equal ? cut.quota - equal : 0;
            const u64 kept = sm.red[i][0] + (e < left ? e : left) * cut.W;
            if (target < start + kept) {
                if (i == warp) {
                    for (int base = s0; base < s1; base += 32) {
                        const int at = base + lane;
                        const float x = at < s1 ? value(sm, r, at) : -INFINITY;
                        const uint32_t k = ordered(x);
                        const Token t = weigh(r, x);
                        const bool tie = t.in && k == cut.key;
                        const unsigned ties = __ballot_sync(~0u, tie);
                        const bool kept_tie = tie && equal + __popc(ties & ((1u << lane) - 1u)) < cut.quota;
                        u64 inc = (t.in && k > cut.key) || kept_tie ? t.W : 0;
#pragma unroll
                        for (int o = 1; o < 32; o <<= 1) {
                            const u64 v = __shfl_up_sync(~0u, inc, o);
                            if (lane >= o) inc += v;
                        }
                        const unsigned past = __ballot_sync(~0u, start + inc > target);
                        if (past) {
                            if (lane == __ffs(past) - 1) {
                                p.token[b] = r.first + at;
                                if (p.logprob != nullptr)
                                    p.logprob[b] = t.s - logf((float)total * (1.f / kUnit));
                            }
                            break;
                        }
                        start += __shfl_sync(~0u, inc, 31);
                        equal += __popc(ties);
                    }
                }
                break;
            }
            start += kept;
            equal += e;
        }
    }
    ptx::cluster_sync();
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &args, cudaStream_t stream) {
    int ranks = 1;
    while (ranks < kMaxCluster && (args.V > ranks * 4096) && (args.V > ranks * kHeld || args.B * ranks * 2 <= 152)) ranks *= 2;
    const int smem = (int)sizeof(Shared);
    const cudaError_t e = raise_smem_limit((const void *)sample_kernel, current_device(), smem);
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
    return cudaLaunchKernelEx(&cfg, sample_kernel, args);
}

}  // namespace lowbit
