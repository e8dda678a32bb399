// attention_prompt.cu -- attention over a paged cache of 8 or 4 bits for many new tokens
// (prompts), on the tcgen05 tensor cores with accumulators in tensor memory.
//
// Mathematics: as attention.cu (codes multiplied as fp16 numbers, page exponents
// applied in fp32, V's exponent inside the softmax exponent).  As m may lag behind the
// maximum (attention.cuh), the rescaling of O, a round trip through tensor memory, is rare.
// A 4-bit cache's codes are turned into their values / 64, exact in fp16 (attention4.cu), so that
// there are no exponents then; 64 is in the row's factor of the scores and in the last division.
//
// Work split.  A CTA takes 256 rows (new tokens x heads of a group) of one sequence
// and kv head, as two 128-row tiles whose softmax and products alternate: while one
// tile's weights are computed, the other's products run.  Keys come 128 at a time.
// Where CTAs are few or some sequences far longer than others, the keys of the tiles are
// split between several, and a second launch joins their parts (find_listed, prompt_grid).
// Tiles with the most keys start first.
//
// Tensor memory (512 columns): S of both tiles (128 fp32 columns each, as two halves of
// 64 keys; the fp16 weights P take the place of the half they come from), O of both.
// The halves are two buffers: while one is weighed, the other's products run, so that
// four chains (two tiles, two halves) keep the tensor cores fed.
// Warps: 0-3 and 4-7 softmax of tile 0 and 1 (one thread a row, which holds the
// row's 128 scores in registers: 184 a thread, taken from the other warps), 8-11 turn
// e4m3 codes into fp16 operand tiles (once per 256 rows), 12 TMA producer, 13 and 14 MMA
// issuers, one for each tile, so that neither waits for the other's weights.  Order of an
// issuer, half-step by half-step: PV(h) QK(h + 2), products of one issuer running in order.
// Bound: shared memory, nearly.  256 rows x 128 keys at D = 128 take the tensor cores 2048
// cycles, the exponentials as many, and shared memory about 3070: 1536 for the operands of
// QK (q is read again for every half; both halves in one product read it once, 2560 in all,
// but leave the weights waiting: 152 us against 132), 512 for V, 1024 to bring in, turn and
// store the codes.  A step takes 3100; a CTA beside its steps about 15000 (its queries and
// first keys 8000, its last product and result 6000).  4096 tokens, 32 heads of 128 over 8:
// 126 us, 1.1 PFLOP/s (0.57 of the rate of a library product); over 4 bits 124.  (What keeps scores past 2^22 right costs
// 0.8 and 1.5 us of them: code that does not run, but stands between the maximum and the weights.  In a loop of its own, or as
// weights of its own, it cost 2 to 6.)
#include <algorithm>

#include "attention.cuh"
#include "int4.cuh"

namespace lowbit {
namespace {

using namespace attn;

constexpr int kKeys = 128;                       // keys of a step
constexpr int kHalf = 64;                        // keys of a half-step
constexpr int kRows = 256;                       // rows of a CTA
constexpr int kUnit = 64;                        // keys of a raw TMA unit
constexpr int kRaw = 4;                          // raw units in flight
constexpr int kBuf = 2;                          // fp16 K and V tiles
constexpr int kExps = 8;                         // steps whose page exponents are kept
constexpr int kSoftmaxWarps = 8, kConvertWarps = 4;
constexpr int kProducer = 12, kIssuer = 13;      // and 14
constexpr int kThreads = 16 * 32;              // whole warpgroups, for the register split
constexpr int kSoftmaxRegs = 184, kConvertRegs = 80, kOtherRegs = 64;   // 2 x 184 + 80 + 64 = 4 x 128
constexpr int kMinSteps = 2;                     // of a part
constexpr int kShortSteps = 8;                   // of sequences whose tiles are never split
constexpr float kCtaCost = 5.f;                  // what a CTA costs beside its steps, in steps (2, 10: nothing changes)
constexpr float kJoinCost = 0.03f;               // what a part costs when it is joined (0.01: the same; 0.1: chunks 117 -> 140 us)
constexpr int kMostCtas = 5 * kSms;              // where keys may be split
constexpr int kLongSteps = 32;                   // of sequences whose tiles are split although they fill the SMs

__device__ unsigned int g_prompt_timeouts;

template <int D, bool FOUR>
struct Smem {
    // A raw unit: codes, then a 4-bit cache's scales.
    static constexpr int kQ = 128 * D * 2, kTile = kKeys * D * 2, kRawCodes = kUnit * D / (FOUR ? 2 : 1);
    static constexpr int kRawBytes = kRawCodes + (FOUR ? kUnit / 16 * 128 : 0);
    // A copy's place in shared memory is a multiple of 128 bytes: so far apart are the scales of pages in a unit.
    static __device__ __forceinline__ int slot(int box) { return max(box * (D / kGroup4), 128); }
    alignas(1024) uint8_t q[2][kQ];
    alignas(1024) uint8_t k[kBuf][kTile];
    alignas(1024) uint8_t v[kBuf][kTile];
    alignas(1024) uint8_t raw[kRaw][kRawBytes];
    float4 exps[kExps][kKeys / 16];              // (8 bits) of each 16 keys: 2^ke, ve, 2^-ve (0 below kDeep), whether one of the 64 is below
    uint64_t raw_full[kRaw], raw_empty[kRaw], k_full[kBuf], v_full[kBuf], kv_empty[kBuf];
    uint64_t s_full[2][2], p_full[2][2], o_full, e_full[kExps];
    uint32_t tmem;
    int poisoned;
};

// MN-major operand (the 64 contiguous values of an atom run along N): 128-byte
// swizzle atoms of 8 k-rows, 1024 bytes from one to the next along K, `lead` bytes
// to the next 64 values along N.
__device__ __forceinline__ uint64_t sw128_mn_desc(uint32_t smem_addr, uint32_t lead) {
    return (uint64_t)((smem_addr & 0x3FFFFu) >> 4) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(1024u >> 4) << 32) |
           ((uint64_t)1u << 46) | ((uint64_t)2u << 61);
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,"
        "%30,%31}, [%32];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
          "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
          "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
        : "r"(taddr));
}

// The MMA issuer runs as a whole warp and elects the issuing lane in each instruction:
// with the control flow uniform, descriptors stay in uniform registers.  Issued from a
// lane-0 branch instead, each product took 90 cycles to issue and the tensor cores
// waited.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|q, 0xFFFFFFFF;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|q, 0xFFFFFFFF;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xFFFFFFFF;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
        ::"r"(bar) : "memory");
}
// 8 bytes from global to shared memory, zeros beyond `bytes`.
__device__ __forceinline__ void cp_async8(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint4 lds_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
template <int N>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// The CTA's part of the work.
struct Work {
    int b, h, row0, nrows, start, first, len;    // rows row0 .. of nrows; first: position of the first new token
    int lo, n;                                   // first step of 128 keys, and how many
    int part, parts, slot;                       // this part of how many of the row tile's keys; the first one's place
    int steps;                                   // of all parts together
    bool live;
    // The first step of a part: at most 2^24 steps, and no more parts than SMs.
    __device__ int first_of(int i) const { return (int)((uint32_t)steps * (uint32_t)i / (uint32_t)parts); }
};

// The steps of row tile t of a sequence: how many, and the first.
__device__ __forceinline__ int steps_of(const AttentionArgs &p, const Span &s, int t, int &lo) {
    const int first = s.len - s.n, pos_lo = first + t * kRows / p.G, pos_hi = first + (min((t + 1) * kRows, s.n * p.G) - 1) / p.G;
    lo = p.window > 0 ? max(pos_lo - p.window + 1, 0) / kKeys : 0;
    return pos_hi >= 0 ? pos_hi / kKeys + 1 - lo : 0;
}

// Where the keys may be split, the parts of all sequences' tiles form one list.  With
// `all` the steps of all tiles and `most` those of the longest, there are u = all / most
// tiles' worth of work; cut into q parts each, it goes through the SMs in ceil(u q / SMs)
// rounds of most / q steps and what a CTA costs beside them.  The best of 1 and the q
// that fill one to four rounds gives the length of a part; sequences with fewer keys have fewer.
// Finds the index'th part (or tile, if not by_part) of the list.  (Rounded operations
// throughout: the join has to come to the same parts.)
struct Listed { int b, tiles, parts, rest, before; };       // rest: index in the sequence; before: parts of earlier ones
__device__ __forceinline__ Listed find_listed(const AttentionArgs &p, const PromptGrid &g, int index, bool by_part) {
    const int lane = threadIdx.x & 31;
    auto tiles_of = [&](const Span &s) { return s.n * p.G > p.few_rows ? (s.n * p.G + kRows - 1) / kRows : 0; };
    float all = 0.f;
    int most = 1, tiles = 0, steps = 0;
    for (int b = lane; b < p.B; b += 32) {
        const Span s = span(p, b);
        int lo;
        tiles = tiles_of(s), steps = tiles > 0 ? steps_of(p, s, tiles - 1, lo) : 0;
        if (tiles > 0) all = __fadd_rn(all, __fmul_rn((float)tiles * 0.5f, (float)(steps_of(p, s, 0, lo) + steps)));
        most = max(most, steps);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all = __fadd_rn(all, __shfl_xor_sync(~0u, all, o));
    most = __reduce_max_sync(~0u, most);
    const float u = fmaxf(__fdiv_rn(__fmul_rn(all, (float)p.Hk), (float)most), 1e-3f);
    float least = INFINITY;
    int length = most;
#pragma unroll
    for (int r = 0; r <= 4; ++r) {                                    // 0: whole tiles
        const float q = floorf(fminf(fmaxf(__fdiv_rn((float)(kSms * r), u), 1.f), (float)g.splits));
        const float rounds = fmaxf(ceilf(__fadd_rn(__fmul_rn(__fmul_rn(u, q), 1.f / kSms), -0.01f)), 1.f);
        const float each = ceilf(__fdiv_rn((float)most, q));
        float cost = __fmul_rn(rounds, __fadd_rn(each, kCtaCost));
        if (q > 1.f) cost = __fadd_rn(cost, __fmul_rn(__fmul_rn(u, q), kJoinCost));
        if (cost < least) least = cost, length = (int)each;
    }
    length = max(length, kMinSteps);
    Listed at{0, 0, 1, -1, 0};
    for (int b0 = 0; b0 < p.B && at.rest < 0; b0 += 32) {
        if (p.B > 32) {
            tiles = steps = 0;
            if (b0 + lane < p.B) {
                const Span s = span(p, b0 + lane);
                int lo;
                tiles = tiles_of(s), steps = tiles > 0 ? steps_of(p, s, tiles - 1, lo) : 0;
            }
        }
        const int parts = max(min((steps + length - 1) / length, g.splits), 1), count = tiles * p.Hk;
        int listed = count * parts, found = by_part ? listed : count;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int l = __shfl_up_sync(~0u, listed, o), f = __shfl_up_sync(~0u, found, o);
            if (lane >= o) listed += l, found += f;
        }
        const uint32_t hit = __ballot_sync(~0u, index < found);
        if (hit != 0) {
            const int l = __ffs(hit) - 1;
            at.b = b0 + l;
            at.tiles = __shfl_sync(~0u, tiles, l), at.parts = __shfl_sync(~0u, parts, l);
            at.rest = index - __shfl_sync(~0u, found - (by_part ? count * parts : count), l);
            at.before += __shfl_sync(~0u, listed - count * parts, l);
        } else {
            index -= __shfl_sync(~0u, found, 31);
            at.before += __shfl_sync(~0u, listed, 31);
        }
    }
    // From lane 0, so that the work is uniform for the compiler too.
    at.b = __shfl_sync(~0u, at.b, 0), at.tiles = __shfl_sync(~0u, at.tiles, 0), at.parts = __shfl_sync(~0u, at.parts, 0);
    at.rest = __shfl_sync(~0u, at.rest, 0), at.before = __shfl_sync(~0u, at.before, 0);
    return at;
}

// The work of a CTA, or (not by_part) of the tile-th tile for the join.
__device__ __forceinline__ Work work_of(const AttentionArgs &p, const PromptGrid &g, int id, bool by_part) {
    Work w{};
    const int G = p.G;
    int b, t;
    w.parts = 1;
    if (g.splits > 1) {
        const Listed at = find_listed(p, g, id, by_part);
        if (at.rest < 0) return w;
        const int tile = by_part ? at.rest / at.parts : at.rest;
        w.part = by_part ? at.rest - tile * at.parts : 0;
        w.parts = at.parts, w.slot = at.before + tile * at.parts;
        b = at.b, t = at.tiles - 1 - tile / p.Hk, w.h = tile % p.Hk;
    } else {
        // Ids count down over the row tiles, so that tiles with the most keys start first.
        w.h = id % p.Hk;
        const int tile = g.tiles - 1 - id / p.Hk;
        if (p.cu_q == nullptr) {
            const int per = g.tiles / p.B;
            b = tile % p.B, t = tile / p.B;
            if (t >= per) return w;
        } else {
            // Sequence b owns the tiles from cu_q[b] G / 256 + b on: enough for its rows.
            auto base = [&](int i) { return (int)((int64_t)min(max(p.cu_q[i], 0), p.T) * G / kRows) + i; };
            int lo = 0, hi = p.B - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (base(mid) <= tile) lo = mid;
                else hi = mid - 1;
            }
            b = lo, t = tile - base(lo);
        }
    }
    const Span s = span(p, b);
    w.b = b, w.start = s.start, w.len = s.len, w.first = s.len - s.n;
    w.nrows = s.n * G, w.row0 = t * kRows;
    w.live = t >= 0 && w.row0 < w.nrows && w.nrows > p.few_rows;
    if (!w.live) return w;
    int lo;
    const uint32_t n = (uint32_t)steps_of(p, s, t, lo);
    w.steps = (int)n;
    w.lo = lo, w.n = (int)n;
    if (w.parts > 1) w.lo += w.first_of(w.part), w.n = w.first_of(w.part + 1) - w.first_of(w.part);
    return w;
}

// Workspace of a part: D / 4 groups of four sums of each of the 256 rows, then
// the rows' (m, l) pairs.
template <int D>
__device__ __forceinline__ float *part_of(const AttentionArgs &p, const PromptGrid &g, int slot) {
    return p.workspace + g.workspace + (int64_t)slot * (kRows * (D + 2));
}

struct Maps { CUtensorMap k, v, k_scale, v_scale; };      // the scales' of a 4-bit cache only

// A word of eight 4-bit codes as eight values / 64: in the order 0, 4, 1, 5, 2, 6, 3, 7 (attention4.cu).
__device__ __forceinline__ uint4 turn4(uint32_t w, __half2 s, __half2 t) {
    auto values = [&](uint32_t in) {
        const uint32_t one = ptx::lop3_and_or(in, 0x00F000F0u, 0x3C003C00u);
        const __half2 y = __hfma2(*reinterpret_cast<const __half2 *>(&one), s, t);
        return *reinterpret_cast<const uint32_t *>(&y);
    };
    return make_uint4(values(w << 4), values(w), values(w >> 4), values(w >> 8));
}

template <int D, bool FOUR>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ Maps maps, const AttentionArgs p, const PromptGrid grid) {
    constexpr float kValueUnit = FOUR ? 64.f : 1.f;            // what a cached value counts in the products
    extern __shared__ uint8_t raw_smem[];
    Smem<D, FOUR> &sm = *reinterpret_cast<Smem<D, FOUR> *>(raw_smem + ((1024 - (ptx::smem_u32(raw_smem) & 1023)) & 1023));
    const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;      // the warp number, uniform
    auto at = [](const uint64_t &bar) { return ptx::smem_u32(&bar); };
    if (tid == 0) {
        for (int i = 0; i < kRaw; ++i) ptx::mbar_init(at(sm.raw_full[i]), 1), ptx::mbar_init(at(sm.raw_empty[i]), kConvertWarps);
        for (int i = 0; i < kBuf; ++i) {
            ptx::mbar_init(at(sm.k_full[i]), kConvertWarps), ptx::mbar_init(at(sm.v_full[i]), kConvertWarps);
            ptx::mbar_init(at(sm.kv_empty[i]), 2);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(at(sm.s_full[i][0]), 1), ptx::mbar_init(at(sm.s_full[i][1]), 1);
            ptx::mbar_init(at(sm.p_full[i][0]), 4), ptx::mbar_init(at(sm.p_full[i][1]), 4);
        }
        for (int i = 0; i < kExps; ++i) ptx::mbar_init(at(sm.e_full[i]), 1);
        ptx::mbar_init(at(sm.o_full), 2);
        sm.poisoned = 0;
        ptx::fence_mbar_init();
        ptx::prefetch_tensormap(&maps.k);
        ptx::prefetch_tensormap(&maps.v);
        if constexpr (FOUR) {
            ptx::prefetch_tensormap(&maps.k_scale);
            ptx::prefetch_tensormap(&maps.v_scale);
        }
    }
    __syncthreads();
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();
    const Work w = work_of(p, grid, blockIdx.x, true);
    if (!w.live || (w.n == 0 && w.parts > 1)) return;          // the join leaves empty parts out too
    const int G = p.Hq / p.Hk, P = p.P;
    if (warp == kIssuer) {
        ptx::tmem_alloc(ptx::smem_u32(&sm.tmem), 512);
        ptx::tmem_relinquish();
    }
    // The softmax warps and the issuers meet here when the q tile is there; the first keys are
    // fetched and turned meanwhile.
    auto meet = [&] {
        ptx::tc_fence_before();
        ptx::named_sync(1, 32 * (kSoftmaxWarps + 2));
        ptx::tc_fence_after();
        return sm.tmem;
    };
    // Steps in which some row of the CTA does not see some key.
    const int pos_lo = w.first + w.row0 / G, pos_hi = w.first + (min(w.row0 + kRows, w.nrows) - 1) / G;
    auto partial = [&](int key0, int keys = kKeys) { return key0 + keys - 1 > pos_lo || (p.window > 0 && key0 <= pos_hi - p.window); };

    if (warp < kSoftmaxWarps) {
        // ------------------------------------------------ softmax: a thread owns a row.
        more_registers<kSoftmaxRegs>();
        const int t = warp >> 2, r = t * 128 + (warp & 3) * 32 + lane, row = w.row0 + r;
        const uint32_t quarter = (uint32_t)((warp & 3) * 32) << 16;
        const bool live = row < w.nrows;
        const int token = live ? row / G : 0, head = w.h * G + (live ? row - token * G : 0);
        const int pos = live ? w.first + token : -1;
        const int low = p.window > 0 ? pos - p.window : -1;    // keys low < key <= pos are seen
        float qs = 0.f;
        if (w.n > 0) {
            // The warp's rows of q are copied to their places in the swizzled operand tile, whole
            // rows at a time, and turned there by a thread each into fp16 times a power of two. A
            // negative scale goes into q: the maximum is taken before scaling.  (Turned on the way,
            // a row over the lanes, with a reduction each, they took three times as long.)
            constexpr int kLanes = D / 4, kAtOnce = 32 / kLanes;       // lanes of a row (8 bytes each), rows of a copy
            const int r0 = (warp & 3) * 32, rows = min(32, w.nrows - (w.row0 + t * 128 + r0)), in = lane % kLanes;
            const uint16_t *mine = p.q + (int64_t)(w.start + token) * p.q_token + head * p.q_head;     // this lane's row
            const uint32_t base = ptx::smem_u32(sm.q[t]), to = base + (uint32_t)(in / 16) * 16384u + (in & 1) * 8;
#pragma unroll 8
            for (int i = lane / kLanes; i < 32; i += kAtOnce) {
                const uint16_t *from = reinterpret_cast<const uint16_t *>(__shfl_sync(~0u, reinterpret_cast<uint64_t>(mine), i)) + in * 4;
                cp_async8(to + (r0 + i) * 128 + (((in >> 1 & 7) ^ (i & 7)) << 4), from, i < rows ? 8 : 0);
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncwarp();
            const uint32_t own = base + (r0 + lane) * 128;
            uint4 x[D / 8];
            uint32_t top = 0u;                                         // largest finite magnitude, as bf16 bits
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
                x[c] = lds_v4(own + (c >> 3) * 16384u + (((c & 7) ^ (lane & 7)) << 4));
                top = __vmaxu2(top, __vmaxu2(__vmaxu2(x[c].x & 0x7FFF7FFFu, x[c].y & 0x7FFF7FFFu),
                                             __vmaxu2(x[c].z & 0x7FFF7FFFu, x[c].w & 0x7FFF7FFFu)));
            }
            top = max(top & 0xFFFFu, top >> 16);
            if (top >= 0x7F80u) {
                top = 0u;
#pragma unroll
                for (int c = 0; c < D / 8; ++c) {
                    const uint32_t words[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t a = words[k] & 0x7FFFu, b = words[k] >> 16 & 0x7FFFu;
                        top = max(top, max(a < 0x7F80u ? a : 0u, b < 0x7F80u ? b : 0u));
                    }
                }
            }
            const int up = query_shift(__uint_as_float(top << 16));
            const float f = __uint_as_float(__float_as_uint(exp2_int(up)) | (p.scale_log2 < 0.f ? 0x80000000u : 0u));
            qs = exp2_int(-up) * fabsf(p.scale_log2) * kValueUnit;
            if constexpr (FOUR) qs = fminf(qs, 3.4028234663852886e38f);    // an infinite factor would make NaN of sums that are 0
            auto turn = [&](uint32_t v) {
                const float2 y = ptx::fmul2(make_float2(bf16_lo(v), bf16_hi(v)), make_float2(f, f));
                return f32x2_to_f16x2(y.x, y.y);
            };
#pragma unroll
            for (int c = 0; c < D / 8; ++c)
                if constexpr (FOUR) {                                  // in the order of a word's codes
                    const uint4 y = make_uint4(turn(ptx::prmt(x[c].x, x[c].z, 0x5410u)), turn(ptx::prmt(x[c].x, x[c].z, 0x7632u)),
                                               turn(ptx::prmt(x[c].y, x[c].w, 0x5410u)), turn(ptx::prmt(x[c].y, x[c].w, 0x7632u)));
                    sts_v4(own + (c >> 3) * 16384u + (((c & 7) ^ (lane & 7)) << 4), y.x, y.y, y.z, y.w);
                } else {
                    sts_v4(own + (c >> 3) * 16384u + (((c & 7) ^ (lane & 7)) << 4), turn(x[c].x), turn(x[c].y), turn(x[c].z), turn(x[c].w));
                }
            ptx::fence_proxy_async_smem();
        }
        bool ok = true;
        float m = -INFINITY, l = 0.f;
        float ref = 0.f, limit = -INFINITY;      // of m: what is taken off the scores, what they outgrow it by
        const uint32_t tmem = meet(), sc = tmem + t * 128 + quarter, oc = tmem + 256 + t * D + quarter;
        for (int hs = 0; hs < 2 * w.n; ++hs) {                          // half-steps of 64 keys
            const int j = hs >> 1, h = hs & 1, key0 = (w.lo + j) * kKeys + h * kHalf;
            if (!FOUR && h == 0 && ok) ok = ptx::mbar_wait(at(sm.e_full[j % kExps]), (j / kExps) & 1, &g_prompt_timeouts);
            if (ok) ok = ptx::mbar_wait(at(sm.s_full[t][h]), j & 1, &g_prompt_timeouts);
            ptx::tc_fence_after();
            const float4 *exps = sm.exps[j % kExps] + h * (kHalf / 16);
            auto ex = [&](int g) { return FOUR ? make_float4(1.f, 0.f, 1.f, 0.f) : exps[g]; };
            float v[kHalf];
            tmem_ld32(sc + h * kHalf, v);
            tmem_ld32(sc + h * kHalf + 32, v + 32);
            ptx::tmem_ld_wait();
            // A factor of 0 would make masked scores NaN.
            auto factor = [&](int g) { return fmaxf(qs * ex(g).x, 1.2e-38f); };
            // The row's maximum, by 16 keys (all of one page).
            auto largest = [&] {
                float mx = -INFINITY;
#pragma unroll
                for (int g = 0; g < kHalf / 16; ++g) {
                    const float *x = v + g * 16;
                    const float a = max3(max3(x[0], x[1], x[2]), x[3], x[4]), b = max3(max3(x[5], x[6], x[7]), x[8], x[9]);
                    const float c = max3(max3(x[10], x[11], x[12]), x[13], x[14]);
                    mx = fmaxf(mx, fmaf(max3(max3(a, b, c), x[15], x[15]), factor(g), ex(g).y));
                }
                return mx;
            };
            float deep = 0.f;                                          // of l: the keys with ve below kDeep
            if (partial(key0, kHalf) || ex(0).w != 0.f) {
                const int hi = pos - key0, lo = low - key0;            // of the keys, those in (lo, hi] are seen
#pragma unroll
                for (int k = 0; k < kHalf; ++k)
                    if (k > hi || k <= lo) v[k] = -INFINITY;
                if (ex(0).w != 0.f) {
                    const float mx = largest(), to = mx - m > kPeak ? mx - kStart : m, off = to == -INFINITY ? 0.f : to;
#pragma unroll
                    for (int k = 0; k < kHalf; ++k) {
                        const float f = factor(k / 16);
                        deep += ex(k / 16).y < kDeep ? ex2(fabsf(off) >= kFar ? __fsub_rn(__fmul_rn(v[k], f), off) : fmaf(v[k], f, -off)) : 0.f;
                    }
                }
            }
            constexpr int kF = FOUR ? 1 : kHalf / 16;                  // factors of 16 keys each
            float f[kF];
#pragma unroll
            for (int g = 0; g < kF; ++g) f[g] = factor(g);
            // m follows the maximum when it has been outgrown; rows far from zero (limit: -inf) always come here.
            const float mx = largest();
            if (__any_sync(~0u, mx > limit)) {
                const bool move = mx > limit && mx - m > kPeak;        // what this row alone asks for
                const Rescale by(move ? m - (mx - kStart) : 0.f);
                const float a = by.of_o();
                if (move) m = mx - kStart;
                l = by.of_l(l);
                if (hs > 0) {
                    // The last half-step's product has to be done: its issuer's next signal says so.
                    if (ok) ok = ptx::mbar_wait(at(sm.s_full[t][h ^ 1]), ((hs + 1) >> 1) & 1, &g_prompt_timeouts);
                    ptx::tc_fence_after();
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) {
                        uint32_t o[16];
                        ptx::tmem_ld16(oc + c * 16, o);
                        ptx::tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * a);
                        ptx::tmem_st16(oc + c * 16, o);
                    }
                }
                ref = m == -INFINITY ? 0.f : m, limit = m + kPeak;
                if (fabsf(ref) >= kFar) {                              // products are rounded before m is taken off
                    limit = -INFINITY;
                    if constexpr (!FOUR) ref = 0.f;
#pragma unroll
                    for (int k = 0; k < kHalf; ++k)
                        v[k] = FOUR ? v[k] * f[0] : __fsub_rn(__fsub_rn(fmaf(v[k], f[k / 16 % kF], ex(k / 16).y), m), ex(k / 16).y);
#pragma unroll
                    for (int g = 0; g < kF; ++g) f[g] = 1.f;
                }
            }
            l += deep;
            // Weights, their sum, and fp16 pairs in the place of the scores.
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t hp[16];
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const float4 e = ex(2 * c + g);
                    const float2 ff = make_float2(f[(2 * c + g) % kF], f[(2 * c + g) % kF]), d = make_float2(e.y - ref, e.y - ref);
                    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                    for (int k = 0; k < 16; k += 2) {
                        float2 x = make_float2(v[c * 32 + g * 16 + k], v[c * 32 + g * 16 + k + 1]);
                        ptx::ffma2(x, x, ff, d);
                        x.x = ex2(x.x), x.y = ex2(x.y);
                        sum = ptx::fadd2(sum, x);
                        hp[g * 8 + k / 2] = f32x2_to_f16x2(x.x, x.y);
                    }
                    l = fmaf(sum.x + sum.y, e.z, l);
                }
                ptx::tmem_st16(sc + h * kHalf + c * 16, hp);
            }
            ptx::tmem_st_wait();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(at(sm.p_full[t][h]));
        }
        // ------------------------------------------------ the row's result.
        if (w.n > 0) {
            if (ok) ok = ptx::mbar_wait(at(sm.o_full), 0, &g_prompt_timeouts);
            ptx::tc_fence_after();
        }
        // NaN among the V codes of partly seen steps was taken out of the product; a
        // row that sees such a code takes it here.
        uint32_t nan[D / 32];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) nan[i] = 0u;
        if (sm.poisoned && live) {
            for (int j = 0; j < w.n; ++j) {
                const int key0 = (w.lo + j) * kKeys;
                if (!partial(key0)) continue;
                for (int key = max(key0, low + 1); key <= min(key0 + kKeys - 1, pos); ++key) {
                    const int page = p.page_table[(int64_t)w.b * p.table_stride + key / P];
                    if ((unsigned)page >= (unsigned)p.pages) continue;
                    if constexpr (FOUR) {                              // a scale that is no number: its 32 values
                        const uint8_t *scale = p.v_scale + page * p.scale_page_stride + w.h * p.scale_head_stride + (int64_t)(key % P) * (D / kGroup4);
#pragma unroll
                        for (int i = 0; i < D / 32; ++i)
                            if ((scale[i] & 0x7C) == 0x7C) nan[i] = ~0u;
                        continue;
                    }
                    const uint8_t *code = p.v_cache + page * p.page_stride + w.h * p.head_stride + (int64_t)(key % P) * D;
#pragma unroll
                    for (int i = 0; i < D / 32; ++i)
                        for (int d = 0; d < 32; ++d)
                            if ((code[i * 32 + d] & 0x7F) == 0x7F) nan[i] |= 1u << d;
                }
            }
        }
        // Rows go out by way of shared memory (the q tile's place: its products are done), so
        // that stores cover whole rows; parts for the join go out value by value, a layout in
        // which the lanes' rows are neighbours.
        float4 *part = w.parts > 1 ? reinterpret_cast<float4 *>(part_of<D>(p, grid, w.slot + w.part)) + r : nullptr;
        const float inv = (l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l)) * kValueUnit;
        const int lr = r & 127;
        const uint32_t stage = ptx::smem_u32(sm.q[t]) + lr * (D * 2);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            float v[32];
            if (w.n > 0) {
                tmem_ld32(oc + c * 32, v);
                ptx::tmem_ld_wait();
            } else {
#pragma unroll
                for (int k = 0; k < 32; ++k) v[k] = 0.f;
            }
            if constexpr (FOUR) {                                      // back from the order of a word's codes
#pragma unroll
                for (int k = 0; k < 32; k += 8) {
                    const float y[8] = {v[k], v[k + 2], v[k + 4], v[k + 6], v[k + 1], v[k + 3], v[k + 5], v[k + 7]};
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[k + i] = y[i];
                }
            }
            if (nan[c] != 0u) {
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    if (nan[c] >> k & 1u) v[k] = __int_as_float(0x7FFFFFFF);
            }
            if (part != nullptr) {
#pragma unroll
                for (int k = 0; k < 32; k += 4)
                    if (live) part[(c * 8 + k / 4) * kRows] = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
            } else {
#pragma unroll
                for (int k = 0; k < 32; k += 8)
                    sts_v4(stage + (((c * 4 + k / 8) ^ (lr & 7)) << 4), f32x2_to_bf16x2(v[k] * inv, v[k + 1] * inv),
                           f32x2_to_bf16x2(v[k + 2] * inv, v[k + 3] * inv), f32x2_to_bf16x2(v[k + 4] * inv, v[k + 5] * inv),
                           f32x2_to_bf16x2(v[k + 6] * inv, v[k + 7] * inv));
            }
        }
        if (part == nullptr) {
            __syncwarp();
            constexpr int E = D / 32;
            const int r0 = (warp & 3) * 32, rows = min(32, w.nrows - (w.row0 + t * 128 + r0));
            const int64_t mine = (int64_t)(w.start + token) * p.o_token + head * p.o_head;     // this lane's row
#pragma unroll 8
            for (int i = 0; i < 32; ++i) {
                uint16_t *o = p.out + __shfl_sync(~0u, mine, i) + lane * E;
                if (i >= rows) continue;
                const uint8_t *from = sm.q[t] + (r0 + i) * (D * 2) + (((lane * E / 8) ^ (i & 7)) << 4) + (lane * E * 2 & 15);
                if constexpr (E == 4)
                    *reinterpret_cast<uint2 *>(o) = *reinterpret_cast<const uint2 *>(from);
                else
                    *reinterpret_cast<uint32_t *>(o) = *reinterpret_cast<const uint32_t *>(from);
            }
        }
        if (live) {
            if (part != nullptr)
                *reinterpret_cast<float2 *>(part_of<D>(p, grid, w.slot + w.part) + kRows * D + 2 * r) = make_float2(m, l);
            else if (p.lse != nullptr)
                p.lse[(w.start + token) * p.lse_token + head] = l == 0.f ? -INFINITY : kLn2 * (m + log2f(l));
        }
        ptx::tc_fence_before();
    } else if (warp < kProducer) {
        // ------------------------------------------------ codes to fp16 operand tiles.
        fewer_registers<kConvertRegs>();
        // A thread's 16-code chunks of a unit: chunk c of every 128 * 16 / D-th key, so all
        // addresses but the key's are the thread's own.  A chunk makes the 16-byte pieces
        // 2 (c % 4) and + 1 of half c / 4 of the key's row; halves alternate which piece goes
        // first: eight lanes then fill all banks.
        // A 4-bit cache's chunk holds 32 codes, all of one scale, and makes the pieces 4 (c % 2) to + 3 of
        // half c / 2; halves begin two pieces apart.
        constexpr int kOf = FOUR ? 32 : 16;                              // codes of a chunk
        constexpr int kChunks = kUnit * D / kOf / (kConvertWarps * 32), kStep = 128 * kOf / D;
        const int ct = tid - kSoftmaxWarps * 32, c = ct % (D / kOf), key_in = ct / (D / kOf), half = c / (64 / kOf), sw = key_in & 7;
        const uint32_t row_off = half * 16384 + key_in * 128;
        const uint32_t first = row_off + (((2 * (c & 3) + half) ^ sw) << 4), second = row_off + (((2 * (c & 3) + (half ^ 1)) ^ sw) << 4);
        int scale_at[FOUR ? kChunks : 1];
        if constexpr (FOUR) {
            const int box = min(P, kUnit);
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                const int key = key_in + i * kStep;
                scale_at[i] = Smem<D, FOUR>::kRawCodes + key / box * Smem<D, FOUR>::slot(box) + key % box * (D / kGroup4) + c;
            }
        }
        bool ok = true;
        int unit = 0;
        for (int j = 0; j < w.n; ++j) {
            const int key0 = (w.lo + j) * kKeys, buf = j % kBuf;
            const bool mask = partial(key0);
#pragma unroll 1
            for (int which = 0; which < 2; ++which) {
                uint64_t &full = which ? sm.v_full[buf] : sm.k_full[buf];
                const uint32_t dst = ptx::smem_u32(which ? sm.v[buf] : sm.k[buf]);
                // Release e frees K(e) and V(e - 1): K(j) waits for e = j - 2, V(j) for e = j - 1.
                const int freed = j - kBuf + which;
                if (ok && freed >= which) ok = ptx::mbar_wait(at(sm.kv_empty[freed % kBuf]), (freed / kBuf) & 1, &g_prompt_timeouts);
#pragma unroll 1
                for (int u = 0; u < kKeys / kUnit; ++u, ++unit) {
                    const int st = unit % kRaw;
                    if (ok) ok = ptx::mbar_wait(at(sm.raw_full[st]), (unit / kRaw) & 1, &g_prompt_timeouts);
                    uint4 x[kChunks];
                    uint32_t scale[FOUR ? kChunks : 1];
#pragma unroll
                    for (int i = 0; i < kChunks; ++i) x[i] = *reinterpret_cast<const uint4 *>(sm.raw[st] + (ct + i * 128) * 16);
                    if constexpr (FOUR) {
#pragma unroll
                        for (int i = 0; i < kChunks; ++i) scale[i] = sm.raw[st][scale_at[i]];
                    }
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(at(sm.raw_empty[st]));
                    if (mask && which) {
                        // Codes past the end, and NaN that not all rows may see, are cleared.
#pragma unroll
                        for (int i = 0; i < kChunks; ++i) {
                            if constexpr (FOUR) {
                                if (key0 + u * kUnit + key_in + i * kStep >= w.len) scale[i] = 0u;
                                if ((scale[i] & 0x7Cu) == 0x7Cu) scale[i] = 0u, sm.poisoned = 1;
                                continue;
                            }
                            uint32_t *in = reinterpret_cast<uint32_t *>(&x[i]), any = 0u;
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                if (key0 + u * kUnit + key_in + i * kStep >= w.len) in[k] = 0u;
                                const uint32_t hit = (((in[k] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7;
                                in[k] &= ~(hit * 0xFFu);
                                any |= hit;
                            }
                            if (any) sm.poisoned = 1;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < kChunks; ++i) {
                        if constexpr (FOUR) {
                            const __half2 s = __half2half2(__ushort_as_half((unsigned short)(scale[i] << 8)));
                            const __half2 t = __hmul2(s, __float2half2_rn(-1.125f));
                            const uint32_t key_at = dst + (u * kUnit + i * kStep) * 128 + row_off;
                            const uint32_t at = ((4 * (c & 1) + (half != 0 ? 2 : 0)) ^ sw) << 4;      // the first piece's
                            const uint32_t w[4] = {half ? x[i].z : x[i].x, half ? x[i].w : x[i].y, half ? x[i].x : x[i].z, half ? x[i].y : x[i].w};
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const uint4 y = turn4(w[k], s, t);
                                sts_v4(key_at + (at ^ k << 4), y.x, y.y, y.z, y.w);
                            }
                            continue;
                        }
                        uint32_t o[8];
                        e4m3x4_to_f16x2(x[i].x, o[0], o[1]);
                        e4m3x4_to_f16x2(x[i].y, o[2], o[3]);
                        e4m3x4_to_f16x2(x[i].z, o[4], o[5]);
                        e4m3x4_to_f16x2(x[i].w, o[6], o[7]);
                        const uint32_t key_at = dst + (u * kUnit + i * kStep) * 128;
                        const bool flip = half != 0;                     // piece `first` holds the upper 8 values
                        sts_v4(key_at + first, flip ? o[4] : o[0], flip ? o[5] : o[1], flip ? o[6] : o[2], flip ? o[7] : o[3]);
                        sts_v4(key_at + second, flip ? o[0] : o[4], flip ? o[1] : o[5], flip ? o[2] : o[6], flip ? o[3] : o[7]);
                    }
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(at(full));
            }
        }
    } else if (warp >= kProducer) {
        fewer_registers<kOtherRegs>();
    }
    if (warp == kProducer) {
        // ------------------------------------------------ TMA producer: K then V of each step, 64 keys a unit.
        const int parts = P < kUnit ? kUnit / P : 1, box = min(P, kUnit);
        int unit = 0;
        bool ok = true;
        // Lane 8 i + k looks up the page of the k-th 16 keys of step i of four, a window ahead.
        int page = -1, next = -1, ke = 0, ve = 0, nke = 0, nve = 0;
        auto look = [&](int j) {
            next = -1;
            const int key = (w.lo + j + (lane >> 3)) * kKeys + (lane & 7) * 16;
            if (j + (lane >> 3) < w.n && key < w.len) {
                next = p.page_table[(int64_t)w.b * p.table_stride + (key >> p.pshift)];
                if (next < 0) next = p.pages;                          // outside the cache: read as zeros
            }
        };
        auto look_exps = [&] {
            nke = nve = 0;
            if ((unsigned)next < (unsigned)p.pages) {
                nke = p.k_exp[(int64_t)next * p.Hk + w.h];
                nve = p.v_exp[(int64_t)next * p.Hk + w.h];
            }
        };
        look(0);
        for (int j = 0; j < w.n && ok; ++j) {
            if ((j & 3) == 0) page = next;
            for (int i = 0; i < 2 * (kKeys / kUnit) && ok; ++i, ++unit) {
                const int u = i % (kKeys / kUnit), st = unit % kRaw;
                if (unit >= kRaw)
                    ok = __all_sync(~0u, ptx::mbar_wait(at(sm.raw_empty[st]), (unit / kRaw - 1) & 1, &g_prompt_timeouts));
                if (!ok) break;
                const int part = lane % parts, key = u * kUnit + part * box;
                const int id = __shfl_sync(~0u, page, (j & 3) * 8 + ((key / 16) & 7));
                const bool mine = lane < parts && id >= 0;
                const uint32_t bytes = __popc(__ballot_sync(~0u, mine)) * (uint32_t)(box * (FOUR ? D / 2 + D / kGroup4 : D));
                const uint32_t bar = at(sm.raw_full[st]);
                if (lane == 0) ptx::mbar_arrive_expect_tx(bar, bytes);
                __syncwarp();
                if (mine) {
                    const int row = ((w.lo + j) * kKeys + key) & (P - 1);
                    ptx::tma_load_4d(ptx::smem_u32(sm.raw[st]) + part * box * (Smem<D, FOUR>::kRawCodes / kUnit),
                                     i < kKeys / kUnit ? &maps.k : &maps.v, 0, FOUR ? row / 16 : row, w.h, id, bar);
                    if constexpr (FOUR)
                        ptx::tma_load_4d(ptx::smem_u32(sm.raw[st]) + Smem<D, FOUR>::kRawCodes + part * Smem<D, FOUR>::slot(box),
                                         i < kKeys / kUnit ? &maps.k_scale : &maps.v_scale, row * (D / kGroup4) / 4, w.h, id, 0, bar);
                }
                __syncwarp();
            }
            if (!FOUR && (j == 0 || (j & 3) == 2)) look_exps();
            if (FOUR) {
                if ((j & 3) == 0) look(j + 4);
                continue;
            }
            if ((j & 3) == 0) {
                ke = min(max(nke, kExpMin), kExpMax), ve = min(max(nve, kExpMin), kExpMax);
                look(j + 4);
            }
            // Steps back to j - kExps have long been weighed: K of step j - 2 is released after them.
            const uint32_t deep = __ballot_sync(~0u, (float)ve < kDeep);
            if ((lane >> 3) == (j & 3))
                sm.exps[j % kExps][lane & 7] = make_float4(exp2_int(ke), (float)ve, (float)ve < kDeep ? 0.f : exp2_int(-ve),
                                                           deep >> (lane & ~3) & 0xFu ? 1.f : 0.f);
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(at(sm.e_full[j % kExps]));
        }
        for (int i = max(0, unit - kRaw); i < unit; ++i)
            if (!ptx::mbar_wait(at(sm.raw_full[i % kRaw]), (i / kRaw) & 1, &g_prompt_timeouts)) break;
    } else if (warp == kIssuer || warp == kIssuer + 1) {
        // ------------------------------------------------ MMA issuers.
        const int t = warp - kIssuer;
        const uint32_t qk = (1u << 4) | ((uint32_t)(kHalf >> 3) << 17) | (8u << 24);             // fp16 x fp16 -> fp32, M = 128
        const uint32_t pv = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | (8u << 24);    // B along N
        constexpr uint64_t kTileStep = Smem<D, FOUR>::kTile >> 4;
        const uint64_t qd = ptx::sw128_desc(ptx::smem_u32(sm.q)) + (uint64_t)t * kTileStep;
        const uint64_t kd0 = ptx::sw128_desc(ptx::smem_u32(sm.k)), vd0 = sw128_mn_desc(ptx::smem_u32(sm.v), 16384);
        const uint32_t tmem = meet(), sd = tmem + t * 128, od = tmem + 256 + t * D;
        bool ok = w.n > 0;
        auto wait = [&](const uint64_t &bar, int parity) {
            if (ok) ok = ptx::mbar_wait(at(bar), (uint32_t)parity, &g_prompt_timeouts);
        };
        auto scores = [&](int j, int h) {        // S_t half h = q_t K(j)^T
            const uint64_t kd = kd0 + (uint64_t)(j % kBuf) * kTileStep + (uint64_t)h * (kHalf * 128 >> 4);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const uint64_t off = (uint64_t)((k >> 2) * (16384 >> 4) + (k & 3) * 2);
                mma_ss(sd + h * kHalf, qd + off, kd + off, qk, k > 0);
            }
        };
        wait(sm.k_full[0], 0);
        if (__all_sync(~0u, ok)) {
            ptx::tc_fence_after();
            scores(0, 0);
            commit(at(sm.s_full[t][0]));
            scores(0, 1);
            commit(at(sm.s_full[t][1]));
            commit(at(sm.kv_empty[0]));
        }
        for (int j = 0; j < w.n; ++j) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (h == 0) wait(sm.v_full[j % kBuf], (j / kBuf) & 1);
                wait(sm.p_full[t][h], j & 1);
                if (!__all_sync(~0u, ok)) break; // a wait that gave up: nothing more is issued
                ptx::tc_fence_after();
                const uint64_t vd = vd0 + (uint64_t)(j % kBuf) * kTileStep + (uint64_t)h * (kHalf * 128 >> 4);
#pragma unroll
                for (int k = 0; k < kHalf / 16; ++k)                    // O_t += P_t V(j), half h
                    mma_ts(od, sd + h * kHalf + k * 8, vd + (uint64_t)(k * (2048 >> 4)), pv, j > 0 || h > 0 || k > 0);
                if (j + 1 < w.n) {
                    if (h == 0) {
                        wait(sm.k_full[(j + 1) % kBuf], ((j + 1) / kBuf) & 1);
                        if (!__all_sync(~0u, ok)) break;
                        ptx::tc_fence_after();
                    }
                    scores(j + 1, h);
                }
                // Also after the last products, for who waits for them to move O.
                commit(at(sm.s_full[t][h]));
                // Frees K(j + 1) and V(j).
                if (h == 1) commit(at(sm.kv_empty[(j + 1) % kBuf]));
            }
        }
        if (w.n > 0) {
            __syncwarp();
            commit(at(sm.o_full));
            ptx::mbar_wait(at(sm.o_full), 0, &g_prompt_timeouts);      // nothing in flight when tensor memory is freed
        }
    }
    __syncthreads();
    if (warp == kIssuer) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(sm.tmem, 512);
    }
}

// Joins the splits: block (unit, y) takes 32 rows of a unit, a lane each; warp i takes
// every eighth group of four values.
template <int D, bool FOUR>
__global__ void __launch_bounds__(256) prompt_join_kernel(const AttentionArgs p, const PromptGrid grid) {
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();
    const Work w = work_of(p, grid, blockIdx.x, false);
    const int r = blockIdx.y * 32 + (threadIdx.x & 31), warp = threadIdx.x >> 5, row = w.row0 + r;
    if (!w.live || w.parts == 1 || row >= w.nrows) return;
    if (w.slot + w.parts > (int)gridDim.x * grid.splits) return;     // cu_q that does not rise
    const int i = row / p.G, token = w.start + i, head = w.h * p.G + row - i * p.G;
    constexpr int kGroups = D / 4 / 8;
    float m = -INFINITY, l = 0.f;
    float4 o[kGroups];
#pragma unroll
    for (int k = 0; k < kGroups; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = 0; s < w.parts; ++s) {
        const bool any = w.first_of(s) != w.first_of(s + 1);       // without keys nothing was written
        const float *part = part_of<D>(p, grid, w.slot + s);
        const float2 ml = any ? __ldcs(reinterpret_cast<const float2 *>(part + kRows * D + 2 * r)) : make_float2(-INFINITY, 0.f);
        const float mx = fmaxf(m, ml.x), ref = mx == -INFINITY ? 0.f : mx;
        const Rescale old(m - ref), more(ml.x - ref);
        const float a = old.of_o(), b = more.of_o();
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
            const float4 v = any ? __ldcs(reinterpret_cast<const float4 *>(part) + (warp + 8 * k) * kRows + r) : make_float4(0.f, 0.f, 0.f, 0.f);
            o[k].x = o[k].x * a + v.x * b, o[k].y = o[k].y * a + v.y * b;
            o[k].z = o[k].z * a + v.z * b, o[k].w = o[k].w * a + v.w * b;
        }
        l = old.of_l(l) + more.of_l(ml.y);
        m = mx;
    }
    const float inv = (l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l)) * (FOUR ? 64.f : 1.f);
    uint16_t *out = p.out + token * p.o_token + head * p.o_head;
#pragma unroll
    for (int k = 0; k < kGroups; ++k)
        *reinterpret_cast<uint2 *>(out + (warp + 8 * k) * 4) =
            make_uint2(f32x2_to_bf16x2(o[k].x * inv, o[k].y * inv), f32x2_to_bf16x2(o[k].z * inv, o[k].w * inv));
    if (warp == 0 && p.lse != nullptr) p.lse[token * p.lse_token + head] = l == 0.f ? -INFINITY : kLn2 * (m + log2f(l));
}

template <int D, bool FOUR>
cudaError_t launch(const AttentionArgs &p, const PromptGrid &g, cudaStream_t stream) {
    // A head's page is one run of bytes: lines of a key (8 bits), or of 16 (4 bits, as words: the box's limit is 256 elements).
    const uint32_t rows = (uint32_t)std::min(p.P, kUnit);
    constexpr uint32_t kLine = FOUR ? 16 * D / 2 : D, kKeysOf = FOUR ? 16 : 1;
    const CUtensorMapDataType type = FOUR ? CU_TENSOR_MAP_DATA_TYPE_UINT32 : CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const uint32_t box[4] = {FOUR ? kLine / 4 : kLine, rows / kKeysOf, 1, 1};
    const uint64_t dims[4] = {box[0], (uint64_t)p.P / kKeysOf, (uint64_t)p.Hk, (uint64_t)p.pages};
    const uint64_t strides[3] = {(uint64_t)kLine, (uint64_t)p.head_stride, (uint64_t)p.page_stride};
    Maps maps{};
    if (!encode_tiled(&maps.k, type, 4, p.k_cache, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE) ||
        !encode_tiled(&maps.v, type, 4, p.v_cache, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE))
        return cudaErrorInvalidValue;
    if constexpr (FOUR) {                                               // a page's scales of a head are one run of bytes
        const uint64_t sdims[4] = {(uint64_t)p.P * D / kGroup4 / 4, (uint64_t)p.Hk, (uint64_t)p.pages, 1};
        const uint64_t sstrides[3] = {(uint64_t)p.scale_head_stride, (uint64_t)p.scale_page_stride, (uint64_t)p.scale_page_stride};
        const uint32_t sbox[4] = {rows * D / kGroup4 / 4, 1, 1, 1};
        if (!encode_tiled(&maps.k_scale, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, p.k_scale, sdims, sstrides, sbox, CU_TENSOR_MAP_SWIZZLE_NONE) ||
            !encode_tiled(&maps.v_scale, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, p.v_scale, sdims, sstrides, sbox, CU_TENSOR_MAP_SWIZZLE_NONE))
            return cudaErrorInvalidValue;
    }
    const int smem = (int)sizeof(Smem<D, FOUR>) + 1024;
    cudaError_t e = raise_smem_limit((const void *)prompt_kernel<D, FOUR>, current_device(), smem);
    if (e != cudaSuccess) return e;
    const unsigned units = (unsigned)(g.tiles * p.Hk);
    e = launch_pdl(prompt_kernel<D, FOUR>, dim3(units * (unsigned)g.splits), dim3(kThreads), smem, stream, maps, p, g);
    if (e != cudaSuccess || g.splits == 1) return e;
    return launch_pdl(prompt_join_kernel<D, FOUR>, dim3(units, kRows / 32), dim3(256), 0, stream, p, g);
}

}  // namespace

PromptGrid prompt_grid(int64_t T, int B, int max_q, bool uniform, int Hq, int Hk, int64_t max_len) {
    const int G = Hq / Hk;
    PromptGrid g{};
    g.tiles = uniform ? B * (int)(((int64_t)max_q * G + kRows - 1) / kRows) : (int)(T * G / kRows) + B;
    // The most parts that find_listed may choose.  Where splitting is in question, the list
    // and the join's launch cost 5-7 us (two prompts of 256 tokens: 18.9 us without, 25.3
    // with), and CTAs without a part 1.5 us each on their SM (4096 tokens, 512 tiles: 124 us
    // against 150 with as many such then); what it gains: 701 tokens behind 8300 beside three short
    // prompts 127 -> 117 us, two of 512 behind 15500 (one shorter) 217 -> 135, eight of 100
    // behind up to 5900 100 -> 65.  The lengths are not known here, and the page table's width
    // stands for them: with a table of 2048 pages of 64 a prompt of 66 tokens behind nothing takes
    // 17.2 us and 100 MB of workspace, with one of 2 pages 10.2 us and none.
    const int64_t units = std::max<int64_t>(1, (int64_t)g.tiles * Hk), steps = (max_len + kKeys - 1) / kKeys;
    g.splits = steps < kShortSteps || (units >= kSms * 3 / 4 && steps < kLongSteps) ? 1
               : (int)std::max<int64_t>(1, std::min(std::min<int64_t>(steps / kMinSteps, kSms), kMostCtas / units));
    return g;
}

size_t prompt_workspace_bytes(const PromptGrid &g, int Hk, int D) {
    return g.splits == 1 ? 0 : (size_t)g.tiles * Hk * g.splits * kRows * (D + 2) * sizeof(float);
}

cudaError_t launch_prompt(const AttentionArgs &p, const PromptGrid &g, cudaStream_t stream) {
    if (p.k_scale != nullptr) return p.D == 128 ? launch<128, true>(p, g, stream) : launch<64, true>(p, g, stream);
    return p.D == 128 ? launch<128, false>(p, g, stream) : launch<64, false>(p, g, stream);
}

uint32_t prompt_timeouts(bool reset) {
    unsigned int v = 0;
    cudaMemcpyFromSymbol(&v, g_prompt_timeouts, sizeof(v));
    if (reset) {
        const unsigned int zero = 0;
        cudaMemcpyToSymbol(g_prompt_timeouts, &zero, sizeof(zero));
    }
    return v;
}

}  // namespace lowbit
