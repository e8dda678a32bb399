// api.cu -- the C ABI of liblowbit (declared in include/lowbit.h).
//
// Every entry point validates its arguments on the host before it touches
// CUDA, then enqueues the kernel on the caller's stream.  Nothing here
// allocates device memory or synchronises.
#include <atomic>
#include <cstdint>

#include "common.cuh"
#include "ptx.cuh"

namespace {

// Self-test of the bounded wait: one thread waits on an mbarrier that nothing
// arrives on, through the same helper every kernel uses.  After the helper's
// limit the wait gives up, counts itself in g_selftest_timeouts and the kernel
// returns; nothing faults and the context stays usable.
__device__ unsigned int g_selftest_timeouts;

__global__ void wait_selftest_kernel(uint32_t *gave_up) {
    __shared__ __align__(8) uint64_t bar;
    const uint32_t b = lowbit::ptx::smem_u32(&bar);
    lowbit::ptx::mbar_init(b, 1);
    lowbit::ptx::fence_mbar_init();
    const bool ok = lowbit::ptx::mbar_wait(b, 0, &g_selftest_timeouts);   // phase 0 never completes
    *gave_up = ok ? 0u : 1u;
}

uint32_t selftest_timeouts(bool reset) {
    unsigned int v = 0;
    cudaMemcpyFromSymbol(&v, g_selftest_timeouts, sizeof(v));
    if (reset) {
        const unsigned int zero = 0;
        cudaMemcpyToSymbol(g_selftest_timeouts, &zero, sizeof(zero));
    }
    return v;
}

bool bits_ok(int bits) { return bits >= 1 && bits <= 7; }
bool group_ok(int g) { return g == 32 || g == 64 || g == 128 || g == 256; }
bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Largest sizes accepted: every index the kernels form stays inside int32 for
// per-row quantities and int64 for whole-buffer offsets.
constexpr int64_t kMaxDim = (int64_t)1 << 30;

// 0 = unknown, 1 = sm_103, 2 = other.  One slot per device ordinal.
std::atomic<int> g_device_ok[64];

lowbit_status check_device() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return LOWBIT_ECUDA;
    if (dev < 0 || dev >= 64) return LOWBIT_EUNSUPPORTED;
    int state = g_device_ok[dev].load(std::memory_order_relaxed);
    if (state == 0) {
        int major = 0, minor = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
            return LOWBIT_ECUDA;
        state = (major == 10 && minor == 3) ? 1 : 2;
        g_device_ok[dev].store(state, std::memory_order_relaxed);
    }
    return state == 1 ? LOWBIT_OK : LOWBIT_EUNSUPPORTED;
}

lowbit_status from_cuda(cudaError_t e) { return e == cudaSuccess ? LOWBIT_OK : LOWBIT_ECUDA; }

lowbit_status check_pack_args(const void *in, const void *out, int64_t N, int64_t K, int bits,
                              const void *code_buf) {
    if (!bits_ok(bits) || N < 0 || K < 0 || N > kMaxDim || K > kMaxDim || K % 8 != 0)
        return LOWBIT_EINVAL;
    if (N == 0 || K == 0) return LOWBIT_OK;
    if (in == nullptr || out == nullptr || !aligned(code_buf, 8)) return LOWBIT_EINVAL;
    return LOWBIT_OK;
}

lowbit_status check_linear_args(const uint16_t *x, const uint8_t *w, const uint16_t *s,
                                const uint16_t *z, const uint16_t *bias, const uint16_t *y,
                                int64_t M, int64_t K, int64_t N, int bits, int group) {
    if (!bits_ok(bits) || !group_ok(group)) return LOWBIT_EINVAL;
    if (M < 0 || N < 0 || K <= 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim) return LOWBIT_EINVAL;
    if (K % group != 0) return LOWBIT_EINVAL;
    if (M == 0 || N == 0) return LOWBIT_OK;
    if (!x || !w || !s || !z || !y) return LOWBIT_EINVAL;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(s, 2) || !aligned(z, 2) || !aligned(y, 2))
        return LOWBIT_EINVAL;
    if (bias != nullptr && !aligned(bias, 2)) return LOWBIT_EINVAL;
    return LOWBIT_OK;
}

bool empty(const lowbit_sequences *s) { return s->batch == 0 || s->tokens == 0; }

// The sizes alone: what the workspace's size follows from.
lowbit_status check_sizes(const lowbit_cache *c, const lowbit_sequences *s, int heads) {
    if (c == nullptr || s == nullptr) return LOWBIT_EINVAL;
    if (s->batch < 0 || s->tokens < 0 || s->batch > kMaxDim || s->tokens > kMaxDim || s->width < 0 || s->width > kMaxDim)
        return LOWBIT_EINVAL;
    if (c->kv_heads <= 0 || c->kv_heads > 65535 || heads <= 0 || heads % c->kv_heads != 0 || c->pages < 0 ||
        (c->head_dim != 64 && c->head_dim != 128))
        return LOWBIT_EINVAL;
    if (c->page < 16 || c->page > 256 || (c->page & (c->page - 1)) != 0) return LOWBIT_EINVAL;
    // Rows (tokens times heads of a group), lengths and a sequence's tiles stay inside int32.
    if ((int64_t)s->tokens * (heads / c->kv_heads) > kMaxDim || (int64_t)s->width * c->page > kMaxDim ||
        (int64_t)s->width * c->page * c->kv_heads > (int64_t)1 << 34)
        return LOWBIT_EINVAL;
    if (empty(s)) return LOWBIT_OK;
    if (s->cu_q == nullptr ? s->tokens % s->batch != 0 : s->max_q <= 0) return LOWBIT_EINVAL;
    return c->pages == 0 || s->width == 0 ? LOWBIT_EINVAL : LOWBIT_OK;
}

lowbit_status check_cache(const lowbit_cache *c, const lowbit_sequences *s, int heads) {
    const lowbit_status st = check_sizes(c, s, heads);
    if (st != LOWBIT_OK || empty(s)) return st;
    if (s->table_stride < s->width) return LOWBIT_EINVAL;
    if (!c->k || !c->v || !c->k_exp || !c->v_exp || !s->page_table || !s->lens) return LOWBIT_EINVAL;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(s->page_table, 4) || !aligned(s->lens, 4) ||
        (s->cu_q != nullptr && !aligned(s->cu_q, 4)))
        return LOWBIT_EINVAL;
    const int64_t tile = (int64_t)c->page * c->head_dim;
    if (c->head_stride < tile || c->page_stride < tile || c->head_stride % 16 != 0 || c->page_stride % 16 != 0 ||
        c->head_stride >= ((int64_t)1 << 40) || c->page_stride >= ((int64_t)1 << 40))
        return LOWBIT_EINVAL;
    return LOWBIT_OK;
}

// Rows of head_dim 16-bit values that can be moved in 16-byte vectors.
bool vector_rows(const void *p, int64_t token, int64_t head) { return aligned(p, 16) && token % 8 == 0 && head % 8 == 0; }

// Crossover between the decode kernels and the batched tensor-core kernel
// (qmm), measured on GB300 in-stream at b = 4 for the Llama-3.1-8B shapes and
// the 3B gate+up and down, g = 32 / 64 / 128, M = 2..16.  The tensor-core
// decode kernel reads the weights once per launch of up to 2 (g = 32), 4
// (g = 64) or 8 (g >= 128) rows of x, so its time grows with the launches
// ("passes"); qmm's is nearly flat in M but grows as g shrinks (a K step of
// 128 codes has 128 / g groups to rescale): gate+up takes 47 / 78 / 141 us at
// g = 128 / 64 / 32.  The decode path wins up to 128 / g passes (M <= 8 for
// g <= 128): e.g. g = 32 gate+up at M = 4: 30 against 141 us; g = 64 o at
// M = 8: 11.4 against 15.0 us.  For N >= 24576 (gate+up: qmm runs 232 row
// tiles, a second wave on 80 of the 152 SMs) twice as many passes still win
// (g = 128 at M = 12 / 16: 37.6 / 44.4 against 46.9 / 47.1 us).  With
// K > 8192 the decode kernel splits K over clusters of three or more CTAs and
// loses beyond 4 / 6 / 8 rows at g = 128 / 64 / 32 (down at g = 128, M = 5:
// 26.4 against 24.1 us; g = 64, M = 8: 35.8 against 32.2 us).  Where the
// decode kernel does not take the shape, the CUDA-core kernel reads the
// weights once per two rows of x and wins up to M = 2, or up to M = 6 for
// layers of N >= 9424 outputs.
constexpr int64_t kQmvMaxM = 2;
constexpr int64_t kQmvMaxMWide = 6;
constexpr int64_t kWideN = 9424;          // 76 row tiles of 124: half the SMs
constexpr int64_t kClusterK = 8192;       // above: the decode kernel splits K over >= 3 CTAs
constexpr int64_t kTwoWaveN = 24576;      // qmm needs more than one wave of row tiles at M <= 128

// Decode passes that still beat qmm, and rows of x beyond which a K split over
// clusters loses.  (Group 256 keeps one pass: its qmm rescales once per two K
// steps, and its two-pass crossover was not measured.)
int64_t decode_max_passes(int group, int64_t N) {
    const int64_t p = group >= 128 ? 1 : 128 / group;
    return (N >= kTwoWaveN && group <= 128) ? 2 * p : p;
}
int64_t cluster_max_rows(int group) { return group >= 128 ? 4 : (group == 64 ? 6 : 8); }

}  // namespace

extern "C" {

const char *lowbit_status_string(lowbit_status status) {
    switch (status) {
        case LOWBIT_OK: return "ok";
        case LOWBIT_EINVAL: return "invalid argument";
        case LOWBIT_EUNSUPPORTED: return "unsupported device (needs sm_103 / GB300)";
        case LOWBIT_ECUDA: return "CUDA error";
        default: return "unknown status";
    }
}

size_t lowbit_packed_bytes(int64_t N, int64_t K, int bits) {
    // Range first, so that K * bits cannot overflow.
    if (!bits_ok(bits) || N < 0 || K < 0 || N > kMaxDim || K > kMaxDim) return 0;
    if ((K * bits) % 8 != 0) return 0;
    return (size_t)(N * (K * bits / 8));
}

lowbit_status lowbit_pack_weights(const uint8_t *codes, uint8_t *packed, int64_t N, int64_t K,
                                  int bits, lowbit_stream_t stream) {
    lowbit_status st = check_pack_args(codes, packed, N, K, bits, codes);
    if (st != LOWBIT_OK || N == 0 || K == 0) return st;
    if ((st = check_device()) != LOWBIT_OK) return st;
    return from_cuda(lowbit::launch_pack(codes, packed, N, K, bits, (cudaStream_t)stream));
}

lowbit_status lowbit_unpack_weights(const uint8_t *packed, uint8_t *codes, int64_t N, int64_t K,
                                    int bits, lowbit_stream_t stream) {
    lowbit_status st = check_pack_args(packed, codes, N, K, bits, codes);
    if (st != LOWBIT_OK || N == 0 || K == 0) return st;
    if ((st = check_device()) != LOWBIT_OK) return st;
    return from_cuda(lowbit::launch_unpack(packed, codes, N, K, bits, (cudaStream_t)stream));
}

lowbit_status lowbit_quantize_weights(const void *w, lowbit_dtype dtype, uint8_t *packed,
                                      uint16_t *scales, uint16_t *zeros, int64_t N, int64_t K,
                                      int bits, int group, lowbit_stream_t stream) {
    if (!bits_ok(bits) || !group_ok(group) || N < 0 || K <= 0 || N > kMaxDim || K > kMaxDim ||
        K % group != 0)
        return LOWBIT_EINVAL;
    if (dtype != LOWBIT_DTYPE_F32 && dtype != LOWBIT_DTYPE_BF16 && dtype != LOWBIT_DTYPE_F16)
        return LOWBIT_EINVAL;
    if (N == 0) return LOWBIT_OK;
    if (!w || !packed || !scales || !zeros) return LOWBIT_EINVAL;
    if (!aligned(w, 16) || !aligned(scales, 2) || !aligned(zeros, 2))
        return LOWBIT_EINVAL;
    lowbit_status st = check_device();
    if (st != LOWBIT_OK) return st;
    return from_cuda(lowbit::launch_quantize(w, (int)dtype, packed, scales, zeros, N, K, bits,
                                             group, (cudaStream_t)stream));
}

lowbit_path lowbit_select_path(int64_t M, int64_t K, int64_t N, int bits, int group) {
    if (!bits_ok(bits) || !group_ok(group) || M < 0 || N < 0 || K <= 0 || K % group != 0 ||
        M > kMaxDim || N > kMaxDim || K > kMaxDim)
        return LOWBIT_PATH_AUTO;
    // qmm needs K % 128 == 0; other shapes stay on the decode kernels.
    if (K % 128 != 0) return LOWBIT_PATH_QMV;
    if (lowbit::qmv_mma_shape_ok(K, group)) {
        const int64_t rows = lowbit::qmv_mma_rows(group);
        const int64_t passes = (M + rows - 1) / rows;
        return (passes <= decode_max_passes(group, N) && !(K > kClusterK && M > cluster_max_rows(group)))
                   ? LOWBIT_PATH_QMV : LOWBIT_PATH_QMM;
    }
    return (M <= kQmvMaxM || (M <= kQmvMaxMWide && N >= kWideN)) ? LOWBIT_PATH_QMV : LOWBIT_PATH_QMM;
}

lowbit_status lowbit_linear_ex(const uint16_t *x, const uint8_t *packed_w, const uint16_t *scales,
                               const uint16_t *zeros, const uint16_t *bias, uint16_t *y,
                               int64_t M, int64_t K, int64_t N, int bits, int group,
                               lowbit_path path, lowbit_stream_t stream) {
    if (path != LOWBIT_PATH_AUTO && path != LOWBIT_PATH_QMV && path != LOWBIT_PATH_QMM)
        return LOWBIT_EINVAL;
    lowbit_status st = check_linear_args(x, packed_w, scales, zeros, bias, y, M, K, N, bits, group);
    if (st != LOWBIT_OK || M == 0 || N == 0) return st;
    if ((st = check_device()) != LOWBIT_OK) return st;
    if (path == LOWBIT_PATH_AUTO) path = lowbit_select_path(M, K, N, bits, group);
    cudaStream_t s = (cudaStream_t)stream;
    if (path == LOWBIT_PATH_QMV)
        return from_cuda(lowbit::launch_qmv(x, packed_w, scales, zeros, bias, y, M, K, N, bits, group, s));
    if (!lowbit::qmm_supported(K, x, packed_w)) return LOWBIT_EUNSUPPORTED;
    return from_cuda(lowbit::launch_qmm(x, packed_w, scales, zeros, bias, y, M, K, N, bits, group, s));
}

lowbit_status lowbit_linear(const uint16_t *x, const uint8_t *packed_w, const uint16_t *scales,
                            const uint16_t *zeros, const uint16_t *bias, uint16_t *y, int64_t M,
                            int64_t K, int64_t N, int bits, int group, lowbit_stream_t stream) {
    return lowbit_linear_ex(x, packed_w, scales, zeros, bias, y, M, K, N, bits, group,
                            LOWBIT_PATH_AUTO, stream);
}

lowbit_status lowbit_linear_swiglu(const uint16_t *x, const uint8_t *packed_w, const uint16_t *scales,
                                   const uint16_t *zeros, const uint16_t *bias, uint16_t *y,
                                   int64_t M, int64_t K, int64_t F, int bits, int group,
                                   lowbit_stream_t stream) {
    if (F < 0 || F > kMaxDim / 2) return LOWBIT_EINVAL;
    lowbit_status st = check_linear_args(x, packed_w, scales, zeros, bias, y, M, K, 2 * F, bits, group);
    if (st != LOWBIT_OK || M == 0 || F == 0) return st;
    if ((st = check_device()) != LOWBIT_OK) return st;
    return from_cuda(lowbit::launch_qmv_gated(x, packed_w, scales, zeros, bias, y, M, K, F, bits, group,
                                              (cudaStream_t)stream));
}

lowbit_status lowbit_kv_append(const lowbit_kv_append_args *a, const lowbit_cache *c, const lowbit_sequences *s,
                               lowbit_stream_t stream) {
    if (a == nullptr) return LOWBIT_EINVAL;
    lowbit_status st = check_cache(c, s, a->heads);
    if (st != LOWBIT_OK) return st;
    if (a->rotary_dim < 0 || a->rotary_dim > c->head_dim || a->rotary_dim % 2 != 0) return LOWBIT_EINVAL;
    if (s->batch == 0 || s->tokens == 0) return LOWBIT_OK;
    if (!a->q || !a->k || !a->v || !a->q_out || !aligned(a->q, 2) || !aligned(a->k, 2) || !aligned(a->v, 2) ||
        !aligned(a->q_out, 2))
        return LOWBIT_EINVAL;
    if (a->rotary_dim > 0 && (a->turns == nullptr || !aligned(a->turns, 8))) return LOWBIT_EINVAL;
    if ((st = check_device()) != LOWBIT_OK) return st;
    lowbit::AppendArgs p{};
    p.q = a->q, p.k = a->k, p.v = a->v, p.q_out = a->q_out;
    p.k_cache = c->k, p.v_cache = c->v, p.k_exp = c->k_exp, p.v_exp = c->v_exp;
    p.page_table = s->page_table, p.lens = s->lens, p.cu_q = s->cu_q, p.turns = a->turns;
    p.q_token = a->q_token, p.q_head = a->q_head, p.k_token = a->k_token, p.k_head = a->k_head;
    p.v_token = a->v_token, p.v_head = a->v_head, p.o_token = a->o_token, p.o_head = a->o_head;
    p.page_stride = c->page_stride, p.head_stride = c->head_stride, p.table_stride = s->table_stride;
    p.factor = a->factor;
    p.T = s->tokens, p.B = s->batch, p.max_q = s->max_q, p.Hq = a->heads, p.Hk = c->kv_heads;
    p.D = c->head_dim, p.P = c->page, p.pages = c->pages, p.width = s->width, p.R = a->rotary_dim;
    p.interleaved = a->interleaved != 0;
    p.qvec = vector_rows(a->q, a->q_token, a->q_head);
    p.kvec = vector_rows(a->k, a->k_token, a->k_head);
    p.vvec = vector_rows(a->v, a->v_token, a->v_head);
    p.ovec = vector_rows(a->q_out, a->o_token, a->o_head);
    return from_cuda(lowbit::launch_kv_append(p, (cudaStream_t)stream));
}

size_t lowbit_attention_workspace(int32_t heads, const lowbit_cache *c, const lowbit_sequences *s) {
    if (check_sizes(c, s, heads) != LOWBIT_OK || empty(s)) return 0;
    const bool uniform = s->cu_q == nullptr;
    return lowbit::attention_workspace_bytes(s->tokens, s->batch, uniform ? s->tokens / s->batch : s->max_q, uniform,
                                             heads, c->kv_heads, c->head_dim, (int64_t)s->width * c->page);
}

lowbit_status lowbit_attention(const lowbit_attention_args *a, const lowbit_cache *c, const lowbit_sequences *s,
                               lowbit_stream_t stream) {
    if (a == nullptr) return LOWBIT_EINVAL;
    lowbit_status st = check_cache(c, s, a->heads);
    if (st != LOWBIT_OK) return st;
    if (a->window < 0 || !(a->scale > -1e30f && a->scale < 1e30f)) return LOWBIT_EINVAL;
    if (s->batch == 0 || s->tokens == 0) return LOWBIT_OK;
    if (!a->q || !a->out || !aligned(a->q, 8) || !aligned(a->out, 8) || (a->lse != nullptr && !aligned(a->lse, 4)))
        return LOWBIT_EINVAL;
    if (a->q_token % 4 != 0 || a->q_head % 4 != 0 || a->o_token % 4 != 0 || a->o_head % 4 != 0) return LOWBIT_EINVAL;
    if (a->workspace == nullptr || !aligned(a->workspace, 16) ||
        a->workspace_bytes < lowbit_attention_workspace(a->heads, c, s))
        return LOWBIT_EINVAL;
    if ((st = check_device()) != LOWBIT_OK) return st;
    lowbit::AttentionArgs p{};
    p.q = a->q, p.out = a->out, p.lse = a->lse;
    p.k_cache = c->k, p.v_cache = c->v, p.k_exp = c->k_exp, p.v_exp = c->v_exp;
    p.page_table = s->page_table, p.lens = s->lens, p.cu_q = s->cu_q;
    p.workspace = static_cast<float *>(a->workspace);
    p.q_token = a->q_token, p.q_head = a->q_head, p.o_token = a->o_token, p.o_head = a->o_head;
    p.lse_token = a->lse_token;
    p.page_stride = c->page_stride, p.head_stride = c->head_stride, p.table_stride = s->table_stride;
    p.scale_log2 = a->scale * 1.4426950408889634f;
    p.T = s->tokens, p.B = s->batch, p.max_q = s->max_q, p.Hq = a->heads, p.Hk = c->kv_heads;
    p.D = c->head_dim, p.P = c->page, p.pages = c->pages, p.width = s->width;
    // A window of all positions hides nothing, and smaller ones keep positions less windows inside int32,
    // also those of rows before position 0.
    p.window = (int64_t)a->window >= (int64_t)s->width * c->page ? 0 : a->window;
    return from_cuda(lowbit::launch_attention(p, (cudaStream_t)stream));
}

lowbit_status lowbit_sample(const lowbit_sample_args *a, lowbit_stream_t stream) {
    if (a == nullptr || a->rows < 0 || a->rows > kMaxDim / 8 || a->vocab <= 0 || a->vocab > (1 << 19))
        return LOWBIT_EINVAL;
    if (a->dtype != LOWBIT_DTYPE_F32 && a->dtype != LOWBIT_DTYPE_BF16 && a->dtype != LOWBIT_DTYPE_F16)
        return LOWBIT_EINVAL;
    if (a->rows == 0) return LOWBIT_OK;
    if (!a->logits || !a->u || !a->token || !aligned(a->logits, a->dtype == LOWBIT_DTYPE_F32 ? 4 : 2) ||
        !aligned(a->u, 4) || !aligned(a->token, 8) || (a->logprob && !aligned(a->logprob, 4)) ||
        (a->temperature && !aligned(a->temperature, 4)) || (a->top_p && !aligned(a->top_p, 4)) ||
        (a->min_p && !aligned(a->min_p, 4)) || (a->top_k && !aligned(a->top_k, 4)))
        return LOWBIT_EINVAL;
    lowbit_status st = check_device();
    if (st != LOWBIT_OK) return st;
    lowbit::SampleArgs p{};
    p.logits = a->logits, p.u = a->u, p.temperature = a->temperature, p.top_p = a->top_p, p.min_p = a->min_p;
    p.top_k = a->top_k, p.token = a->token, p.logprob = a->logprob, p.row_stride = a->row_stride;
    p.temperature_all = a->temperature_all, p.top_p_all = a->top_p_all, p.min_p_all = a->min_p_all;
    p.top_k_all = a->top_k_all, p.B = a->rows, p.V = a->vocab, p.dtype = (int)a->dtype;
    return from_cuda(lowbit::launch_sample(p, (cudaStream_t)stream));
}

lowbit_status lowbit_wait_timeouts(uint32_t *count, int reset) {
    if (count == nullptr) return LOWBIT_EINVAL;
    lowbit_status st = check_device();
    if (st != LOWBIT_OK) return st;
    if (cudaDeviceSynchronize() != cudaSuccess) return LOWBIT_ECUDA;
    *count = lowbit::qmv_timeouts(reset != 0) + lowbit::mma_timeouts(reset != 0) + lowbit::qmm_timeouts(reset != 0) +
             lowbit::attention_timeouts(reset != 0) + selftest_timeouts(reset != 0);
    return cudaGetLastError() == cudaSuccess ? LOWBIT_OK : LOWBIT_ECUDA;
}

lowbit_status lowbit_selftest_wait_timeout(uint32_t *gave_up, lowbit_stream_t stream) {
    if (gave_up == nullptr || !aligned(gave_up, 4)) return LOWBIT_EINVAL;
    lowbit_status st = check_device();
    if (st != LOWBIT_OK) return st;
    wait_selftest_kernel<<<1, 1, 0, (cudaStream_t)stream>>>(gave_up);
    return from_cuda(cudaGetLastError());
}

}  // extern "C"
