/*
 * lowbit.h -- C ABI of liblowbit, a GB300 (sm_103a) library for the
 * weight-only, groupwise, asymmetric low-bit linear layer
 *
 *     y[m,n] = sum_k x[m,k] * W[n,k] + bias[n],
 *     W[n,k] = scale[n, k/g] * q[n,k] + zero[n, k/g],
 *
 * with q an unsigned b-bit code, b = 1..7, and group size g in {32,64,128,256}.
 *
 * Sources (web pages about low-bit weights in torchao / torchchat):
 *   - torchchat PR #1415 "Add torchao mps ops": the scheme quantises only the
 *     weights, groupwise, with bit width 1..7 and group size 32..256;
 *     activations stay floating point.
 *   - ao PR #2167 "metal lowbit kernels: qmv_fast optimization", Summary:
 *     bullet 1 -- scales and zeros are N x num_groups; bullet 2 -- the codes
 *     are stored contiguously, continuing into the next byte once the current
 *     byte is full; bullet 3 -- a fast matrix-vector kernel (qmv) for decode.
 *     A reviewer on the same page asks whether it carries over to gemm (qmm).
 *   - ao issue #3446 "Revamp int4 MPS support in torchao": bias support, and
 *     the per-bit-width packing op `_pack_weight_{n}bit`.
 *
 * Conventions for every entry point:
 *   - All data pointers are DEVICE pointers owned by the caller.  The library
 *     keeps no pointer after a call returns and allocates no device memory.
 *   - Calls only enqueue work on `stream` (a cudaStream_t; NULL is the legacy
 *     default stream) and return without synchronising.  A launch error is
 *     reported as LOWBIT_ECUDA; an error in the kernel itself surfaces at the
 *     caller's next synchronisation, as for any CUDA kernel.
 *   - Arguments are checked on the host before anything is launched; a call
 *     that returns anything but LOWBIT_OK has launched nothing.
 *   - Overlap with the previous kernel in the stream: the linear entry points
 *     launch with programmatic dependent launch, and the decode kernel starts
 *     reading the packed weights, scales and zeros before the previous kernel
 *     in the stream has finished, when that kernel allows it (this library's
 *     linear kernels do, as soon as they start).  x and bias are read, and y
 *     written, only after the previous kernel has completed.  So the packed
 *     weights, scales and zeros of a linear call must not be written by the
 *     kernel immediately before it in the stream if that kernel is one of
 *     this library's linear kernels (which write only y) or another kernel
 *     that allows early launch (the cache, attention and sampling kernels do,
 *     and write no weights).  Ordinary kernels and copies, and this
 *     library's packing and quantising kernels, do not allow it: weights they
 *     produce are always seen complete.
 *   - 16-bit floats are passed as their bit patterns (uint16_t): bf16 for x and
 *     y, IEEE binary16 (fp16) for scales, zeros and bias.
 *   - The library holds no global handle; calls from several host threads are
 *     safe as long as they do not write the same output buffer.
 *
 * Packed layout (ao PR #2167, Summary, bullet 2, read LSB-first): row n of the
 * packed matrix is a byte string of K*b/8 bytes; code k of that row occupies
 * bits [k*b, k*b+b) of the row's little-endian bit stream, where stream bit j
 * is bit (j % 8) of byte (j / 8) and bit 0 of the code comes first.  A code
 * that does not fit in the current byte continues in the next one.  Rows are
 * stored one after another, so the matrix is [N, K*b/8] row-major.
 */
#ifndef LOWBIT_H
#define LOWBIT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define LOWBIT_API __attribute__((visibility("default")))
#else
#define LOWBIT_API
#endif

/* A cudaStream_t (struct CUstream_st *) without pulling in the CUDA headers. */
typedef struct CUstream_st *lowbit_stream_t;

typedef enum {
    LOWBIT_OK = 0,
    LOWBIT_EINVAL = 1,       /* an argument is out of range, null or misaligned   */
    LOWBIT_EUNSUPPORTED = 2, /* the current device is not an sm_103 (GB300) GPU   */
    LOWBIT_ECUDA = 3         /* a CUDA runtime call or a kernel launch failed     */
} lowbit_status;

/* Which kernel lowbit_linear_ex runs. */
typedef enum {
    LOWBIT_PATH_AUTO = 0,    /* what lowbit_linear picks (see lowbit_select_path)  */
    LOWBIT_PATH_QMV = 1,     /* decode (matrix-vector) kernels, any M (in chunks)  */
    LOWBIT_PATH_QMM = 2      /* tensor-core (tcgen05) matrix-matrix kernel, any M  */
} lowbit_path;

/* Element type of a floating-point input that is not fixed by the method. */
typedef enum {
    LOWBIT_DTYPE_F32 = 0,    /* IEEE binary32                                     */
    LOWBIT_DTYPE_BF16 = 1,   /* bfloat16 bit patterns (uint16_t)                  */
    LOWBIT_DTYPE_F16 = 2     /* IEEE binary16 bit patterns (uint16_t)             */
} lowbit_dtype;

/* Human-readable name of a status code.  Never NULL. */
LOWBIT_API const char *lowbit_status_string(lowbit_status status);

/* Bytes of a packed [N, K] matrix of b-bit codes: N * K * bits / 8.
 * Returns 0 when bits is not in 1..7, N or K is negative, or K*bits is not a
 * multiple of 8 (ao PR #2167, Summary, bullet 2: rows are contiguous bit
 * streams, so a row only ends on a byte boundary when K*b % 8 == 0). */
LOWBIT_API size_t lowbit_packed_bytes(int64_t N, int64_t K, int bits);

/* Pack one-code-per-byte codes into the contiguous b-bit layout
 * (ao PR #2167, Summary, bullet 2; the `_pack_weight_{n}bit` op of
 * ao issue #3446, one function here for every bit width).
 *   codes   [N, K] uint8, row-major, device, 8-byte aligned.  Only the low
 *           `bits` bits of each byte are used; higher bits are ignored.
 *   packed  [N, K*bits/8] uint8, row-major, device, written in full.
 *   N >= 0, K >= 0 with K % 8 == 0, bits in 1..7.
 * Errors: LOWBIT_EINVAL for a bad size, bit width, null pointer (when the
 * matrix is not empty) or misaligned `codes`; LOWBIT_EUNSUPPORTED on a device
 * that is not sm_103; LOWBIT_ECUDA when the launch fails.  N == 0 or K == 0
 * is a valid empty call that launches nothing. */
LOWBIT_API lowbit_status lowbit_pack_weights(const uint8_t *codes, uint8_t *packed,
                                  int64_t N, int64_t K, int bits, lowbit_stream_t stream);

/* Inverse of lowbit_pack_weights: one code per output byte (0 .. 2^bits-1).
 * Same layouts, sizes, alignment and errors as lowbit_pack_weights, with
 * `codes` the output (8-byte aligned). */
LOWBIT_API lowbit_status lowbit_unpack_weights(const uint8_t *packed, uint8_t *codes,
                                    int64_t N, int64_t K, int bits, lowbit_stream_t stream);

/* Quantise a floating-point weight matrix groupwise and write it in the
 * packed layout, with its scales and zeros (the `_quantize` step of
 * ao PR #2167, Summary, bullet 1, which produces N x num_groups scales and
 * zeros; the pages do not define it, so this is the min/max asymmetric reading):
 *     zero  = fp16 rounded toward -inf of min(w over the group)
 *     scale = fp16 rounded toward +inf of (max - zero) / (2^bits - 1)
 *     q     = clamp(round-half-to-even((w - zero) / scale), 0, 2^bits - 1)
 * The minimum of a group holding both signed zeros is the first zero in k
 * order.  A constant group (max == min) gets q = 0 and scale = the larger of
 * 2^-14 and fp16 rounded toward +inf of 2 (min - zero).  Every decision is
 * taken in fp64, so the outputs are fully determined by w.
 * Then |w - (scale*q + zero)| <= scale/2 for every weight.
 *   w        [N, K] of `dtype`, row-major, device, 16-byte aligned.
 *            Values must be finite with magnitude at most 32752, so that a
 *            group's zero and range fit fp16.
 *   packed   [N, K*bits/8] uint8, device, written in full (any alignment).
 *   scales   [N, K/group] fp16, row-major, device, 2-byte aligned.
 *   zeros    [N, K/group] fp16, row-major, device, 2-byte aligned.
 *   N >= 0, K > 0, group in {32, 64, 128, 256}, K % group == 0, bits in 1..7.
 *   N == 0 is a valid empty call.  Outputs must not overlap w or each other.
 * Errors: LOWBIT_EINVAL for a bad size, bit width, group, dtype, null or
 * misaligned pointer; LOWBIT_EUNSUPPORTED on a device that is not sm_103;
 * LOWBIT_ECUDA when the launch fails. */
LOWBIT_API lowbit_status lowbit_quantize_weights(const void *w, lowbit_dtype dtype,
                                      uint8_t *packed, uint16_t *scales, uint16_t *zeros,
                                      int64_t N, int64_t K, int bits, int group,
                                      lowbit_stream_t stream);

/* The quantised linear layer (torchchat PR #1415; ao PR #2167 Summary
 * bullets 1-3; bias per ao issue #3446):
 *     y[m,n] = bf16_rn( sum_k x[m,k] * (scale[n,k/g]*q[n,k] + zero[n,k/g]) + bias[n] )
 * accumulated in fp32.
 *   x        [M, K] bf16, row-major, device, 16-byte aligned.
 *   packed_w [N, K*bits/8] uint8 in the packed layout above, 16-byte aligned.
 *   scales   [N, K/group] fp16, row-major, device, 2-byte aligned.
 *   zeros    [N, K/group] fp16, row-major, device, 2-byte aligned.  The zero
 *            is an additive offset: W = scale*q + zero.
 *   bias     [N] fp16 or NULL (no bias), 2-byte aligned.
 *   y        [M, N] bf16, row-major, device, 2-byte aligned; written in full.
 *            y must not overlap any input.
 *   M >= 0, N >= 0, K > 0, group in {32, 64, 128, 256}, K % group == 0,
 *   bits in 1..7.  M == 0 or N == 0 is a valid empty call.
 * The kernel is picked by lowbit_select_path.
 * Errors: LOWBIT_EINVAL for a bad size, bit width, group, null pointer or
 * misaligned pointer; LOWBIT_EUNSUPPORTED on a device that is not sm_103;
 * LOWBIT_ECUDA when a launch fails. */
LOWBIT_API lowbit_status lowbit_linear(const uint16_t *x, const uint8_t *packed_w,
                            const uint16_t *scales, const uint16_t *zeros,
                            const uint16_t *bias, uint16_t *y,
                            int64_t M, int64_t K, int64_t N, int bits, int group,
                            lowbit_stream_t stream);

/* lowbit_linear with the kernel chosen by the caller (both kernels are
 * correct for every M; this is how each is tested and timed on its own).
 * Same arguments and errors as lowbit_linear, plus LOWBIT_EINVAL for an
 * unknown `path` and LOWBIT_EUNSUPPORTED when LOWBIT_PATH_QMM is asked for a
 * shape the tensor-core kernel does not take (K not a multiple of 128). */
LOWBIT_API lowbit_status lowbit_linear_ex(const uint16_t *x, const uint8_t *packed_w,
                               const uint16_t *scales, const uint16_t *zeros,
                               const uint16_t *bias, uint16_t *y,
                               int64_t M, int64_t K, int64_t N, int bits, int group,
                               lowbit_path path, lowbit_stream_t stream);

/* Gate and up projections of a gated MLP fused into one decode call: with the
 * packed matrix holding 2F rows -- rows [0, F) the gate projection, rows
 * [F, 2F) the up projection, each quantised as for lowbit_linear --
 *     a[m,f] = sum_k x[m,k] W[f,k]   + bias[f]
 *     u[m,f] = sum_k x[m,k] W[F+f,k] + bias[F+f]
 *     y[m,f] = silu(a[m,f]) * u[m,f],   silu(a) = a / (1 + e^-a),
 * computed in fp32 and rounded once to bf16 (a and u are never rounded).
 * This is the decode step the pages time (torchchat PR #1415 and ao PR #2167
 * measure Llama token generation, whose MLP applies this activation to its
 * gate and up projections); it saves one launch and one pass over a and u.
 * It runs the decode kernels for every M (up to 8 rows of x per launch on the
 * tensor-core decode kernel, two on the CUDA-core one), so it is meant for
 * decode-sized M.
 *   x        [M, K] bf16, as for lowbit_linear.
 *   packed_w [2F, K*bits/8], scales and zeros [2F, K/group], bias NULL or
 *            [2F] fp16: layouts, alignment and ownership as for lowbit_linear
 *            with N = 2F.
 *   y        [M, F] bf16, device, 2-byte aligned, written in full.
 *   F >= 0; every other size limit as for lowbit_linear.  M == 0 or F == 0 is
 *   a valid empty call.
 * Errors: as for lowbit_linear (LOWBIT_EINVAL also for F < 0). */
LOWBIT_API lowbit_status lowbit_linear_swiglu(const uint16_t *x, const uint8_t *packed_w,
                                   const uint16_t *scales, const uint16_t *zeros,
                                   const uint16_t *bias, uint16_t *y,
                                   int64_t M, int64_t K, int64_t F, int bits, int group,
                                   lowbit_stream_t stream);

/* ---------------------------------------------------------------------------
 * Between the linear layers of a decoder: rotary positions and the write into an
 * 8-bit key-value cache, attention over that cache, and sampling.  (The cache in 4 bits,
 * and what may stand before the rotation, follow: lowbit_cache4, lowbit_kv_prologue.)
 *
 * The cache holds keys and values in pages of `page` tokens, as e4m3 codes with
 * one exponent for each page and key-value head: value = code * 2^exp.  (A power
 * of two, so that scaling is exact, and a page whose exponent grows keeps its
 * older codes but for those that become subnormal.)  Sequence b's token at
 * position i is slot i % page of page page_table[b][i / page].
 *
 * Both calls take sequences of any lengths in one batch: the new tokens of all
 * sequences stand one after another in q, k and v (`tokens` rows), sequence b's
 * at rows [cu_q[b], cu_q[b+1]), or tokens / batch of them each when cu_q is NULL.
 * lens[b] counts the sequence with its new tokens, so new token i of n stands at
 * position lens[b] - n + i.  Lengths, offsets and pages are read on the device:
 * nothing waits for the host, and a captured call follows their values.
 */
typedef struct {
    uint8_t *k, *v;          /* [pages, kv_heads, page, head_dim] e4m3, 16-byte aligned  */
    int8_t *k_exp, *v_exp;   /* [pages, kv_heads], each in [-64, 64]                      */
    int64_t page_stride;     /* bytes from a page to the next, of k and of v               */
    int64_t head_stride;     /* bytes from a head to the next; a head's page is contiguous;
                                both multiples of 16                                      */
    int32_t pages, kv_heads;
    int32_t head_dim;        /* 64 or 128                                                  */
    int32_t page;            /* tokens of a page: 16, 32, 64, 128 or 256                   */
} lowbit_cache;

typedef struct {
    const int32_t *page_table;  /* [batch, width], rows table_stride apart.  Entries past a
                                   sequence's end are not read; one outside the cache is
                                   not written, and reads as zeros                         */
    const int32_t *lens;        /* [batch]                                                 */
    const int32_t *cu_q;        /* [batch + 1], rising from 0 to `tokens`, or NULL          */
    int64_t table_stride;       /* elements                                                */
    int32_t width;              /* columns of page_table: lengths are at most width * page  */
    int32_t batch, tokens;
    int32_t max_q;              /* bound of a sequence's new tokens (cu_q given); tokens past
                                   it are left out: no output of theirs is written, and the
                                   tokens before them keep their positions                 */
} lowbit_sequences;

/* Rotary positions on q and k, and k and v into the cache, in one launch.
 * Pair j of a head's first rotary_dim values turns by 2 pi frac(pos turns[j] / 2^64)
 * (turns[j]: the pair's frequency in turns per position times 2^64; the product
 * wraps exactly, so positions of any size are as exact as small ones):
 *     (a, b) -> factor * (a cos - b sin, a sin + b cos),
 * a pair being values (j, j + rotary_dim/2), or (2j, 2j+1) when `interleaved`.  The
 * rest of the head passes unchanged.  Computed in fp32; q_out is rounded to bf16, the
 * codes to e4m3 (nearest even; infinities and values past 448 * 2^64 stored as 448).
 * A page's exponent is the smallest e >= -64 with every finite new value of that
 * page and head within 448 * 2^e, and at least its present one if the page holds
 * older tokens of the sequence, whose codes are then rounded to the new one.
 *   q, q_out [tokens, heads, head_dim], k, v [tokens, kv_heads, head_dim] bf16, with
 *            strides in elements for tokens and heads, head_dim contiguous, 2-byte
 *            aligned (16-byte aligned rows are read in vectors).  q_out may be q;
 *            otherwise the outputs overlap nothing.
 *   turns    [rotary_dim / 2] int64, device; NULL with rotary_dim == 0.
 *   heads a multiple of kv_heads; rotary_dim even, 0 .. head_dim.
 * New tokens before position 0 or past width * page are rotated but not stored.
 * tokens == 0 or batch == 0 is a valid empty call.
 * Errors: LOWBIT_EINVAL for a bad size, null or misaligned pointer or stride;
 * LOWBIT_EUNSUPPORTED on a device that is not sm_103; LOWBIT_ECUDA when the launch
 * fails. */
typedef struct {
    const uint16_t *q, *k, *v;
    uint16_t *q_out;
    int64_t q_token, q_head, k_token, k_head, v_token, v_head, o_token, o_head;
    const int64_t *turns;
    float factor;
    int32_t heads, rotary_dim, interleaved;
} lowbit_kv_append_args;
LOWBIT_API lowbit_status lowbit_kv_append(const lowbit_kv_append_args *args, const lowbit_cache *cache,
                                          const lowbit_sequences *seqs, lowbit_stream_t stream);

/* What may stand before the rotation and the write, in the same pass:
 *   norms      each head's q and k over its root mean square, times weights:
 *              y = (x r) w, r = 1 / sqrt(mean x^2 + eps), in fp32, every operation rounded
 *              to nearest by itself and the squares added in pairs (neighbours, then neighbouring
 *              sums), so that without a rotation codes next to a border come out the same in any
 *              implementation.  (Cosines and sines of a rotation are off by up to 2 units.)
 *              q_norm, k_norm [head_dim] of norm_dtype, naturally aligned, each may be NULL.
 *   positions  token t's pairs turn by positions[t * positions_token + axis[j]] instead of
 *              its place in its sequence (which still says where it is written): several
 *              axes, as time, height and width of an image's patches.  positions int32,
 *              [tokens, axes] (negative ones turn the other way); axis uint8
 *              [rotary_dim / 2], or NULL: axis 0 for all.  An axis past the last counts as the
 *              last.  axes 1 .. 255.
 * A NULL descriptor, or one with NULL members: none of them. */
typedef struct {
    const void *q_norm, *k_norm;
    const int32_t *positions;
    const uint8_t *axis;
    int64_t positions_token;             /* elements */
    float eps;                           /* not negative */
    int32_t axes;
    lowbit_dtype norm_dtype;
} lowbit_kv_prologue;

/* lowbit_kv_append with norms, or positions of the caller's own, before the write.
 * Errors: also LOWBIT_EINVAL for an eps, axes or norm_dtype out of range, and
 * misaligned pointers. */
LOWBIT_API lowbit_status lowbit_kv_append_ex(const lowbit_kv_append_args *args, const lowbit_kv_prologue *before,
                                             const lowbit_cache *cache, const lowbit_sequences *seqs,
                                             lowbit_stream_t stream);

/* The cache in 4 bits: a token's head in groups of 32 values, each with a scale,
 *     value = (code - 8) * scale,
 * scale an e5m2 number (the upper byte of an fp16), code 4 bits, two to a byte (the even
 * value in the low bits).  Written are codes 1 .. 15 and the smallest scale s >= 2^-14 with
 * amax <= 7.5 s, amax the largest finite magnitude of the group, code - 8 the nearest
 * whole number to value / s (ties to even, within -7 .. 7).  Infinities, and values
 * past 7 * 57344, are stored as 7 s; a group that holds a NaN gets a NaN scale.
 * Scales are read as they are: they have to be finite and not negative, or NaN, which makes
 * all 32 values NaN. */
typedef struct {
    uint8_t *k, *v;              /* [pages, kv_heads, page, head_dim / 2], 16-byte aligned           */
    uint8_t *k_scale, *v_scale;  /* [pages, kv_heads, page, head_dim / 32] e5m2, 16-byte aligned      */
    int64_t page_stride, head_stride;              /* bytes, of k and v, as for lowbit_cache          */
    int64_t scale_page_stride, scale_head_stride;  /* bytes, of k_scale and v_scale, the same rules   */
    int32_t pages, kv_heads;
    int32_t head_dim;            /* 64 or 128                                                        */
    int32_t page;                /* tokens of a page: 16, 32, 64, 128 or 256                         */
} lowbit_cache4;

/* lowbit_kv_append_ex into a 4-bit cache.  A token's codes depend on no other token. */
LOWBIT_API lowbit_status lowbit_kv_append4(const lowbit_kv_append_args *args, const lowbit_kv_prologue *before,
                                           const lowbit_cache4 *cache, const lowbit_sequences *seqs,
                                           lowbit_stream_t stream);

/* The values that a cache holds, for inspection or another use of them: bf16 (exact)
 * [pages, kv_heads, page, head_dim], contiguous, 16-byte aligned.  Codes and scales may
 * be anything.  Errors: LOWBIT_EINVAL for sizes that lowbit_kv_append refuses, null or
 * misaligned pointers or strides; LOWBIT_EUNSUPPORTED, LOWBIT_ECUDA as elsewhere. */
LOWBIT_API lowbit_status lowbit_cache_values(const lowbit_cache *cache, uint16_t *k_out, uint16_t *v_out,
                                             lowbit_stream_t stream);
LOWBIT_API lowbit_status lowbit_cache4_values(const lowbit_cache4 *cache, uint16_t *k_out, uint16_t *v_out,
                                              lowbit_stream_t stream);

/* Softmax attention of the new tokens over the cache: for query row (token, head)
 * at position pos, over the keys t <= pos (and t > pos - window when window > 0)
 *     out = sum_t softmax_t(scale q.k_t) v_t,   lse = ln sum_t e^(scale q.k_t),
 * with k and v the cached values (code * 2^exp), head h reading key-value head
 * h / (heads / kv_heads).  Scores, softmax and sums in fp32 (a weight e^s is off by what fp32
 * rounds of s, over 8 bits with v's exponent added to it); for the product with
 * the codes of v the weights are rounded to fp16, to 2^-11 of themselves, or to 2^-32
 * of the row's largest e^(..) 2^exp (weight times page scale of v) where that is more;
 * out rounded once to bf16.  A row that sees no key gives out 0 and lse -infinity.  What the cache holds
 * at keys that a row does not see (NaN codes among it) does not reach that row.
 *   q, out   [tokens, heads, head_dim] bf16, strides in elements (multiples of 4),
 *            head_dim contiguous, 8-byte aligned.
 *   lse      [tokens, heads] fp32 or NULL, heads contiguous, rows lse_token apart.
 *   workspace  device memory of at least lowbit_attention_workspace bytes, 16-byte
 *            aligned, for this call alone until it has run.
 * tokens == 0 or batch == 0 is a valid empty call.
 * Errors: as for lowbit_kv_append, and LOWBIT_EINVAL for a workspace that is too small. */
typedef struct {
    const uint16_t *q;
    uint16_t *out;
    float *lse;
    int64_t q_token, q_head, o_token, o_head, lse_token;
    void *workspace;
    size_t workspace_bytes;
    float scale;
    int32_t heads, window;
} lowbit_attention_args;
LOWBIT_API lowbit_status lowbit_attention(const lowbit_attention_args *args, const lowbit_cache *cache,
                                          const lowbit_sequences *seqs, lowbit_stream_t stream);

/* Bytes of workspace that lowbit_attention needs for these sizes (of the cache,
 * head counts and dim; of the sequences, batch, tokens, width, max_q and whether
 * cu_q is NULL).  Host-only.  0 for sizes that lowbit_attention rejects. */
LOWBIT_API size_t lowbit_attention_workspace(int32_t heads, const lowbit_cache *cache, const lowbit_sequences *seqs);

/* lowbit_attention over a 4-bit cache, with the same arguments, sizes and guarantees.
 * Scores are taken from the codes and scaled in fp32, for any row of q whose largest |q|
 * times |scale| is a finite fp32 number; the weights are rounded to fp16 for
 * the product with v, to 2^-11 of themselves, or to 2^-32 of the row's largest where that
 * is more. */
LOWBIT_API lowbit_status lowbit_attention4(const lowbit_attention_args *args, const lowbit_cache4 *cache,
                                           const lowbit_sequences *seqs, lowbit_stream_t stream);
LOWBIT_API size_t lowbit_attention4_workspace(int32_t heads, const lowbit_cache4 *cache, const lowbit_sequences *seqs);

/* One token for each row of logits, from a given uniform number.  With m the row's
 * largest logit, s_i = (x_i - m) / temperature and W_i = rint(2^30 e^s_i) (weights
 * are whole numbers, so that sums are exact and a result does not depend on how the
 * work is split): of the tokens in the order (logit falling, index rising) are kept
 *     those with e^s_i >= min_p,
 *     of these the first top_k (top_k <= 0: all),
 *     of these the ones before which less than ceil(top_p * their total W) comes
 *     (top_p >= 1: all; at least one),
 * and token is the first index whose running total of kept W, in index order, passes
 * floor(u * kept total).  logprob is s - ln(kept total / 2^30): the token's
 * log-probability in the distribution that it was drawn from.
 * temperature <= 0: the largest logit's index (the lowest of equals), logprob 0.
 * NaN logits count as -infinity; a row without any logit above that gives token -1
 * and logprob -infinity.  Tokens under 2^-31 of the likeliest are never drawn.
 *   logits   [rows, vocab] of `dtype`, rows row_stride elements apart, naturally aligned.
 *            Read in aligned vectors of 16 bytes: up to 15 bytes before and after a row are
 *            read with it, and not used.
 *   u        [rows] fp32 in [0, 1).
 *   temperature, top_p, min_p [rows] fp32 and top_k [rows] int32, device; each may be
 *            NULL: the scalar of the same name holds for every row then.
 *   token    [rows] int64; logprob [rows] fp32 or NULL.
 *   rows >= 0, 1 <= vocab <= 2^19.  rows == 0 is a valid empty call.
 * Errors: as for lowbit_kv_append. */
typedef struct {
    const void *logits;
    const float *u, *temperature, *top_p, *min_p;
    const int32_t *top_k;
    int64_t *token;
    float *logprob;
    int64_t row_stride;
    float temperature_all, top_p_all, min_p_all;
    int32_t top_k_all, rows, vocab;
    lowbit_dtype dtype;
} lowbit_sample_args;
LOWBIT_API lowbit_status lowbit_sample(const lowbit_sample_args *args, lowbit_stream_t stream);

/* The kernel lowbit_linear runs for this problem, from crossovers measured on
 * GB300: LOWBIT_PATH_QMV when the tensor-core decode kernel takes the shape
 * (K a multiple of 256 up to 32768 with K/group a multiple of 8; one launch
 * per 2 rows of x for group 32, 4 for group 64, 8 for groups 128 and 256) in
 * at most 128/group launches (one for groups 128 and 256), twice as many when
 * N >= 24576 and group <= 128, and, when K > 8192, for M <= 4 (groups 128,
 * 256), 6 (64) or 8 (32); for other K, M <= 2, or M <= 6 when N >= 9424; and
 * whenever K is not a multiple of 128.
 * LOWBIT_PATH_QMM otherwise.  The choice assumes x, the packed weights,
 * scales and zeros 16-byte aligned (the decode path still runs, slower,
 * when they are not).
 * Host-only; never touches the GPU.  Returns LOWBIT_PATH_AUTO for arguments
 * lowbit_linear would reject. */
LOWBIT_API lowbit_path lowbit_select_path(int64_t M, int64_t K, int64_t N, int bits, int group);

/* Every wait inside the library's kernels (a stage of streamed weights, a
 * tensor-core completion) is bounded: one that has not completed after about
 * one second gives up, the kernel finishes without that data (its outputs are
 * then unspecified) and a device-side counter is incremented.  This returns
 * the counter for the current device in *count (0 in normal operation) and
 * clears it when `reset` is non-zero.  Synchronises the current device.
 * Errors: LOWBIT_EINVAL for a NULL `count`; LOWBIT_EUNSUPPORTED on a device
 * that is not sm_103; LOWBIT_ECUDA when the synchronisation or the read
 * fails (for instance after an earlier kernel fault). */
LOWBIT_API lowbit_status lowbit_wait_timeouts(uint32_t *count, int reset);

/* Self-test of the bounded waits: enqueues one single-thread kernel that waits,
 * through the library's bounded-wait helper, on a barrier nothing completes.
 * After the wait limit (about one second) it gives up, writes 1 to *gave_up
 * and counts one timeout (seen by lowbit_wait_timeouts); the kernel then
 * returns normally, so the device stays usable.
 *   gave_up  device pointer to one uint32_t, 4-byte aligned, written by the kernel.
 * Errors: LOWBIT_EINVAL for a NULL or misaligned pointer; LOWBIT_EUNSUPPORTED
 * on a device that is not sm_103; LOWBIT_ECUDA when the launch fails. */
LOWBIT_API lowbit_status lowbit_selftest_wait_timeout(uint32_t *gave_up, lowbit_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LOWBIT_H */
