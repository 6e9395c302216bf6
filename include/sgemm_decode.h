/*
 * sgemm_decode.h -- C ABI of the operators that stand between the projections
 * of a decode step (GB300, sm_103a; the same library as sgemm_skinny.h):
 *
 *   sgemm_bf16_add_rmsnorm       residual add + RMS norm, BF16 or 8-bit output
 *   sgemm_bf16_latent_append     append to a paged latent cache, rotating on the way
 *   sgemm_bf16_latent_attention  attention over that cache (absorbed form)
 *
 * The conventions are those of sgemm_skinny.h: device pointers owned by the
 * caller on the current device, raw BF16 bits, asynchronous work on `stream`,
 * argument checks on the host before anything is enqueued, a status in return.
 * No call allocates or synchronizes, so every call can be captured into a CUDA
 * graph.  Results are deterministic: the same inputs give the same bits.
 * Strides are in elements.  The argument structures are HOST memory, read
 * during the call only; clear them (memset) before filling them in.
 * The kernels are always launched as programmatic dependents of the previous
 * kernel on the stream, and wait for it before they read or write any memory,
 * so the order is that of plain launches.  (One thing is asked of a previous
 * kernel that is a programmatic dependent itself: that it waits for its own,
 * griddepcontrol.wait, as all of this library's do.)
 * `flags`: 0, or SGEMM_FLAG_PDL: the kernel also lets the next one, if it is a
 * programmatic dependent, launch early.  SGEMM_FLAG_WEIGHTS_READONLY is taken
 * beside it and changes nothing; other bits are refused.
 */
#ifndef SGEMM_DECODE_H
#define SGEMM_DECODE_H

#include "sgemm_skinny.h"

#ifdef __cplusplus
extern "C" {
#endif

/* What sgemm_bf16_add_rmsnorm writes as y. */
enum {
    SGEMM_NORM_BF16 = 0,          /* y: BF16 */
    SGEMM_NORM_E4M3_ROW = 1,      /* y: 8 bits (e4m3), one FP32 scale per row */
    SGEMM_NORM_E4M3_GROUP128 = 2  /* y: 8 bits (e4m3), one FP32 scale per 128 columns of a row */
};

/* For every row t < T, with h[c] = x[t][c] + residual[t][c] (residual may be
 * NULL: h = x), in FP32 and not rounded in between:
 *     y[t][c] = h[c] / sqrt(mean_c h[c]^2 + eps) * weight[c]
 *     residual_out[t][c] = RNE_bf16(h[c])                   (where it is not NULL)
 * SGEMM_NORM_BF16 rounds y once to BF16.  The 8-bit forms write, for each row
 * or group of 128 columns (the last group of a row may be shorter), the scale
 *     s = max |y| / 448   (1 where that maximum is 0; rounded up where it is
 *                          subnormal, so never 0; NaN where a y is NaN)
 * to scales[t][group], and e4m3(y / s), round-to-nearest-even, to y.  The
 * quotient may be off by about 2^-23 of itself (it is y times 1 / s, both FP32), so
 * that one this near to the middle of two e4m3 values may round to either.
 * - x, residual, residual_out: [T, D] with their row strides >= D; weight [D];
 *   y: [T, D] BF16 (2-byte aligned) or bytes; scales: [T, groups], 4-byte
 *   aligned, groups = 1 or ceil(D / 128).
 * - residual_out may be x or residual itself (same pointer and stride), and so
 *   may a BF16 y; otherwise outputs overlap no input and not each other.
 * - T >= 0 (0 rows enqueue nothing), 1 <= D <= 2^30, eps >= 0 and finite. */
typedef struct {
    const sgemm_bf16_t *x;
    const sgemm_bf16_t *residual;
    const sgemm_bf16_t *weight;
    sgemm_bf16_t *residual_out;
    void *y;
    float *scales;
    long long ldx, ldr, ldro, ldy, lds;
    long long T;
    int D;
    int form; /* SGEMM_NORM_* */
    float eps;
    unsigned flags;
} sgemm_add_rmsnorm_t;

sgemm_status_t sgemm_bf16_add_rmsnorm(const sgemm_add_rmsnorm_t *args, sgemm_stream_t stream);

/* A paged latent cache: `pages` pages of `page_size` rows of R + E BF16
 * elements each: R of the token's latent vector (what attention reads as its
 * values, and as the first part of its keys), then E rotated elements.  Row
 * `i` of page `p` starts at cache + p * page_stride + i * row_stride.  Slot
 * p * page_size + i names that row.
 *
 * For every token t < T, with (c_i, s_i) = cos_sin[positions[t]][i],
 * cos_sin[positions[t]][E/2 + i]:
 *     latent[j] = kv[t][j]                                     (weight NULL)
 *               = kv[t][j] / sqrt(mean_j kv[t][j]^2 + eps) * weight[j]     else
 *     rotated pair i of a vector v: (a c_i - b s_i, b c_i + a s_i)
 *         (a, b) = (v[2i], v[2i+1]) if interleaved, else (v[i], v[E/2 + i])
 *     cache row slots[t] = [ latent (R) | rotated kv[t][R:] (E) ]
 *     q_out[t][h] = rotated q[t][h]   (E elements), for every head h < H
 * in FP32, each element rounded once to BF16.
 * - slots[t] < 0 marks a padded token: no row is written (q_out is).  A slot
 *   past the cache writes nothing and sets bit 1 of the device error word; so
 *   does a position outside 0 .. max_position - 1 (of a token that is not
 *   padded), whose rotated elements are written as NaN.
 * - Two tokens of one call must not name the same slot.
 * - H = 0 (q and q_out NULL) leaves the queries out.  q_out may be q itself
 *   (same pointer and strides); otherwise outputs overlap no input.
 * - T >= 0, 1 <= R <= 8192, E even, 2 <= E <= 512, 0 <= H <= 65536,
 *   page_size >= 1, max_position >= 1.
 *   BF16 arrays 2-byte, cos_sin 4-byte, positions and slots 8-byte aligned. */
typedef struct {
    const sgemm_bf16_t *kv;    /* [T, R + E], row stride ldkv */
    const sgemm_bf16_t *weight; /* [R] or NULL */
    const float *cos_sin;      /* [max_position, E], row stride ldcs: cosines, then sines */
    const long long *positions; /* [T] */
    const long long *slots;    /* [T] */
    sgemm_bf16_t *cache;
    const sgemm_bf16_t *q;     /* [T, H, E], strides q_token, q_head */
    sgemm_bf16_t *q_out;       /* [T, H, E], strides qo_token, qo_head */
    long long ldkv, ldcs, row_stride, page_stride;
    long long q_token, q_head, qo_token, qo_head;
    long long T, max_position, pages;
    int page_size;
    int R, E, H;
    int interleaved;
    float eps;
    unsigned flags;
    int reserved;
} sgemm_latent_append_t;

sgemm_status_t sgemm_bf16_latent_append(const sgemm_latent_append_t *args, sgemm_stream_t stream);

/* Attention of new tokens over a paged latent cache, absorbed form: queries
 * that already carry the up-projection of the keys, values read as the first R
 * elements of each cached row, so that all heads share one row per token.
 * Sequence b has len = seq_lens[b] cached rows (its new tokens' rows among
 * them), row j in page block_table[b][j / page_size], and n new tokens, whose
 * queries are rows cu_q[b] .. cu_q[b+1]-1 of q (cu_q NULL: n = max_q for every
 * sequence, back to back).  Token i of them sees the rows j < len - n + i + 1:
 *     s_j = scale * q[t][h] . row_j                (R + E elements, FP32 sums)
 *     out[t][h] = sum_j softmax(s)_j row_j[:R]     (rounded once to BF16)
 *     lse[t][h] = log sum_j exp(s_j)               (natural; where lse is not NULL)
 * The products' weights exp(s_j - m) are rounded to BF16; sums are FP32.
 * - A token that sees no row (len = 0, or len < n) gets out = 0 and lse = -inf.
 *   What lies in rows past a sequence's end, or past what a token sees, never
 *   reaches its result, NaN and infinities included.  (A row that it sees with
 *   an infinity and a score of -inf, so with weight 0, adds NaN where the
 *   infinity is, or nothing where an earlier token of the call does not see
 *   the row.)
 * - The work is split over the SMs by the lengths, and by ceil(max_q * H / 64)
 *   CTAs for the rows of the sequence with the most new tokens.  Sequences with
 *   fewer leave some of those CTAs idle, and from 77 on (39 tokens of 128
 *   heads) the sequences' contexts are not split at all.  Put sequences with
 *   many new tokens and sequences with few into calls of their own.
 * - R: 128, 256, 384 or 512; E: a multiple of 8, 8 .. 64; 1 <= H <= 1024;
 *   1 <= max_q, the largest n of the call (a larger n in cu_q is computed up
 *   to max_q tokens only and sets bit 1 of the device error word).
 * - page_size: 8, 16, 32 or a multiple of 64.  A sequence longer than its
 *   table's width * page_size is cut there, and a table entry outside
 *   0 .. pages - 1 among the first ceil(len / page_size) reads as zeros; both
 *   set bit 1 of the device error word.
 * - q and cache are 16-byte aligned and all their strides multiples of 8; out
 *   is 4-byte aligned with even strides (else SGEMM_ERR_MISALIGNED).
 * - out, lse and the scratch overlap no input and not each other.  (Column
 *   ranges of one buffer, with its strides, are apart.)
 * - workspace: device scratch of at least sgemm_latent_attention_workspace
 *   bytes (16-byte aligned; may be NULL where that is 0).  Its contents need
 *   no preparation and do not survive the call.  Calls that may overlap on the
 *   GPU need scratch of their own.
 * - Waits inside the kernel are bounded (see sgemm_device_errors): one that
 *   runs out sets bit 0 and writes NaN outputs.  SGEMM_FLAG_TEST_STALL is
 *   accepted here, as for the GEMM calls. */
typedef struct {
    const sgemm_bf16_t *q;   /* [total_q, H, R + E], strides q_token, q_head */
    const sgemm_bf16_t *cache;
    const int *block_table;  /* [B, table_width], row stride ldt */
    const int *seq_lens;     /* [B] */
    const int *cu_q;         /* [B + 1] or NULL */
    sgemm_bf16_t *out;       /* [total_q, H, R], strides out_token, out_head */
    float *lse;              /* [total_q, H], strides lse_token, 1; or NULL */
    void *workspace;
    long long q_token, q_head, row_stride, page_stride, ldt, out_token, out_head, lse_token;
    long long pages, workspace_bytes, total_q;
    int page_size, table_width;
    int B, H, R, E, max_q;
    float scale;
    unsigned flags;
    int reserved;
} sgemm_latent_attention_t;

/* No call needs more scratch than this. */
#define SGEMM_LATENT_WORKSPACE_MAX (64LL << 20)

/* Bytes of scratch a call with these sizes needs on the current device (device
 * pointers and strides are not looked at).  0 .. SGEMM_LATENT_WORKSPACE_MAX. */
sgemm_status_t sgemm_latent_attention_workspace(const sgemm_latent_attention_t *args,
                                                long long *bytes);

sgemm_status_t sgemm_bf16_latent_attention(const sgemm_latent_attention_t *args,
                                           sgemm_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_DECODE_H */
