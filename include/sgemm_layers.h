/*
 * sgemm_layers.h -- C ABI of the operators that make whole layers of a decode
 * or verification step (GB300, sm_103a; the same library as sgemm_skinny.h):
 *
 *   sgemm_bf16_moe_route              a router's experts and weights for a few tokens
 *   sgemm_bf16_moe_experts            the chosen experts' products
 *   sgemm_bf16_latent_tree_attention  latent attention for a tree of drafted tokens
 *   sgemm_bf16_linear_step            linear attention with decays, one token a sequence
 *   sgemm_bf16_linear_attention       the same for prompts, in chunks
 *
 * The conventions are those of sgemm_decode.h: device pointers owned by the
 * caller on the current device, raw BF16 bits, asynchronous work on `stream`,
 * argument checks on the host before anything is enqueued, a status in return,
 * no allocation and no synchronization, launches as programmatic dependents
 * that wait for the kernel before them, `flags` 0 or SGEMM_FLAG_PDL (and
 * SGEMM_FLAG_WEIGHTS_READONLY, which changes nothing), the same inputs give
 * the same bits.  Strides are in elements.  The argument structures are HOST
 * memory, read during the call only; clear them (memset) before filling them in.
 * Outputs and scratch overlap no input and not each other, but for what is said
 * to be updated in place.
 */
#ifndef SGEMM_LAYERS_H
#define SGEMM_LAYERS_H

#include "sgemm_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------ mixture of experts */

/* How sgemm_bf16_moe_route turns logits into scores. */
enum {
    SGEMM_ROUTE_SOFTMAX = 0, /* over all experts */
    SGEMM_ROUTE_SIGMOID = 1  /* of each by itself */
};

/* For every token t < T: logits[e] = x[t] . w[e] (FP32 sums), score = softmax or
 * sigmoid of them.  The k experts of the largest score[e] + bias[e] (bias NULL:
 * score[e]) are chosen, the largest first, equal ones by the lower index (without
 * a bias by the logits, whose order is the scores'), and
 *     ids[t][j] = the j-th expert
 *     weights[t][j] = score / (sum of the k chosen scores, if renormalize) * scale
 * - A NaN score (or score + bias) is chosen after all others.
 * - A sum of 0 of the chosen scores gives weights of NaN, as 0 / 0 does.
 * - 0 <= T <= 2^20, 1 <= k <= 16, k <= E <= 1024, D a multiple of 8 and at most 2^20.
 * - x and w are 16-byte aligned, their row strides multiples of 8. */
typedef struct {
    const sgemm_bf16_t *x;    /* [T, D], row stride ldx */
    const sgemm_bf16_t *w;    /* [E, D], row stride ldw */
    const float *bias;        /* [E] or NULL */
    int *ids;                 /* [T, k], row stride ldi */
    float *weights;           /* [T, k], row stride ldwt */
    long long ldx, ldw, ldi, ldwt;
    long long T;
    int D, E, k;
    int scoring;              /* SGEMM_ROUTE_* */
    int renormalize;
    float scale;
    unsigned flags;
    int reserved;
} sgemm_moe_route_t;

sgemm_status_t sgemm_bf16_moe_route(const sgemm_moe_route_t *args, sgemm_stream_t stream);

/* For every token t < T, over its entries j < k with ids[t][j] = e >= 0:
 *     h = silu(x[t] . w_gate_up[e][:F]) * (x[t] . w_gate_up[e][F:])      (F elements)
 *     y[t] = sum_j weights[t][j] * (h . w_down[e])      rounded once to BF16
 * silu(v) = v / (1 + exp(-v)).  weights * h is rounded to BF16, as the operand of
 * the second product; sums are FP32.  Only experts that some entry names are read,
 * each element once (by each of the GPU's SMs at most).
 * - ids[t][j] < 0: an entry that is not used (a padded token, an expert that is
 *   elsewhere).  A token without any gets zeros.  An expert that a token names
 *   twice counts with the sum of its weights.  ids past E - 1 are not used and
 *   set bit 1 of the device error word.
 * - Experts that every token takes are entries like the others: ids[t][j] of them
 *   with weight 1.
 * - An infinity or a NaN in x[t] reaches y[t] only, one in the weights of an expert
 *   the tokens that chose it.  (The tokens share the products: outputs that come as
 *   NaN are summed again one by one, which takes longer.)
 * - 0 <= T <= 128; D and F multiples of 8, at most 2^20; 1 <= E <= 1024, 1 <= k <= 32;
 *   D and F at least 8.
 * - x, w_gate_up, w_down are 16-byte aligned, all their strides multiples of 8;
 *   y, ids and weights are aligned to their elements.
 * - workspace: device scratch of at least sgemm_moe_experts_workspace bytes
 *   (128-byte aligned).  Its contents need no preparation and do not survive the
 *   call.  Calls that may overlap on the GPU need scratch of their own.
 * - Waits inside the kernels are bounded: one that runs out sets bit 0 of the
 *   device error word, and outputs that miss something are NaN.
 *   SGEMM_FLAG_TEST_STALL is accepted. */
typedef struct {
    const sgemm_bf16_t *x;          /* [T, D], row stride ldx */
    const sgemm_bf16_t *w_gate_up;  /* [E, 2F, D], strides gu_expert, gu_row */
    const sgemm_bf16_t *w_down;     /* [E, D, F], strides dn_expert, dn_row */
    const int *ids;                 /* [T, k], row stride ldi */
    const float *weights;           /* [T, k], row stride ldwt */
    sgemm_bf16_t *y;                /* [T, D], row stride ldy */
    void *workspace;
    long long ldx, gu_expert, gu_row, dn_expert, dn_row, ldi, ldwt, ldy;
    long long workspace_bytes;
    int T, D, F, E, k;
    unsigned flags;
} sgemm_moe_experts_t;

/* Bytes of scratch a call with these sizes needs (pointers and strides are not looked at). */
sgemm_status_t sgemm_moe_experts_workspace(const sgemm_moe_experts_t *args, long long *bytes);

sgemm_status_t sgemm_bf16_moe_experts(const sgemm_moe_experts_t *args, sgemm_stream_t stream);

/* -------------------------------------------------- attention for drafted tokens */

/* sgemm_bf16_latent_attention where a sequence's new tokens are a tree (or any
 * other set) of drafts: token i of its n sees all rows j < len - n, and the row
 * len - n + j of new token j where bit j of its mask is set,
 *     bit j: tree[t * ld_tree + j / 64] >> (j % 64) & 1        (t: the token's row of q)
 * so that a token that is to see itself has its own bit.  Bits of tokens that the
 * sequence does not have, and of rows before the cache's first, change nothing.
 * All else is as sgemm_bf16_latent_attention has it, but that the work is split evenly
 * whatever numbers of new tokens the sequences have, and that the scratch is
 * sgemm_latent_tree_attention_workspace bytes.  (What a new token's row holds, infinities
 * and NaN included, never reaches a token that does not see it.  A row that a token
 * sees with an infinity and a score of -inf, so with weight 0, adds nothing.)
 * - (table_width * page_size / 64 + 3) * (total_q * H / 16 + B) < 2^30.  Where cu_q falls and rises again over the
 *   same rows of q, so that its sequences come to 2^30 or more of what is bounded so (64 cached rows for
 *   16, 32 or 64 rows of q), nothing is computed and bit 1 of the device error word is set.
 * - words >= 1: 64-bit words a token, max_q <= 64 * words; words <= ld_tree < 2^28;
 *   tree is 8-byte aligned and overlaps no output. */
sgemm_status_t sgemm_bf16_latent_tree_attention(const sgemm_latent_attention_t *args,
                                                const long long *tree, long long ld_tree, int words,
                                                sgemm_stream_t stream);

/* 0 .. SGEMM_LATENT_WORKSPACE_MAX, as for the attention without drafted tokens. */
sgemm_status_t sgemm_latent_tree_attention_workspace(const sgemm_latent_attention_t *args, long long *bytes);

/* ------------------------------------------- linear attention, a decay for each head */

/* One token of each of B sequences.  Value head h reads key head h / (Hv / Hk).
 * With S = state[slots[b]][h] (Dk x Dv, FP32), updated in place:
 *     S[i][j] = exp(g[b][h]) S[i][j] + k[b][h'][i] v[b][h][j]
 *     out[b][h][j] = scale * sum_i q[b][h'][i] S[i][j]        (rounded once to BF16)
 * - slots[b] < 0 marks a padded sequence: no state is touched, its out is 0.  A
 *   slot past the pool is treated the same and sets bit 1 of the device error word.
 * - Two sequences of one call must not name the same slot.
 * - g is a logarithm: 0 keeps the state, -inf drops it (its finite part; an infinity
 *   or a NaN in a dropped state gives NaN).
 * - Dk and Dv: 64 or 128; Hv a multiple of Hk, Hv <= 1024; B < 2^28 / Hv; less than 2^31
 *   slots; strides below 2^29.
 * - q, k, v are 16-byte aligned with strides that are multiples of 8; out is 4-byte
 *   aligned with even strides; state is 16-byte aligned with strides that are
 *   multiples of 4 (each head's Dk x Dv is dense).  g's strides may be 0. */
typedef struct {
    const sgemm_bf16_t *q;   /* [B, Hk, Dk], strides q_token, q_head */
    const sgemm_bf16_t *k;   /* [B, Hk, Dk], strides k_token, k_head */
    const sgemm_bf16_t *v;   /* [B, Hv, Dv], strides v_token, v_head */
    const float *g;          /* [B, Hv], strides g_token, g_head */
    float *state;            /* [slots, Hv, Dk, Dv], strides s_slot, s_head */
    const long long *slots;  /* [B] */
    sgemm_bf16_t *out;       /* [B, Hv, Dv], strides o_token, o_head */
    long long q_token, q_head, k_token, k_head, v_token, v_head, g_token, g_head;
    long long s_slot, s_head, o_token, o_head;
    long long B, pool;       /* sequences, slots of the pool */
    int Hk, Hv, Dk, Dv;
    float scale;
    unsigned flags;
} sgemm_linear_step_t;

sgemm_status_t sgemm_bf16_linear_step(const sgemm_linear_step_t *args, sgemm_stream_t stream);

/* The same recurrence over whole sequences: sequence b has the tokens (rows of q, k,
 * v, g, out) cu[b] .. cu[b+1]-1, starts from state[slots[b]] (from zeros where
 * fresh[b] is not 0, whatever the slot holds) and leaves its last state there.
 * Computed in chunks of 64 tokens, with G_i = sum of g over the chunk's tokens up to i:
 *     o_i = scale (exp(G_i) q_i^T S + sum_{j <= i} exp(G_i - G_j) (q_i . k_j) v_j)
 *     S'  = exp(G) S + sum_j exp(G - G_j) k_j v_j^T
 * Sums and states are FP32.  Rounded to BF16, as operands of products: the weights
 * exp(G_i - G_j) (q_i . k_j), and S in the outputs; decayed keys are three BF16 values
 * each, whose sum is the FP32 product, so that the states keep FP32's accuracy.
 * - slots[b] < 0: starts from zeros, and the last state is not kept.  A slot past
 *   the pool is treated the same and sets bit 1 of the device error word.
 * - A sequence without tokens leaves its slot as it is (zeros where fresh).
 * - cu rises from 0 or more to at most N; where it does not, the sequence is taken
 *   as one without tokens whose slot stays as it is, and bit 1 of the error word is
 *   set.  Rows of out before cu[0] and from cu[B] on are left as they are.  Where cu
 *   falls and rises again over the same tokens, the rows that two sequences share have
 *   the values of either; where the sequences come to 2^30 or more chunks of all heads
 *   so, nothing is computed and bit 1 of the error word is set.
 * - Two sequences of one call must not name the same slot.
 * - Sequences are left whole where that takes less time than cutting them, in calls of up
 *   to 256 sequences and 64 pairs of a sequence and a head for each SM; larger
 *   calls are always cut, which shows as a step in time of about a tenth.
 * - g <= 0 is what this is made for.  exp(g) may exceed 1 as long as no exp(G_i - G_j)
 *   overflows; g = -inf drops what came before.  An infinity or a NaN in q reaches its
 *   token only, in k or g its sequence and head from its token on, in v the same for its
 *   element (as an infinity or NaN).
 * - Sizes, alignments and strides as for sgemm_bf16_linear_step; N < 2^31 / Hv; strides
 *   of q, k and v along dimensions of more than one element are at least 8.
 * - SGEMM_FLAG_TEST_STALL is accepted.
 * - workspace: device scratch of at least sgemm_linear_attention_workspace bytes
 *   (16-byte aligned; may be NULL where that is 0), as for the other operators.
 * - Waits inside the kernels are bounded, as in sgemm_bf16_moe_experts. */
typedef struct {
    const sgemm_bf16_t *q;   /* [N, Hk, Dk], strides q_token, q_head */
    const sgemm_bf16_t *k;   /* [N, Hk, Dk], strides k_token, k_head */
    const sgemm_bf16_t *v;   /* [N, Hv, Dv], strides v_token, v_head */
    const float *g;          /* [N, Hv], strides g_token, g_head */
    float *state;            /* [slots, Hv, Dk, Dv], strides s_slot, s_head */
    const long long *slots;  /* [B] */
    const int *cu;           /* [B + 1] */
    const int *fresh;        /* [B] or NULL: none is */
    sgemm_bf16_t *out;       /* [N, Hv, Dv], strides o_token, o_head */
    void *workspace;
    long long q_token, q_head, k_token, k_head, v_token, v_head, g_token, g_head;
    long long s_slot, s_head, o_token, o_head;
    long long N, B, pool, workspace_bytes;
    int Hk, Hv, Dk, Dv;
    float scale;
    unsigned flags;
} sgemm_linear_attention_t;

sgemm_status_t sgemm_linear_attention_workspace(const sgemm_linear_attention_t *args, long long *bytes);

sgemm_status_t sgemm_bf16_linear_attention(const sgemm_linear_attention_t *args, sgemm_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_LAYERS_H */
