// Checks that the two forms of linear attention (linear_step.cu, linear_attention.cu) share.
#pragma once

#include "decode_common.h"
#include "sgemm_layers.h"

namespace sk {
namespace linear {

// The arrays of a call: n tokens, `pool` states.
struct LinearView {
    const uint16_t *q, *k, *v;
    const float *g;
    const float *state;
    const uint16_t *out;
    long long q_token, q_head, k_token, k_head, v_token, v_head, g_token, g_head, s_slot, s_head, o_token, o_head, n, pool;
    int Hk, Hv, Dk, Dv;
};

// Whether no two of the n x heads rows of `w` elements share one.
inline bool rows_apart(long long n, long long tok, int heads, long long head, long long w) {
    const long long none = 1LL << 62;
    if (n <= 1) tok = none;
    if (heads == 1) head = none;
    const long long lo = tok < head ? tok : head, hi = tok < head ? head : tok;
    if (lo == none) return true;
    const long long inner = tok < head ? n : heads;
    return lo >= w && (hi == none || hi >= (inner - 1) * lo + w);
}

// Whether `bytes` bytes at b lie in what a call writes.
inline bool linear_touches(const LinearView &a, const void *b, long long bytes) {
    if (!b || bytes < 1) return false;
    const Heads out{a.out, 2LL * a.Dv, 2 * a.o_token, 2 * a.o_head};
    const long long head = 4LL * a.Dk * a.Dv;
    return rows_overlap(b, bytes, 0, a.out, out.extent(a.n, a.Hv), 0, 1) ||
           (a.pool > 0 && block_touches(b, bytes, a.state, (a.Hv - 1) * 4 * a.s_head + head, 4 * a.s_slot, a.pool));
}

// Strides, alignment and overlap (the sizes are checked before).
inline sgemm_status_t check_linear(const LinearView &a) {
    const long long far = 1LL << 29;  // strides: their products with 2^31 rows, in bytes, stay in 64 bits
    const long long strides[] = {a.q_token, a.q_head, a.k_token, a.k_head, a.v_token, a.v_head, a.g_token, a.g_head,
                                 a.s_slot, a.s_head, a.o_token, a.o_head};
    for (long long s : strides)
        if (s < 0 || s >= far) return SGEMM_ERR_INVALID_ARG;
    const long long each = static_cast<long long>(a.Dk) * a.Dv;
    if (!rows_apart(a.n, a.o_token, a.Hv, a.o_head, a.Dv) || !rows_apart(a.pool, a.s_slot, a.Hv, a.s_head, each))
        return SGEMM_ERR_INVALID_ARG;
    if (!aligned(a.q, 16) || !aligned(a.k, 16) || !aligned(a.v, 16) || a.q_token % 8 || a.q_head % 8 || a.k_token % 8 ||
        a.k_head % 8 || a.v_token % 8 || a.v_head % 8 || !aligned(a.g, 4) || !aligned(a.state, 16) || a.s_slot % 4 ||
        a.s_head % 4 || !aligned(a.out, 4) || a.o_token % 2 || a.o_head % 2)
        return SGEMM_ERR_MISALIGNED;
    const Heads out{a.out, 2LL * a.Dv, 2 * a.o_token, 2 * a.o_head};
    const Heads q{a.q, 2LL * a.Dk, 2 * a.q_token, 2 * a.q_head}, k{a.k, 2LL * a.Dk, 2 * a.k_token, 2 * a.k_head};
    const Heads v{a.v, 2LL * a.Dv, 2 * a.v_token, 2 * a.v_head}, g{a.g, 4, 4 * a.g_token, 4 * a.g_head};
    // out against the inputs: ranges of one buffer's rows are apart
    auto row = [&](const Heads &x, int heads) { return x.extent(1, heads); };
    if (rows_overlap(a.out, row(out, a.Hv), out.tok, a.q, row(q, a.Hk), q.tok, a.n) ||
        rows_overlap(a.out, row(out, a.Hv), out.tok, a.k, row(k, a.Hk), k.tok, a.n) ||
        (heads_overlap(out, v, a.n, a.Hv) && rows_overlap(a.out, row(out, a.Hv), out.tok, a.v, row(v, a.Hv), v.tok, a.n)) ||
        rows_overlap(a.out, out.extent(a.n, a.Hv), 0, a.g, g.extent(a.n, a.Hv), 0, 1))
        return SGEMM_ERR_INVALID_ARG;
    // the states against everything
    if (a.pool > 0) {
        const long long head = 4 * each, slot = (a.Hv - 1) * 4 * a.s_head + head;
        auto in_states = [&](const Heads &x, int heads) {
            return block_touches(x.p, x.extent(a.n, heads), a.state, slot, 4 * a.s_slot, a.pool);
        };
        if (in_states(q, a.Hk) || in_states(k, a.Hk) || in_states(v, a.Hv) || in_states(g, a.Hv) || in_states(out, a.Hv))
            return SGEMM_ERR_INVALID_ARG;
    }
    return SGEMM_OK;
}

}  // namespace linear
}  // namespace sk
