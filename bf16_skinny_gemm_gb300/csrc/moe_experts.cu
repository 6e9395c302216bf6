// The experts' products for a few tokens (declared in include/sgemm_layers.h):
//
//     h[t,e] = silu(x_t Wg_e^T) * (x_t Wu_e^T),   y_t = sum_e w[t,e] h[t,e] Wd_e^T
//
// What bounds it.  Every chosen expert's 3 F D weights are read once, for the few tokens that
// chose it: 2 operations a byte and token.  Up to 128 tokens the bytes bound it.
//
// So the tensor cores have time to spare, and the kernels spend it on not sorting anything: the
// products are made for ALL tokens of the call (N = 16, 32, 64 or 128 columns of tcgen05.mma, the
// weights' rows on the M side), and the first kernel's epilogue keeps what a token chose.
//
//  * Up: tiles of 8..128 gate rows and the same up rows of one expert against x (T x D), two accumulators,
//    so that gate and up of an element are in one lane of tensor memory.  The epilogue writes
//    w[t,e] silu(gate) up, BF16, as row t of expert e's block of scratch; zeros for tokens that did
//    not choose e.  (The rounding of that product to BF16, the operand type of the second one,
//    is the only one between x and y: 2^-8 of it at most, at random over F elements.)
//  * Down: with those zeros, y = sum_e H_e Wd_e^T is ONE product over k = (expert, element of F),
//    accumulated in tensor memory over all experts, in the order of their indices.  The 2, 4 or 8 CTAs
//    of a cluster take a part of that k each for 8..128 rows of y, and swap FP32 partial sums
//    through distributed shared memory (st.async), a part of the tokens each, added in rank order.
//    No atomics, no sorting: the result does not depend on timing.  (Zeros times an infinity or a NaN among the
//    weights of an expert are NaN for the tokens that did not choose it: outputs that come as NaN are worked out
//    again from the token's own experts, see chosen_only.)
//
// Both kernels stream with TMA into a ring: one warp copies the weights, one the other operand (x or H,
// from the L2 cache), one issues the MMAs, four do the epilogue.  A slot holds one or more chunks of 64
// elements of k: a copy, its wait and its products take about 600 cycles to issue whatever their size.  A ring
// takes most of the shared memory (64 tokens, 128 experts of 4096 x 1024: 493 us; with about half of it each, so that
// the second kernel's CTAs are there while the first one's run, 548 to 580; 1 token 38.1, 39.5 to 40.5).  The rows a tile has, the chunks a
// slot and the CTAs a cluster are chosen on the host, see shape_of.
//
// Measured on one GB300, both kernels, calls one after the other on changing weights:
//   64 tokens, 8 of 128 experts of 4096 x 1024 (3.2 GB)   493 us   6.4 TB/s
//   128 tokens, the same (3.2 GB)                         551 us  5.8 TB/s
//   8 tokens, 6 of 64 experts of 2048 x 1408, 29 chosen   89 us   5.7 TB/s (35 chosen: 99 us, 6.1)
//   1 token, 8 of 128 experts (201 MB)                    38 us   5.3 TB/s
//   2 tokens, 2 of 16 experts of 1024 x 512               13 us
// With few tokens the two starts are what is left: tables 0.7 us, the first slots 2 to 3 us (every SM asks for all
// of its ring at once), between the kernels 2.9 us (copying early saves 1.2), the cluster's exchange 0.9 us.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>

#include "decode_common.h"
#include "sgemm_layers.h"
#include "tc05_roles.cuh"
#include "tensor_map.h"

namespace sk {
namespace moe {

using namespace roles;

constexpr int kMostExperts = 1024;
constexpr int kMostTokens = 128;
constexpr int kMostEntries = 32;  // a token
constexpr int kThreadsExperts = 32 * 7;  // weights, MMA, 4 of epilogue, the other operand
constexpr int kRing = 16;         // slots at most
constexpr int kRingBytes = 180 * 1024;

struct ExpertParams {
    // Chunks of 64 elements of k have a dimension of their own where k is a multiple of 64, so that a box
    // holds several; else there is one, {k, rows, 1, ..}
    CUtensorMap tw;  // the weights: {64, 2F, D / 64, E}, or {64, D, F / 64, E}
    CUtensorMap tb;  // the other operand: x {64, T, D / 64, 1}, or H {64, T, F / 64, experts}
    const int *ids;
    const float *weights;
    uint16_t *h;     // H, [expert of the list][T][F]
    const uint16_t *down;  // the down matrices, as tw has them (for single outputs)
    long long dn_expert, dn_row;
    uint16_t *y;
    int *err;
    long long ldi, ldwt, ldy;
    int T, D, F, E, k;
    int rows;        // of weights (of gate and of up, or of down) a tile
    int tiles;       // of an expert (up)
    int box;         // rows of a box of the other operand
    int deep;        // chunks of k a slot
    int even;        // whether chunks have a dimension of their own
    int split;       // CTAs of a cluster (down)
    int slots, flags;
};

// A slot: `deep` chunks of weights, then as many of the other operand.
__host__ __device__ constexpr int slot_bytes(bool up, int rows, int n, int deep) { return deep * ((up ? 2 : 1) * rows + n) * 128; }
// behind the ring: an MMA reads 128 rows of weights though a tile may have fewer
__host__ __device__ constexpr int tail_bytes(int rows, int n, int deep) {
    return 128 > rows + deep * n ? (128 - rows - deep * n) * 128 : 0;
}

// y[t][d] of `own` tokens from `first` on, where it is NaN: over the experts that t chose, and no others, an element of h
// times its weight after the other, FP32.  For outputs that the shared product gives as NaN, which they are not where it
// comes from 0 x an infinity or a NaN in the weights of an expert that t did not choose.  What is NaN indeed ends the
// sum at once.  (A function by itself, after the sums: where it is not
// called 2 tokens of 16 experts take 17.6 us for 17.4 without it, 1 token of 128 experts 43.8 for 43.7, 64 490 for 490.)
__device__ __noinline__ void chosen_only(const ExpertParams &p, const unsigned *chosen, int first, int own, int d) {
    for (int t = first; t < first + own; ++t) {
        uint16_t *y = p.y + t * p.ldy + d;
        if ((*y & 0x7fff) <= 0x7f80) continue;
        const int *ids = p.ids + t * p.ldi;
        float s = 0.0f;
        for (int j = 0; j < p.k; ++j) {
            const int id = ids[j];
            bool take = id >= 0 && id < p.E;
            for (int i = 0; i < j; ++i) take = take && ids[i] != id;  // (its block of h has all of its weights)
            if (!take) continue;
            int a = __popc(chosen[id >> 5] & ((1u << (id & 31)) - 1u));
            for (int i = 0; i < id >> 5; ++i) a += __popc(chosen[i]);
            const uint4 *h = reinterpret_cast<const uint4 *>(p.h + (static_cast<long long>(a) * p.T + t) * p.F);
            const uint4 *w = reinterpret_cast<const uint4 *>(p.down + id * p.dn_expert + d * p.dn_row);
            for (int f = 0; f < p.F / 8 && s == s; ++f) {
                const uint4 x = __ldcg(h + f), v = __ldcg(w + f);
                const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, vs[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    s = fmaf(bf16_lo(xs[m]), bf16_lo(vs[m]), s);
                    s = fmaf(bf16_hi(xs[m]), bf16_hi(vs[m]), s);
                }
            }
        }
        *y = f32_to_bf16_rn(s);
    }
}

template <int N, bool UP>
__global__ void __launch_bounds__(kThreadsExperts, 1) moe_experts_kernel(const __grid_constant__ ExpertParams p) {
    constexpr int kAcc = UP ? 2 * N : N;                    // columns of a tile's accumulators
    constexpr int kTmem = UP ? 2 * kAcc : N < 32 ? 32 : N;  // (up: two tiles in turn)
    constexpr uint32_t kIdescN = (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
                                 (static_cast<uint32_t>(128 >> 4) << 24);
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t bars[2 * kRing + 2 * 2 + 2];
    __shared__ uint32_t tmem_slot;
    __shared__ int stop;
    __shared__ unsigned chosen[kMostExperts / 32];
    __shared__ int list[kMostExperts], count;
    __shared__ float wt[kMostTokens];
    __shared__ int on[kMostTokens];
    uint8_t *base = raw + ((1024u - (saddr(raw) & 1023u)) & 1023u);  // swizzled operands start on 1 KiB
    // partial sums, [rank][token][128]
    float *red = reinterpret_cast<float *>(base + p.slots * slot_bytes(UP, p.rows, N, p.deep) + tail_bytes(p.rows, N, p.deep));

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = p.slots, per_slot = slot_bytes(UP, p.rows, N, p.deep);
    const int half_bytes = p.deep * p.rows * 128, w_bytes = (UP ? 2 : 1) * half_bytes;  // gate's, all of the weights'
    const uint32_t ring = saddr(base);
    const uint32_t full = saddr(bars), empty = full + 8 * kRing, afull = empty + 8 * kRing, aempty = afull + 16,
                   fin = aempty + 16, redb = fin + 8;
    const uint32_t rank = UP ? 0u : cluster_rank();

    if (warp == 0) {
        if (lane == 0) {
            prefetch_tmap(&p.tw);
            prefetch_tmap(&p.tb);
            stop = 0;
        }
        for (int i = lane; i < 2 * S; i += 32) bar_init(i < S ? full + 8 * i : empty + 8 * (i - S), i < S ? 2 : 1);
        if (lane < 6) bar_init(afull + 8 * lane, lane == 2 || lane == 3 ? 4 : 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    for (int i = threadIdx.x; i < kMostExperts / 32; i += kThreadsExperts) chosen[i] = 0u;
    __syncthreads();
    if (!UP) cluster_arrive_relaxed();  // this CTA has started (paired with the wait before the partial sums)
    if (UP) pdl_wait();
    // the experts that some token chose, in the order of their indices
    for (int i = threadIdx.x; i < p.T * p.k; i += kThreadsExperts) {
        const int t = i / p.k, id = __ldcg(p.ids + t * p.ldi + (i - t * p.k));
        if (id >= p.E) {
            if (blockIdx.x == 0) atomicOr(p.err, kErrBadIndex);
        } else if (id >= 0) {
            atomicOr(&chosen[id >> 5], 1u << (id & 31));
        }
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&tmem_slot)), "r"(kTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    __syncthreads();
    if (warp == 2) {
        unsigned bits = chosen[lane];
        int before = __popc(bits);
        const int mine = before;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, before, off);
            if (lane >= off) before += y;
        }
        if (lane == 31) count = before;
        before -= mine;
        while (bits) {
            list[before++] = 32 * lane + __ffs(bits) - 1;
            bits &= bits - 1;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // The down kernel's CTAs may come once nothing runs that was before the up kernel: this stands behind the up
    // kernel's wait, and has to.  For they read the ids and begin to copy weights at once,
    // while up's last CTAs run, and wait for those with everything else (64 tokens of 128
    // experts 497 -> 493 us, 8 of 64 93.4 -> 90.7, 1 of 128 40.1 -> 38.9).  The caller's next kernel comes where
    // asked.  Neither comes before this CTA has its tensor memory: a kernel that takes some before it waits
    // would hold what this one, which it waits for, wants.
    if (UP || (p.flags & kFlagPdl)) pdl_launch_dependents();
    const uint32_t tmem = tmem_slot;
    const bool stall = (p.flags & kFlagTestStall) != 0;

    // this CTA's tiles, and its slots of k: of each tile (up), or of the one tile it has (down)
    const int kc = (((UP ? p.D : p.F) + 63) / 64 + p.deep - 1) / p.deep;
    const long long all = static_cast<long long>(count) * (UP ? p.tiles : kc);
    const int t0 = UP ? static_cast<int>(all * blockIdx.x / gridDim.x) : 0;
    const int t1 = UP ? static_cast<int>(all * (blockIdx.x + 1) / gridDim.x) : 1;
    const int c0 = UP ? 0 : static_cast<int>(all * rank / p.split);
    const int c1 = UP ? kc : static_cast<int>(all * (rank + 1) / p.split);
    const int d0 = UP ? 0 : static_cast<int>(blockIdx.x) / p.split * p.rows;
    if (!UP && warp != 0) pdl_wait();  // (warp 0 copies weights only)
    int issued = 0;  // slots that this warp's copies were issued for

    if (warp == 0 || warp == 6) {
        // -------------------------------------------------------------------- the copies
        const uint64_t policy = policy_of(warp == 0);
        const int step0 = p.even ? 0 : 64, step2 = p.even ? p.deep : 0;  // coordinates a slot
        int slot = 0, n = 0;
        unsigned ph = 1;
        bool ok = true;
        for (int t = t0; ok && t < t1; ++t) {
            const int a = UP ? t / p.tiles : c0 / kc;
            int slotted = a, c = UP ? 0 : c0 - a * kc;
            const int f0 = UP ? (t - a * p.tiles) * p.rows : d0;
            int e = c0 < c1 ? alike(list[slotted]) : 0;
            for (int i = c0; i < c1; ++i, ++n) {
                if (!(ok = n < S || all_wait(empty + 8 * slot, ph, &stop))) break;
                if (!stall) issued = n + 1;
                const uint32_t dst = ring + slot * per_slot, bar = full + 8 * slot;
                if (elect()) {
                    if (warp == 0) {
                        bar_expect_tx(bar, static_cast<unsigned>(w_bytes));
                        if (!stall) {
                            tma_4d(dst, &p.tw, step0 * c, f0, step2 * c, e, bar, policy);
                            if (UP) tma_4d(dst + half_bytes, &p.tw, step0 * c, p.F + f0, step2 * c, e, bar, policy);
                        }
                    } else {
                        // (a box has p.box rows, an operand N: chunks lie as close as the box has them)
                        bar_expect_tx(bar, static_cast<unsigned>(p.deep * p.box * 128));
                        if (!stall) tma_4d(dst + w_bytes, &p.tb, step0 * c, 0, step2 * c, UP ? 0 : slotted, bar, policy);
                    }
                }
                __syncwarp();
                if (++slot == S) {
                    slot = 0;
                    ph ^= 1;
                }
                if (++c == kc && !UP) {
                    c = 0;
                    if (i + 1 < c1) e = alike(list[++slotted]);
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------------ the products
        int slot = 0, n = 0;
        unsigned ph = 0;
        bool ok = true;
        const uint32_t base_d = alike(static_cast<int>(tmem));
        for (int t = t0; ok && t < t1; ++t) {
            const int i = t - t0;
            ok = i < 2 || all_wait(aempty + 8 * (i & 1), ((i >> 1) - 1) & 1, &stop);
            tc_fence_after();
            const uint32_t d = base_d + (UP ? (i & 1) * kAcc : 0);
            for (int c = c0; ok && c < c1; ++c, ++n) {
                if (!(ok = all_wait(full + 8 * slot, ph, &stop))) break;
                tc_fence_after();
                if (elect()) {
                    for (int m = 0; m < p.deep; ++m) {
                        const uint64_t a = tc05::sw128_desc(ring + slot * per_slot + m * p.rows * 128);
                        const uint64_t b = tc05::sw128_desc(ring + slot * per_slot + w_bytes + m * p.box * 128);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            mma(d, a + ((32 * kk) >> 4), b + ((32 * kk) >> 4), kIdescN, c != c0 || m != 0 || kk != 0);
                            if (UP) mma(d + N, a + ((half_bytes + 32 * kk) >> 4), b + ((32 * kk) >> 4), kIdescN, c != c0 || m != 0 || kk != 0);
                        }
                    }
                    mma_commit(empty + 8 * slot);
                    if (c + 1 == c1) mma_commit(afull + 8 * (i & 1));
                }
                __syncwarp();
                if (++slot == S) {
                    slot = 0;
                    ph ^= 1;
                }
            }
        }
        finish(fin, &stop);
    } else {
        // ------------------------------------------------------------------ the epilogue
        const int q = warp & 3, row = 32 * q + lane, tid = threadIdx.x - 64;
        const uint32_t quarter = static_cast<uint32_t>(32 * q) << 16;
        const float nan = __int_as_float(0x7fc00000);
        if constexpr (UP) {
            int last = -1, told = -1;
            bool ok = true;
            for (int t = t0; t < t1; ++t) {
                const int i = t - t0, a = t / p.tiles, f0 = (t - a * p.tiles) * p.rows;
                if (a != last) {
                    // the tokens' weights for this expert
                    const int e = list[a];
                    if (last >= 0) asm volatile("bar.sync 1, 128;" ::: "memory");  // the last one's are read
                    if (tid < p.T) {
                        float w = 0.0f;
                        int any = 0;
                        for (int j = 0; j < p.k; ++j)
                            if (p.ids[tid * p.ldi + j] == e) {
                                w += p.weights[tid * p.ldwt + j];
                                any = 1;
                            }
                        wt[tid] = w;
                        on[tid] = any;
                    }
                    last = a;
                }
                ok = ok && wait_or_stop(afull + 8 * (i & 1), (i >> 1) & 1, &stop);
                ok = __all_sync(0xffffffffu, ok);
                if (ok) tc_fence_after();
                uint16_t *out = p.h + static_cast<long long>(a) * p.T * p.F + f0 + row;
                const bool mine = row < p.rows && f0 + row < p.F;
                if (a != told) {
                    asm volatile("bar.sync 1, 128;" ::: "memory");  // the weights are there
                    told = a;
                }
#pragma unroll 1
                for (int c = 0; c < p.T; c += 8) {
                    uint32_t g[8], u[8];
                    if (ok) {
                        tmem_ld8(tmem + quarter + (i & 1) * kAcc + c, g);
                        tmem_ld8(tmem + quarter + (i & 1) * kAcc + N + c, u);
                        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
                    } else {
#pragma unroll
                        for (int m = 0; m < 8; ++m) g[m] = u[m] = __float_as_uint(nan);
                    }
                    if (mine)
#pragma unroll
                        for (int m = 0; m < 8; ++m)
                            if (c + m < p.T) {
                                const float x = __uint_as_float(g[m]);
                                const float h = x / (1.0f + expf(-x)) * __uint_as_float(u[m]) * wt[c + m];
                                out[(c + m) * p.F] = on[c + m] ? f32_to_bf16_rn(h) : 0;
                            }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(aempty + 8 * (i & 1));
            }
        } else {
            bool ok = true;
            if (c0 < c1) {
                ok = wait_or_stop(afull, 0, &stop);
                ok = __all_sync(0xffffffffu, ok);
                if (ok) tc_fence_after();
            }
            cluster_wait_acquire();  // the other CTA's shared memory and mbarriers are there
            const int each = (p.T + p.split - 1) / p.split;  // tokens a rank adds up
            const int first = static_cast<int>(rank) * each, own = max(0, min(p.T, first + each) - first);
            if (tid == 0) bar_expect_tx(redb, static_cast<unsigned>((p.split - 1) * own * p.rows * 4));
            for (int c = 0; c < N; c += 16) {
                if (c >= p.T) break;
                uint32_t v[16];
#pragma unroll
                for (int m = 0; m < 16; ++m) v[m] = ok ? 0u : __float_as_uint(nan);
                if (ok && c0 < c1) tc05::tmem_ld16(tmem + quarter + c, v);
                if (row < p.rows)
#pragma unroll
                    for (int m = 0; m < 16; ++m) {
                        const int t = c + m;
                        if (t >= p.T) continue;
                        const uint32_t to = static_cast<uint32_t>(t / each);
                        float *at = red + (rank * each + (t - to * each)) * 128 + row;
                        if (to == rank)
                            *at = __uint_as_float(v[m]);
                        else
                            st_async1(cluster_addr(saddr(at), to), __uint_as_float(v[m]), cluster_addr(redb, to));
                    }
            }
            const bool got = bar_wait_cluster(redb, 0);
            if (!got) atomicExch(&stop, 1);
            bool odd = false;
            if (row < p.rows && d0 + row < p.D)
                for (int t = 0; t < own; ++t) {
                    float s = red[t * 128 + row];
                    for (int r = 1; r < p.split; ++r) s += red[(r * each + t) * 128 + row];
                    odd |= s != s;
                    p.y[(first + t) * p.ldy + d0 + row] = f32_to_bf16_rn(got ? s : nan);
                }
            if (odd && got) chosen_only(p, chosen, first, own, d0 + row);
        }
    }
    if (!UP && (warp < 2 || warp == 6)) cluster_wait_acquire();
    __syncwarp();
    // after a stop: the copies issued have landed before the shared memory goes
    if (lane == 0 && *reinterpret_cast<volatile int *>(&stop) && (warp == 0 || warp == 6))
        for (int i = max(0, issued - S); i < issued; ++i) landed(full + 8 * (i % S), (i / S) & 1);
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 32 && stop) atomicOr(p.err, 1);
    if (!UP && stop) {
        // A CTA that gave up may have got here before the other one's stores into it were issued:
        // this barrier waits for every thread of the cluster that has not exited, then (bounded)
        // for those stores.
        cluster_arrive_release();
        cluster_wait_acquire();
        if (warp == 2 && lane == 0) (void)bar_wait_cluster(redb, 0);
    }
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmem) : "memory");
    }
}

int columns_of(int T) { return T <= 16 ? 16 : T <= 32 ? 32 : T <= 64 ? 64 : 128; }

template <bool UP>
const void *kernel_of(int n) {
    return n == 16   ? reinterpret_cast<const void *>(&moe_experts_kernel<16, UP>)
           : n == 32 ? reinterpret_cast<const void *>(&moe_experts_kernel<32, UP>)
           : n == 64 ? reinterpret_cast<const void *>(&moe_experts_kernel<64, UP>)
                     : reinterpret_cast<const void *>(&moe_experts_kernel<128, UP>);
}

// What a launch is cut into.
struct Shape {
    int rows, deep, split;
};

// How many clusters of 2, 4 and 8 CTAs the device runs at a time, a CTA an SM (a cluster lies in one part
// of the GPU, so that larger ones leave SMs over: 76, 36 and 15 here); asked once a device.
bool clusters_of(int (&most)[3]) {
    static std::atomic<unsigned> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    unsigned v = dev < 64 ? known[dev].load(std::memory_order_acquire) : 0u;
    if (!v) {
        const void *fn = reinterpret_cast<const void *>(&moe_experts_kernel<16, false>);
        if (allow_max_dynamic_smem(fn) != cudaSuccess) return false;
        for (int i = 0; i < 3; ++i) {
            cudaLaunchConfig_t cfg;
            std::memset(&cfg, 0, sizeof(cfg));
            cudaLaunchAttribute attr;
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = 2u << i;
            attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
            cfg.gridDim = dim3(1024);
            cfg.blockDim = dim3(kThreadsExperts);
            cfg.dynamicSmemBytes = kRingBytes;
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess || n < 1) return false;
            v |= static_cast<unsigned>(std::min(n, 1023)) << (10 * i);
        }
        if (dev < 64) known[dev].store(v, std::memory_order_release);
    }
    for (int i = 0; i < 3; ++i) most[i] = static_cast<int>(v >> (10 * i) & 1023);
    return true;
}

// The shape that takes the least time, counted in bytes that come from memory: a slot's
// weights, 0.6 of its other operand (from the L2 cache) and 2560 for its waits and its issue (600 cycles at
// an SM's share of the memory rate, some of them hidden); of equals the smallest cluster with the largest
// rows.  `blocks` experts; up: `of` rows each, whose products have `chunks` chunks of k, a tile an SM; down: `of` rows
// in all, whose products have `blocks` times `chunks` chunks, shared by a cluster.
// Measured (us for both products): 64 tokens, 128 experts of 4096 x 1024: tiles of 128 rows, down with 4 CTAs a
// cluster 498; up with 56 rows 517; down with 2 CTAs and 56 rows 533.  8 tokens, 64 experts of 2048 x 1408: 92
// (112 rows, 4 CTAs); up with 64 rows 95, down with 2 CTAs and 64 rows 99 and more.  1 token, 8 of 128
// experts: 38.1 (up 64 rows, down 120); up with 56 rows 38.9, and two slots.
Shape shape_of(bool up, double blocks, long long of, long long chunks, int box, int n, bool even, int sms, const int (&clusters)[3]) {
    Shape best{8, 1, 1};
    double least = -1.0;
    for (int i = 0; i < (up ? 1 : 3); ++i)
        for (int rows = 8; rows <= 128 && rows < of + 8; rows += 8) {
            const int split = up ? 1 : 2 << i;
            int deep = 1;
            while (even && deep < 4 && slot_bytes(up, rows, n, 2 * deep) <= kRingBytes / 3 && deep < chunks) deep *= 2;
            const long long row_tiles = (of + rows - 1) / rows;
            // what the memory takes for all of it, and the busiest SM, which gets 1.15 of its share where others are done
            const double tiles = up ? blocks * static_cast<double>(row_tiles) / sms : static_cast<double>(row_tiles) / clusters[i];
            const double waves = std::max(up ? tiles : static_cast<double>(row_tiles) * split / sms, std::ceil(tiles) / 1.15);
            const double slots = (up ? 1.0 : blocks) * static_cast<double>(chunks) / deep / split;
            const double cost = waves * slots * (deep * ((up ? 2 : 1) * rows * 128 + 0.6 * box * 128) + 2560.0);
            if (least < 0 || cost < 0.999 * least || (cost <= least && split == best.split)) {
                least = cost;
                best = {rows, deep, split};
            }
        }
    return best;
}

sgemm_status_t check_sizes(const sgemm_moe_experts_t &a) {
    if (a.flags & ~(kDecodeFlags | SGEMM_FLAG_TEST_STALL)) return SGEMM_ERR_INVALID_ARG;
    if (a.T < 0 || a.D < 1 || a.F < 1 || a.E < 1 || a.E > kMostExperts || a.k < 1 || a.k > kMostEntries || a.D > (1 << 20) ||
        a.F > (1 << 20))
        return SGEMM_ERR_INVALID_ARG;
    if (a.T > kMostTokens || a.D % 8 || a.F % 8) return SGEMM_ERR_UNSUPPORTED_SHAPE;
    return SGEMM_OK;
}

long long listed(const sgemm_moe_experts_t &a) { return std::min<long long>(a.E, static_cast<long long>(a.T) * a.k); }
long long scratch(const sgemm_moe_experts_t &a) { return listed(a) * a.T * a.F * 2; }

}  // namespace moe
}  // namespace sk

extern "C" sgemm_status_t sgemm_moe_experts_workspace(const sgemm_moe_experts_t *a, long long *bytes) {
    using namespace sk::moe;
    if (!a || !bytes) return SGEMM_ERR_INVALID_ARG;
    *bytes = 0;
    const sgemm_status_t st = check_sizes(*a);
    if (st == SGEMM_OK) *bytes = scratch(*a);
    return st;
}

extern "C" sgemm_status_t sgemm_bf16_moe_experts(const sgemm_moe_experts_t *a, sgemm_stream_t stream) {
    using namespace sk;
    using namespace sk::moe;
    if (!a) return SGEMM_ERR_INVALID_ARG;
    sgemm_status_t st = check_sizes(*a);
    if (st != SGEMM_OK || a->T == 0) return st;
    if (!a->x || !a->w_gate_up || !a->w_down || !a->ids || !a->weights || !a->y || a->workspace_bytes < 0) return SGEMM_ERR_INVALID_ARG;
    const long long far = kMapStride;
    if (a->ldx < a->D || a->gu_row < a->D || a->dn_row < a->F || a->ldi < a->k || a->ldwt < a->k || a->ldy < a->D ||
        (a->E > 1 && (a->gu_expert < (2LL * a->F - 1) * a->gu_row + a->D || a->dn_expert < (a->D - 1LL) * a->dn_row + a->F)) ||
        a->gu_expert < 0 || a->dn_expert < 0)
        return SGEMM_ERR_INVALID_ARG;
    if (a->ldx >= far || a->gu_row >= far || a->dn_row >= far || a->ldi >= far || a->ldwt >= far || a->ldy >= far ||
        a->gu_expert >= far || a->dn_expert >= far)
        return SGEMM_ERR_UNSUPPORTED_SHAPE;
    if (!aligned(a->x, 16) || !aligned(a->w_gate_up, 16) || !aligned(a->w_down, 16) || a->ldx % 8 || a->gu_row % 8 ||
        a->gu_expert % 8 || a->dn_row % 8 || a->dn_expert % 8 || !aligned(a->y, 2) || !aligned(a->ids, 4) ||
        !aligned(a->weights, 4) || !aligned(a->workspace, 128))
        return SGEMM_ERR_MISALIGNED;
    const long long need = scratch(*a);
    if (!a->workspace || a->workspace_bytes < need) return SGEMM_ERR_NO_WORKSPACE;
    // what is written lies apart from what is read, and the scratch from the output
    auto on_inputs = [&](const void *b, long long n) {
        return block_touches(b, n, a->x, 2LL * a->D, 2 * a->ldx, a->T) ||
               block_touches(b, n, a->w_gate_up, (a->gu_row * (2LL * a->F - 1) + a->D) * 2, 2 * a->gu_expert, a->E) ||
               block_touches(b, n, a->w_down, (a->dn_row * (a->D - 1LL) + a->F) * 2, 2 * a->dn_expert, a->E) ||
               block_touches(b, n, a->ids, 4LL * a->k, 4 * a->ldi, a->T) ||
               block_touches(b, n, a->weights, 4LL * a->k, 4 * a->ldwt, a->T);
    };
    auto in_y = [&](const void *b, long long n) { return block_touches(b, n, a->y, 2LL * a->D, 2 * a->ldy, a->T); };
    const long long wx = 2LL * a->D;
    if (rows_overlap(a->y, wx, 2 * a->ldy, a->x, wx, 2 * a->ldx, a->T) ||
        on_inputs(a->workspace, need) || in_y(a->workspace, need) ||
        in_y(a->w_gate_up, ((a->E - 1) * a->gu_expert + a->gu_row * (2LL * a->F - 1) + a->D) * 2) ||
        in_y(a->w_down, ((a->E - 1) * a->dn_expert + a->dn_row * (a->D - 1LL) + a->F) * 2) ||
        in_y(a->ids, 4 * ((a->T - 1) * a->ldi + a->k)) || in_y(a->weights, 4 * ((a->T - 1) * a->ldwt + a->k)))
        return SGEMM_ERR_INVALID_ARG;
    ExpertParams p;
    std::memset(&p, 0, sizeof(p));
    int sms = 0;
    st = device_ready(&sms, &p.err);
    if (st != SGEMM_OK) return st;
    p.ids = a->ids;
    p.weights = a->weights;
    p.h = static_cast<uint16_t *>(a->workspace);
    p.down = a->w_down;
    p.dn_expert = a->dn_expert;
    p.dn_row = a->dn_row;
    p.y = a->y;
    p.ldi = a->ldi;
    p.ldwt = a->ldwt;
    p.ldy = a->ldy;
    p.T = a->T;
    p.D = a->D;
    p.F = a->F;
    p.E = a->E;
    p.k = a->k;
    p.flags = static_cast<int>(a->flags);
    const int n = columns_of(a->T);
    p.box = std::min(n, (a->T + 7) / 8 * 8);
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    static std::atomic<unsigned long long> done[8];
    const int which = n == 16 ? 0 : n == 32 ? 1 : n == 64 ? 2 : 3;
    const long long experts = listed(*a);
    // experts that have tokens, as many as independent choices leave (what they are is known on the device only)
    const double likely = std::max(1.0, a->E * (1.0 - std::pow(1.0 - std::min(1.0, static_cast<double>(a->k) / a->E), a->T)));
    int clusters[3];
    if (!clusters_of(clusters)) return SGEMM_ERR_CUDA;
    auto ring = [&](bool up, const Shape &s) {
        p.rows = s.rows;
        p.deep = s.deep;
        p.split = s.split;
        const int bytes = slot_bytes(up, s.rows, n, s.deep);
        // beside the ring: what an MMA reads behind it, alignment, partial sums, 8 KiB of static arrays
        const int sums = up ? 0 : s.split * ((a->T + s.split - 1) / s.split) * 512;
        const int rest = tail_bytes(s.rows, n, s.deep) + 1024 + sums;
        const int room = std::min(kRingBytes, static_cast<int>(kMaxSmemOptin) - rest - 8 * 1024);
        p.slots = std::min(kRing, room / bytes);  // (2 at least: 60 KiB a slot, 64 KiB of sums at most)
        return static_cast<size_t>(p.slots) * bytes + rest;
    };
    {
        const void *fn = kernel_of<true>(n);
        p.even = a->D % 64 == 0;
        size_t smem = ring(true, shape_of(true, likely, a->F, (a->D + 63) / 64, p.box, n, p.even, sms, clusters));
        if (n >= 64) smem = std::max(smem, kAloneSmem);  // (half of the tensor memory, or all of it)
        p.tiles = (a->F + p.rows - 1) / p.rows;
        if (!map_4d(&p.tw, a->w_gate_up, a->D, 2LL * a->F, a->E, a->gu_row, a->gu_expert, p.rows, p.deep, p.even, CU_TENSOR_MAP_L2_PROMOTION_L2_256B) ||
            !map_4d(&p.tb, a->x, a->D, a->T, 1, a->ldx, a->ldx, p.box, p.deep, p.even, CU_TENSOR_MAP_L2_PROMOTION_L2_128B) ||
            !allow(fn, done[which]))
            return SGEMM_ERR_CUDA;
        const long long ctas = std::min<long long>(sms, experts * p.tiles);
        if (launch(fn, dim3(static_cast<unsigned>(ctas)), dim3(kThreadsExperts), smem, cs, &p) != cudaSuccess) return SGEMM_ERR_CUDA;
    }
    const void *fn = kernel_of<false>(n);
    p.even = a->F % 64 == 0;
    const size_t smem = ring(false, shape_of(false, likely, a->D, (a->F + 63) / 64, p.box, n, p.even, sms, clusters));
    if (!map_4d(&p.tw, a->w_down, a->F, a->D, a->E, a->dn_row, a->dn_expert, p.rows, p.deep, p.even, CU_TENSOR_MAP_L2_PROMOTION_L2_256B) ||
        !map_4d(&p.tb, a->workspace, a->F, a->T, experts, a->F, static_cast<long long>(a->T) * a->F, p.box, p.deep, p.even,
                CU_TENSOR_MAP_L2_PROMOTION_L2_128B) ||
        !allow(fn, done[4 + which]))
        return SGEMM_ERR_CUDA;
    const unsigned tiles = static_cast<unsigned>((a->D + p.rows - 1) / p.rows);
    if (launch(fn, dim3(p.split * tiles), dim3(kThreadsExperts), smem, cs, &p, p.split) != cudaSuccess) return SGEMM_ERR_CUDA;
    return SGEMM_OK;
}
