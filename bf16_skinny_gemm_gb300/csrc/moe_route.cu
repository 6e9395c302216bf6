// The router of a mixture of experts for a few tokens (declared in include/sgemm_layers.h):
// logits = x W^T, the k best experts of every token, and their weights.
//
// What bounds it.  W is E x D (128 x 4096: 1 MiB), the products a few MFLOP: latency.  One launch
// is to do all of it, and the selection needs a token's logits in one place.  So a thread-block
// cluster of 8 CTAs takes 8 tokens: each CTA computes the logits of every eighth block of 16
// experts and sends them to the CTA that selects for the token (distributed shared memory), one
// token a CTA.  With more than 8 tokens each cluster reads W again, from the L2 cache.
//
// The products: mma.sync m16n8k16 with 16 experts as A's rows and the 8 tokens as B's columns.
// The order of k within an operand is free as long as both have the same, so a lane loads 16
// consecutive bytes of its row, 8 elements, which are its share of two MMAs: fragments come
// straight from memory, without shared memory in between.  tcgen05 would want the operands there,
// which costs more than it gives for 16 x 8 outputs a CTA.  A CTA's 16 warps split D, and their sums
// are added in the warps' order (FP32).
//
// Measured on one GB300, calls one after the other: 128 experts of 4096, 8 chosen: 1 token 5.6 us, 64 tokens
// 5.9; 64 experts of 2048, 8 tokens 4.9; 16 of 1024, 2 tokens 3.9.  A launch and one chain: loads, the
// sum over warps, the cluster's barrier, k rounds of the choice.  More than 128 experts are further passes over blocks of
// them, one after the other, and more than 256 take the choice over 32 a lane: 256 experts of 4096 8.5 us (64 tokens
// 8.7), 288 10.5 (12.0), 1024 20.3 (23.6).
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "decode_common.h"
#include "sgemm_layers.h"
#include "skinny_ldg.cuh"

namespace sk {
namespace moe {

constexpr int kTokens = 8;      // tokens a cluster (columns of the MMA)
constexpr int kCtas = 8;        // CTAs a cluster
constexpr int kExperts = 16;    // experts a block (rows of the MMA)
constexpr int kMaxExperts = 1024;
constexpr int kWarps = 16;
constexpr int kThreadsRoute = 32 * kWarps;
constexpr int kBatch = 8;       // 32-element blocks of k whose loads are in flight

struct RouteParams {
    const uint16_t *x, *w;
    const float *bias;
    int *ids;
    float *weights;
    long long ldx, ldw, ldi, ldwt;
    long long T;
    int D, E, k, scoring, renormalize, flags;
    float scale;
};

// A float's bits in an order that is that of the numbers; NaN before all others, and above 0,
// which stands for what was taken.
__device__ __forceinline__ unsigned rank_of(float v) {
    const unsigned b = __float_as_uint(v + 0.0f);  // (-0 is 0)
    if (v != v) return 1u;
    return b & 0x80000000u ? ~b : b | 0x80000000u;  // -inf: 0x007fffff
}

// EACH: experts a lane of the selecting warp holds (4 for up to 128 experts, 8, or 32; a token's k rounds over 32 of
// them: 1 token of 128 experts 6.6 us, 5.6 so)
template <int EACH>
__global__ void __launch_bounds__(kThreadsRoute) moe_route_kernel(const __grid_constant__ RouteParams p) {
    __shared__ float part[kWarps][kExperts][kTokens];
    __shared__ float logits[32 * EACH];  // of the token this CTA selects for
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_rank());
    const long long t0 = static_cast<long long>(blockIdx.x / kCtas) * kTokens;
    if (p.flags & kFlagPdl) pdl_launch_dependents();
    pdl_wait();

    // a warp's blocks of 32 elements of k
    const int blocks = (p.D + 31) / 32;
    const int per = (blocks + kWarps - 1) / kWarps;
    const int b0 = min(blocks, warp * per), b1 = min(blocks, b0 + per);
    const int row = lane >> 2, part_k = 8 * (lane & 3);
    const long long t = t0 + row;
    const uint16_t *xr = p.x + (t < p.T ? t : 0) * p.ldx + part_k;
    const bool have_x = t < p.T;
    bool first = true;
    for (int e0 = rank * kExperts; e0 < p.E; e0 += kCtas * kExperts) {
        const int ea = e0 + row, eb = ea + 8;
        const uint16_t *wa = p.w + (ea < p.E ? ea : 0) * p.ldw + part_k;
        const uint16_t *wb = p.w + (eb < p.E ? eb : 0) * p.ldw + part_k;
        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int b = b0; b < b1; b += kBatch) {
            uint4 a[kBatch], c[kBatch], x[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int at = 32 * (b + i);
                const bool in = b + i < b1 && at + part_k < p.D;
                a[i] = c[i] = x[i] = make_uint4(0u, 0u, 0u, 0u);
                if (in && ea < p.E) a[i] = __ldg(reinterpret_cast<const uint4 *>(wa + at));
                if (in && eb < p.E) c[i] = __ldg(reinterpret_cast<const uint4 *>(wb + at));
                if (in && have_x) x[i] = __ldg(reinterpret_cast<const uint4 *>(xr + at));
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const uint32_t lo[4] = {a[i].x, c[i].x, a[i].y, c[i].y}, hi[4] = {a[i].z, c[i].z, a[i].w, c[i].w};
                mma_bf16_16816(d, lo, x[i].x, x[i].y);
                mma_bf16_16816(d, hi, x[i].z, x[i].w);
            }
        }
        *reinterpret_cast<float2 *>(&part[warp][row][2 * (lane & 3)]) = make_float2(d[0], d[1]);
        *reinterpret_cast<float2 *>(&part[warp][row + 8][2 * (lane & 3)]) = make_float2(d[2], d[3]);
        if (first) {
            // every CTA of the cluster has started before its shared memory is written to
            cluster_arrive_relaxed();
            cluster_wait_acquire();
            first = false;
        }
        __syncthreads();
        if (threadIdx.x < kExperts * kTokens) {
            const int e = threadIdx.x >> 3, m = threadIdx.x & 7;
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) s += part[w][e][m];
            if (e0 + e < p.E) {
                const uint32_t to = cluster_addr(saddr(&logits[e0 + e]), static_cast<uint32_t>(m));
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(s) : "memory");
            }
        }
        __syncthreads();
    }
    if (first) {
        cluster_arrive_relaxed();
        cluster_wait_acquire();
    }
    cluster_arrive_release();
    cluster_wait_acquire();
    if (warp != 0 || t0 + rank >= p.T) return;

    // one warp selects; lane l has experts l, l + 32, ...
    const long long tok = t0 + rank;
    const float inf = __int_as_float(0x7f800000);
    unsigned key[EACH];
    float top = -inf, sum = 0.0f;
    if (p.scoring == SGEMM_ROUTE_SOFTMAX) {
        for (int e = lane; e < p.E; e += 32) top = fmaxf(top, logits[e]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        for (int e = lane; e < p.E; e += 32) sum += expf(logits[e] - top);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    auto score = [&](float v) { return p.scoring == SGEMM_ROUTE_SOFTMAX ? expf(v - top) / sum : 1.0f / (1.0f + expf(-v)); };
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int e = lane + 32 * i;
        key[i] = 0u;
        if (e < p.E) key[i] = rank_of(p.bias ? score(logits[e]) + p.bias[e] : logits[e]);
    }
    float mine = 0.0f, total = 0.0f;  // lane j: the j-th choice's score
    int id = 0;
    for (int j = 0; j < p.k; ++j) {
        unsigned best = 0u;
        int at = 0;
#pragma unroll
        for (int i = 0; i < EACH; ++i)
            if (key[i] > best) {  // the lower index of equal ones
                best = key[i];
                at = i;
            }
        const unsigned most = __reduce_max_sync(0xffffffffu, best);
        const int e = static_cast<int>(__reduce_min_sync(0xffffffffu, best == most ? static_cast<unsigned>(lane + 32 * at) : 0xffffffffu));
#pragma unroll
        for (int i = 0; i < EACH; ++i)
            if (e == lane + 32 * i) key[i] = 0u;
        const float s = score(logits[e]);
        total += s;
        if (lane == j) {
            mine = s;
            id = e;
        }
    }
    if (lane < p.k) {
        p.ids[tok * p.ldi + lane] = id;
        p.weights[tok * p.ldwt + lane] = (p.renormalize ? mine / total : mine) * p.scale;
    }
}

}  // namespace moe
}  // namespace sk

extern "C" sgemm_status_t sgemm_bf16_moe_route(const sgemm_moe_route_t *a, sgemm_stream_t stream) {
    using namespace sk;
    using namespace sk::moe;
    if (!a || !valid_flags(a->flags)) return SGEMM_ERR_INVALID_ARG;
    if (a->T < 0 || a->T > (1 << 20) || a->E < 1 || a->E > kMaxExperts || a->k < 1 || a->k > 16 || a->k > a->E || a->D < 1 ||
        a->D > (1 << 20) || (a->scoring != SGEMM_ROUTE_SOFTMAX && a->scoring != SGEMM_ROUTE_SIGMOID) ||
        (a->renormalize != 0 && a->renormalize != 1) || !std::isfinite(a->scale))
        return SGEMM_ERR_INVALID_ARG;
    if (a->D % 8) return SGEMM_ERR_UNSUPPORTED_SHAPE;
    if (a->T == 0) return SGEMM_OK;
    const long long far = 1LL << 40;  // strides that products with row numbers keep in 64 bits
    if (!a->x || !a->w || !a->ids || !a->weights || a->ldx < a->D || a->ldw < a->D || a->ldi < a->k || a->ldwt < a->k ||
        a->ldx >= far || a->ldw >= far || a->ldi >= far || a->ldwt >= far)
        return SGEMM_ERR_INVALID_ARG;
    if (!aligned(a->x, 16) || !aligned(a->w, 16) || a->ldx % 8 || a->ldw % 8 || !aligned(a->bias, 4) || !aligned(a->ids, 4) ||
        !aligned(a->weights, 4))
        return SGEMM_ERR_MISALIGNED;
    const long long wx = 2LL * a->D;
    auto reads = [&](const void *o, long long ld) {
        return rows_overlap(o, 4LL * a->k, 4 * ld, a->x, wx, 2 * a->ldx, a->T) ||
               block_touches(o, (a->T - 1) * 4 * ld + 4LL * a->k, a->w, wx, 2 * a->ldw, a->E) ||
               block_touches(a->bias, a->bias ? 4LL * a->E : 0, o, 4LL * a->k, 4 * ld, a->T);
    };
    if (reads(a->ids, a->ldi) || reads(a->weights, a->ldwt) ||
        rows_overlap(a->ids, 4LL * a->k, 4 * a->ldi, a->weights, 4LL * a->k, 4 * a->ldwt, a->T))
        return SGEMM_ERR_INVALID_ARG;
    int sms = 0, *err = nullptr;
    const sgemm_status_t st = device_ready(&sms, &err);
    if (st != SGEMM_OK) return st;
    RouteParams p;
    std::memset(&p, 0, sizeof(p));
    p.x = a->x;
    p.w = a->w;
    p.bias = a->bias;
    p.ids = a->ids;
    p.weights = a->weights;
    p.ldx = a->ldx;
    p.ldw = a->ldw;
    p.ldi = a->ldi;
    p.ldwt = a->ldwt;
    p.T = a->T;
    p.D = a->D;
    p.E = a->E;
    p.k = a->k;
    p.scoring = a->scoring;
    p.renormalize = a->renormalize;
    p.scale = a->scale;
    p.flags = static_cast<int>(a->flags);
    const unsigned clusters = static_cast<unsigned>((a->T + kTokens - 1) / kTokens);
    const void *fn = a->E <= 128   ? reinterpret_cast<const void *>(&moe_route_kernel<4>)
                     : a->E <= 256 ? reinterpret_cast<const void *>(&moe_route_kernel<8>)
                                   : reinterpret_cast<const void *>(&moe_route_kernel<32>);
    if (launch(fn, dim3(clusters * kCtas), dim3(kThreadsRoute), 0,
               reinterpret_cast<cudaStream_t>(stream), &p, kCtas) != cudaSuccess)
        return SGEMM_ERR_CUDA;
    return SGEMM_OK;
}
