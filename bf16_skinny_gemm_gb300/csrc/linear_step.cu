// Linear attention with a decay for each head, one token a sequence (declared in
// include/sgemm_layers.h):
//
//     S = exp(g) S + k v^T,   out = scale q^T S
//
// What bounds it.  A head's state (128 x 128 FP32: 64 KiB) is read and written once for 4 operations
// an element: memory.  So a CTA's threads load all of their part of the state before anything
// else happens, 16 bytes a load, and hold it in registers until it is written back.
//
// A CTA takes 32 columns of one head's state (128 bytes of its rows; a whole head a CTA took 2.6 us in place of 1.8 for
// one sequence of 32 heads, 17.2 for 16.2 for 24 of them, 78.9 for 77.6 for 128).  A thread has four columns of every
// 32nd row; the sums over the rows are joined by shuffles within a warp and in shared memory between warps, in a
// fixed order.
//
// Measured on one GB300: 128 sequences, 15 of them padded, 32 heads of 128 x 128 (477 MB) 70.2 us, the rate of a copy;
// one sequence of 32 heads 1.8 us in a graph, 2.8 as calls one after the other.
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "linear_common.h"
#include "skinny_ldg.cuh"

namespace sk {
namespace linear {

constexpr int kStepThreads = 256;

struct StepParams {
    const uint16_t *q, *k, *v;
    const float *g;
    float *state;
    const long long *slots;
    uint16_t *out;
    int *err;
    long long q_token, q_head, k_token, k_head, v_token, v_head, g_token, g_head, s_slot, s_head, o_token, o_head, pool;
    int Hv, share;  // heads, value heads a key head
    int flags;
    float scale;
};

template <int DK, int DV>
__global__ void __launch_bounds__(kStepThreads) linear_step_kernel(const __grid_constant__ StepParams p) {
    constexpr int W = 32, kSlices = DV / W;
    constexpr int kLanes = W / 4, kRows = kStepThreads / kLanes, kEach = DK / kRows;  // lanes a row, rows at a time, rows a thread
    constexpr int kWarps = kStepThreads / 32;
    __shared__ float qs[DK], ks[DK];
    __shared__ __align__(16) float part[kWarps][W];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int slice = static_cast<int>(blockIdx.x) % kSlices, item = static_cast<int>(blockIdx.x) / kSlices;
    const int b = item / p.Hv, h = item - b * p.Hv, hk = h / p.share;
    const int col = slice * W + 4 * (tid % kLanes), row0 = tid / kLanes;
    if (p.flags & kFlagPdl) pdl_launch_dependents();
    pdl_wait();
    const long long slot = p.slots[b];
    uint16_t *out = p.out + b * p.o_token + h * p.o_head + slice * W;
    if (slot < 0 || slot >= p.pool) {
        if (slot >= p.pool && tid == 0 && h == 0 && slice == 0) atomicOr(p.err, kErrBadIndex);
        if (tid < W) out[tid] = 0;
        return;
    }
    float *s = p.state + slot * p.s_slot + h * p.s_head + static_cast<long long>(row0) * DV + col;
    float4 x[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) x[i] = __ldcs(reinterpret_cast<const float4 *>(s + i * kRows * DV));
    const float g = p.g[b * p.g_token + h * p.g_head];
    const uint2 vw = *reinterpret_cast<const uint2 *>(p.v + b * p.v_token + h * p.v_head + col);
    for (int i = tid; i < DK / 2; i += kStepThreads) {
        const uint32_t qw = *reinterpret_cast<const uint32_t *>(p.q + b * p.q_token + hk * p.q_head + 2 * i);
        const uint32_t kw = *reinterpret_cast<const uint32_t *>(p.k + b * p.k_token + hk * p.k_head + 2 * i);
        *reinterpret_cast<float2 *>(&qs[2 * i]) = make_float2(bf16_lo(qw), bf16_hi(qw));
        *reinterpret_cast<float2 *>(&ks[2 * i]) = make_float2(bf16_lo(kw), bf16_hi(kw));
    }
    const float e = expf(g), v0 = bf16_lo(vw.x), v1 = bf16_hi(vw.x), v2 = bf16_lo(vw.y), v3 = bf16_hi(vw.y);
    __syncthreads();
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const float kk = ks[row0 + i * kRows], qq = qs[row0 + i * kRows];
        x[i].x = fmaf(kk, v0, e * x[i].x);
        x[i].y = fmaf(kk, v1, e * x[i].y);
        x[i].z = fmaf(kk, v2, e * x[i].z);
        x[i].w = fmaf(kk, v3, e * x[i].w);
        sum.x = fmaf(qq, x[i].x, sum.x);
        sum.y = fmaf(qq, x[i].y, sum.y);
        sum.z = fmaf(qq, x[i].z, sum.z);
        sum.w = fmaf(qq, x[i].w, sum.w);
        __stcs(reinterpret_cast<float4 *>(s + i * kRows * DV), x[i]);
    }
#pragma unroll
    for (int o = kLanes; o < 32; o <<= 1) {
        sum.x += __shfl_xor_sync(0xffffffffu, sum.x, o);
        sum.y += __shfl_xor_sync(0xffffffffu, sum.y, o);
        sum.z += __shfl_xor_sync(0xffffffffu, sum.z, o);
        sum.w += __shfl_xor_sync(0xffffffffu, sum.w, o);
    }
    if (lane < kLanes) *reinterpret_cast<float4 *>(&part[warp][4 * lane]) = sum;
    __syncthreads();
    if (tid < W) {
        float t = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) t += part[w][tid];
        out[tid] = f32_to_bf16_rn(t * p.scale);
    }
}

const void *step_kernel(int dk, int dv) {
    if (dk == 128)
        return dv == 128 ? reinterpret_cast<const void *>(&linear_step_kernel<128, 128>) : reinterpret_cast<const void *>(&linear_step_kernel<128, 64>);
    return dv == 128 ? reinterpret_cast<const void *>(&linear_step_kernel<64, 128>) : reinterpret_cast<const void *>(&linear_step_kernel<64, 64>);
}

}  // namespace linear
}  // namespace sk

extern "C" sgemm_status_t sgemm_bf16_linear_step(const sgemm_linear_step_t *a, sgemm_stream_t stream) {
    using namespace sk;
    using namespace sk::linear;
    if (!a || !valid_flags(a->flags)) return SGEMM_ERR_INVALID_ARG;
    if (a->B < 0 || a->Hk < 1 || a->Hv < a->Hk || a->Hv % a->Hk || a->Hv > 1024 || !std::isfinite(a->scale)) return SGEMM_ERR_INVALID_ARG;
    if ((a->Dk != 64 && a->Dk != 128) || (a->Dv != 64 && a->Dv != 128)) return SGEMM_ERR_UNSUPPORTED_SHAPE;
    if (a->B == 0) return SGEMM_OK;
    if (a->B > ((1LL << 28) - 1) / a->Hv) return SGEMM_ERR_UNSUPPORTED_SHAPE;
    if (!a->q || !a->k || !a->v || !a->g || (a->pool > 0 && !a->state) || !a->slots || !a->out || a->pool < 0 || a->pool >= (1LL << 31))
        return SGEMM_ERR_INVALID_ARG;
    const LinearView io{a->q, a->k, a->v, a->g, a->state, a->out, a->q_token, a->q_head, a->k_token, a->k_head, a->v_token,
                        a->v_head, a->g_token, a->g_head, a->s_slot, a->s_head, a->o_token, a->o_head, a->B, a->pool, a->Hk,
                        a->Hv, a->Dk, a->Dv};
    sgemm_status_t st = check_linear(io);
    if (st != SGEMM_OK) return st;
    if (!aligned(a->slots, 8)) return SGEMM_ERR_MISALIGNED;
    if (linear_touches(io, a->slots, 8 * a->B)) return SGEMM_ERR_INVALID_ARG;
    StepParams p;
    std::memset(&p, 0, sizeof(p));
    int sms = 0;
    st = device_ready(&sms, &p.err);
    if (st != SGEMM_OK) return st;
    p.q = a->q;
    p.k = a->k;
    p.v = a->v;
    p.g = a->g;
    p.state = a->state;
    p.slots = a->slots;
    p.out = a->out;
    p.q_token = a->q_token;
    p.q_head = a->q_head;
    p.k_token = a->k_token;
    p.k_head = a->k_head;
    p.v_token = a->v_token;
    p.v_head = a->v_head;
    p.g_token = a->g_token;
    p.g_head = a->g_head;
    p.s_slot = a->s_slot;
    p.s_head = a->s_head;
    p.o_token = a->o_token;
    p.o_head = a->o_head;
    p.pool = a->pool;
    p.Hv = a->Hv;
    p.share = a->Hv / a->Hk;
    p.scale = a->scale;
    p.flags = static_cast<int>(a->flags);
    if (launch(step_kernel(a->Dk, a->Dv), dim3(static_cast<unsigned>(a->B * a->Hv * (a->Dv / 32))), dim3(kStepThreads), 0,
               reinterpret_cast<cudaStream_t>(stream), &p) != cudaSuccess)
        return SGEMM_ERR_CUDA;
    return SGEMM_OK;
}
