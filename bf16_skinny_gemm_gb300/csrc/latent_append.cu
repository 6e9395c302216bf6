// Append to a paged latent cache, with the position rotation on the way
// (declared in include/sgemm_decode.h).  For every token: the RMS norm of its
// latent vector (optional), the rotation of its E key elements, both written
// to the token's row of the cache, and the rotation of its queries' E elements
// per head.
//
// Every byte is read and written once and there are a few operations an
// element: bound by memory for many tokens, by latency for few.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "decode_common.h"
#include "skinny_ldg.cuh"

namespace sk {
namespace append {

struct AppendParams {
    sgemm_latent_append_t a;
    int *err;
    int group;  // threads a token (a power of two, a whole number of warps)
};

constexpr int kMaxPieces = 4;  // 16-byte pieces of the latent vector a lane keeps: R <= 1024

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    return static_cast<uint32_t>(f32_to_bf16_rn(a)) | (static_cast<uint32_t>(f32_to_bf16_rn(b)) << 16);
}

__device__ __forceinline__ void unpack(const uint4 &q, float (&v)[8]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(w[i]);
        v[2 * i + 1] = bf16_hi(w[i]);
    }
}

__device__ __forceinline__ uint4 pack(const float (&v)[8]) {
    return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

// The token's row of the cache, or null where none is to be written.
__device__ __forceinline__ uint16_t *row_of(const AppendParams &p, long long slot) {
    const long long ps = p.a.page_size;
    if (slot < 0 || slot >= p.a.pages * ps) return nullptr;
    return p.a.cache + (slot / ps) * p.a.page_stride + (slot % ps) * p.a.row_stride;
}

// 16-byte accesses: every row of every array starts on 16 bytes, R is a multiple of 8 and
// at most 1024, and a rotated row's pieces (E / 8 of 16 bytes if interleaved, else E / 16 pairs of
// them) divide a warp, so that a thread meets the same elements, and angles, in every row.
// `p.group` threads take a token: the first warp its latent vector, all of them its H + 1 rotated
// rows, kBatch pieces at a time.  What a thread loads is requested before it waits for the
// token's position and then its angles, a chain of two loads.
template <bool INTER>
__global__ void __launch_bounds__(512) latent_append_vec_kernel(const __grid_constant__ AppendParams p) {
    constexpr int kBatch = 4, kV = INTER ? 1 : 2;  // 16-byte accesses a piece
    const sgemm_latent_append_t &a = p.a;
    if (a.flags & SGEMM_FLAG_PDL) {
        pdl_launch_dependents();
        pdl_wait();
    }
    const int lane = threadIdx.x & 31, in = threadIdx.x & (p.group - 1);
    const long long t = static_cast<long long>(blockIdx.x) * (blockDim.x / p.group) + threadIdx.x / p.group;
    if (t >= a.T) return;  // whole warps; no block barrier below
    const long long pos = a.positions[t], slot = a.slots[t];
    const uint16_t *kv = a.kv + t * a.ldkv;
    const int per = a.E / (8 * kV), half = a.E / 2, u = in & (per - 1);
    const int items = (a.H + 1) * per, rows = p.group / per;  // pieces; rows a turn
    const uint16_t *q = a.q + t * a.q_token + 8 * u;
    uint16_t *qo = a.q_out + t * a.qo_token + 8 * u;

    // row 0 is the key's, row 1 + h head h's
    uint4 v[kBatch][kV];
    auto load = [&](int i) {
        int row = i / per;
#pragma unroll
        for (int b = 0; b < kBatch; ++b, row += rows)
            if (i + b * p.group < items) {
                const uint16_t *src = row == 0 ? kv + a.R + 8 * u : q + (row - 1) * a.q_head;
#pragma unroll
                for (int w = 0; w < kV; ++w) v[b][w] = *reinterpret_cast<const uint4 *>(src + w * half);
            }
    };
    load(in);
    uint4 latent[kMaxPieces], g[kMaxPieces];
    const int pieces = in < 32 ? a.R / 8 : 0;
#pragma unroll
    for (int i = 0; i < kMaxPieces; ++i)
        if (lane + 32 * i < pieces) {
            latent[i] = *reinterpret_cast<const uint4 *>(kv + 8 * (lane + 32 * i));
            if (a.weight) g[i] = *reinterpret_cast<const uint4 *>(a.weight + 8 * (lane + 32 * i));
        }
    const bool bad = pos < 0 || pos >= a.max_position;
    const float *cs = a.cos_sin + (bad ? 0 : pos) * a.ldcs;
    constexpr int kPairs = INTER ? 4 : 8;  // of a piece
    float c[kPairs], s[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; i += 4) {
        const float4 x = *reinterpret_cast<const float4 *>(cs + kPairs * u + i);
        const float4 y = *reinterpret_cast<const float4 *>(cs + half + kPairs * u + i);
        c[i] = x.x, c[i + 1] = x.y, c[i + 2] = x.z, c[i + 3] = x.w;
        s[i] = y.x, s[i + 1] = y.y, s[i + 2] = y.z, s[i + 3] = y.w;
    }
    if (bad) {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) c[i] = s[i] = __int_as_float(0x7fc00000);
    }
    uint16_t *row0 = row_of(p, slot);
    if (in == 0 && (slot >= a.pages * a.page_size || (bad && slot >= 0))) atomicOr(p.err, kErrBadIndex);
    if (in < 32 && row0) {
        if (a.weight) {
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < kMaxPieces; ++i)
                if (lane + 32 * i < pieces) {
                    float x[8];
                    unpack(latent[i], x);
#pragma unroll
                    for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
                }
            const float rs = rsqrtf(warp_sum(ss) / static_cast<float>(a.R) + a.eps);
#pragma unroll
            for (int i = 0; i < kMaxPieces; ++i)
                if (lane + 32 * i < pieces) {
                    float x[8], y[8];
                    unpack(latent[i], x);
                    unpack(g[i], y);
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = x[j] * rs * y[j];
                    latent[i] = pack(x);
                }
        }
#pragma unroll
        for (int i = 0; i < kMaxPieces; ++i)
            if (lane + 32 * i < pieces) *reinterpret_cast<uint4 *>(row0 + 8 * (lane + 32 * i)) = latent[i];
    }
    for (int i = in; i < items; i += kBatch * p.group) {
        if (i != in) load(i);
        int row = i / per;
#pragma unroll
        for (int b = 0; b < kBatch; ++b, row += rows) {
            if (i + b * p.group >= items || (row == 0 && !row0)) continue;
            uint16_t *dst = row == 0 ? row0 + a.R + 8 * u : qo + (row - 1) * a.qo_head;
            float x[8], y[8];
            unpack(v[b][0], x);
            if constexpr (INTER) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    y[2 * j] = x[2 * j] * c[j] - x[2 * j + 1] * s[j];
                    y[2 * j + 1] = x[2 * j + 1] * c[j] + x[2 * j] * s[j];
                }
                *reinterpret_cast<uint4 *>(dst) = pack(y);
            } else {
                unpack(v[b][kV - 1], y);
                float x2[8], y2[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    x2[j] = x[j] * c[j] - y[j] * s[j];
                    y2[j] = y[j] * c[j] + x[j] * s[j];
                }
                *reinterpret_cast<uint4 *>(dst) = pack(x2);
                *reinterpret_cast<uint4 *>(dst + half) = pack(y2);
            }
        }
    }
}

// Any strides and alignment: element by element, the latent vector read once for its sum
// and once for its output.
__global__ void __launch_bounds__(512) latent_append_any_kernel(const __grid_constant__ AppendParams p) {
    const sgemm_latent_append_t &a = p.a;
    if (a.flags & SGEMM_FLAG_PDL) {
        pdl_launch_dependents();
        pdl_wait();
    }
    const long long t = blockIdx.x;
    const int lane = threadIdx.x & 31;
    const uint16_t *kv = a.kv + t * a.ldkv;
    const long long slot = a.slots[t];
    uint16_t *row = row_of(p, slot);
    if (threadIdx.x < 32) {
        if (lane == 0 && slot >= a.pages * a.page_size) atomicOr(p.err, kErrBadIndex);
        if (!row) return;
        float rs = 0.0f;
        if (a.weight) {
            float ss = 0.0f;
            for (int j = lane; j < a.R; j += 32) ss = fmaf(bf16_lo(kv[j]), bf16_lo(kv[j]), ss);
            rs = rsqrtf(warp_sum(ss) / static_cast<float>(a.R) + a.eps);
        }
        for (int j = lane; j < a.R; j += 32)
            row[j] = a.weight ? f32_to_bf16_rn(bf16_lo(kv[j]) * rs * bf16_lo(a.weight[j])) : kv[j];
        return;
    }
    const int half = a.E / 2;
    const long long pos = a.positions[t];
    const bool bad = pos < 0 || pos >= a.max_position;
    const float *cs = a.cos_sin + (bad ? 0 : pos) * a.ldcs;
    const float nan = __int_as_float(0x7fc00000);
    const long long pairs = static_cast<long long>(a.H + 1) * half;
    for (long long i = static_cast<int>(threadIdx.x) - 32; i < pairs; i += static_cast<int>(blockDim.x) - 32) {
        const int h = static_cast<int>(i / half) - 1, u = static_cast<int>(i % half);
        const uint16_t *src = h < 0 ? kv + a.R : a.q + t * a.q_token + h * a.q_head;
        uint16_t *dst = h < 0 ? row + a.R : a.q_out + t * a.qo_token + h * a.qo_head;
        if (h < 0) {
            if (u == 0 && bad && slot >= 0) atomicOr(p.err, kErrBadIndex);
            if (!row) continue;
        }
        const int i0 = a.interleaved ? 2 * u : u, i1 = a.interleaved ? 2 * u + 1 : half + u;
        const float x = bf16_lo(src[i0]), y = bf16_lo(src[i1]);
        const float c = bad ? nan : cs[u], s = bad ? nan : cs[half + u];
        dst[i0] = f32_to_bf16_rn(x * c - y * s);
        dst[i1] = f32_to_bf16_rn(y * c + x * s);
    }
}

}  // namespace append
}  // namespace sk

extern "C" sgemm_status_t sgemm_bf16_latent_append(const sgemm_latent_append_t *a, sgemm_stream_t stream) {
    using namespace sk;
    if (!a || !valid_flags(a->flags)) return SGEMM_ERR_INVALID_ARG;
    const long long T = a->T, W = static_cast<long long>(a->R) + a->E;
    if (T < 0 || T > 0x7fffffffLL || a->R < 1 || a->R > 8192 || a->E < 2 || a->E > 512 || a->E % 2 || a->H < 0 ||
        a->H > 65536 || a->page_size < 1 || a->pages < 0 || a->max_position < 0 || !(a->eps >= 0.0f) ||
        std::isinf(a->eps) || (a->interleaved != 0 && a->interleaved != 1))
        return SGEMM_ERR_INVALID_ARG;
    if (T == 0) return SGEMM_OK;
    if (a->max_position < 1) return SGEMM_ERR_INVALID_ARG;
    if (!a->kv || !a->cos_sin || !a->positions || !a->slots || !a->cache || (a->H > 0 && (!a->q || !a->q_out)))
        return SGEMM_ERR_INVALID_ARG;
    if (a->ldkv < W || a->ldcs < a->E || a->row_stride < W ||
        a->page_stride < (a->page_size - 1) * a->row_stride + W)
        return SGEMM_ERR_INVALID_ARG;
    if (a->H > 0) {
        // heads inside a token, or tokens inside a head: either way no two rows may share elements
        auto apart = [&](long long tok, long long head) {
            const long long th = T == 1 ? 1LL << 62 : tok, hh = a->H == 1 ? 1LL << 62 : head;
            const long long lo = std::min(th, hh), hi = std::max(th, hh);
            const long long n = th <= hh ? T : a->H;
            return lo >= a->E && (hi == (1LL << 62) || hi >= (n - 1) * lo + a->E);
        };
        if (a->q_token < 0 || a->q_head < 0 || !apart(a->qo_token, a->qo_head)) return SGEMM_ERR_INVALID_ARG;
    }
    if (!aligned(a->kv, 2) || !aligned(a->weight, 2) || !aligned(a->cache, 2) || !aligned(a->cos_sin, 4) ||
        !aligned(a->positions, 8) || !aligned(a->slots, 8) || (a->H > 0 && (!aligned(a->q, 2) || !aligned(a->q_out, 2))))
        return SGEMM_ERR_MISALIGNED;
    // outputs (q_out, the cache) apart from the inputs; q_out may be q itself, or another
    // column range of the same heads
    auto extent = [&](long long tok, long long head) { return 2 * ((T - 1) * tok + (a->H - 1) * head + a->E); };
    const long long cache_bytes =
        a->pages < 1 ? 0 : 2 * ((a->pages - 1) * a->page_stride + (a->page_size - 1) * a->row_stride + W);
    const long long kv_bytes = 2 * ((T - 1) * a->ldkv + W);
    auto overlap = [](const void *x, long long nx, const void *y, long long ny) {
        return rows_overlap(x, nx, 0, y, ny, 0, 1);
    };
    if (overlap(a->cache, cache_bytes, a->kv, kv_bytes)) return SGEMM_ERR_INVALID_ARG;
    if (a->H > 0) {
        const long long qb = extent(a->q_token, a->q_head), ob = extent(a->qo_token, a->qo_head);
        if (overlap(a->q_out, ob, a->kv, kv_bytes) || overlap(a->q_out, ob, a->cache, cache_bytes) ||
            overlap(a->q, qb, a->cache, cache_bytes))
            return SGEMM_ERR_INVALID_ARG;
        const bool alike = (a->q_token == a->qo_token || T == 1) && (a->q_head == a->qo_head || a->H == 1);
        if (!(alike && a->q == a->q_out) && overlap(a->q_out, ob, a->q, qb)) {
            const long long step = a->H > 1 ? a->q_head : a->q_token;
            if (!alike || step < 2 * a->E || (T > 1 && a->q_token % step)) return SGEMM_ERR_INVALID_ARG;
            const uintptr_t x = reinterpret_cast<uintptr_t>(a->q), y = reinterpret_cast<uintptr_t>(a->q_out);
            const long long d = static_cast<long long>((x < y ? y - x : x - y) % static_cast<uintptr_t>(2 * step));
            if (d < 2 * a->E || d + 2 * a->E > 2 * step) return SGEMM_ERR_INVALID_ARG;
        }
    }
    int sms = 0;
    append::AppendParams p;
    std::memset(&p, 0, sizeof(p));
    p.a = *a;
    const sgemm_status_t st = device_ready(&sms, &p.err);
    if (st != SGEMM_OK) return st;

    const bool one = T == 1;
    auto rows16 = [&](const void *q, long long ld) { return aligned(q, 16) && (one || ld % 8 == 0); };
    const int per = a->interleaved ? a->E / 8 : a->E / 16;  // 16-byte pieces (pairs of them) of a rotated row
    const bool vec = a->R % 8 == 0 && a->R <= 256 * append::kMaxPieces && a->E % (a->interleaved ? 8 : 16) == 0 &&
                     32 % per == 0 && rows16(a->kv, a->ldkv) && aligned(a->weight, 16) && aligned(a->cache, 16) &&
                     a->row_stride % 8 == 0 && a->page_stride % 8 == 0 && aligned(a->cos_sin, 16) && a->ldcs % 4 == 0 &&
                     (a->H == 0 || (rows16(a->q, a->q_token) && rows16(a->q_out, a->qo_token) && a->q_head % 8 == 0 &&
                                    a->qo_head % 8 == 0));
    const bool pdl = (a->flags & SGEMM_FLAG_PDL) != 0;
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (vec) {
        // Few tokens: a thread a piece (up to 512 a token), for the shortest chain.  Many: 64
        // threads a token, so that each has several loads in flight.
        const long long items = static_cast<long long>(a->H + 1) * per;
        int group = 64;
        if (T <= 4LL * sms)
            while (group < 512 && group < items) group *= 2;
        p.group = group;
        const int tokens = T <= 4LL * sms ? 1 : 256 / group;
        e = launch(a->interleaved ? reinterpret_cast<const void *>(&append::latent_append_vec_kernel<true>)
                                  : reinterpret_cast<const void *>(&append::latent_append_vec_kernel<false>),
                   dim3(static_cast<unsigned>((T + tokens - 1) / tokens)), dim3(static_cast<unsigned>(group * tokens)), 0, cs,
                   pdl, &p);
    } else {
        const long long work = static_cast<long long>(a->H + 1) * (a->E / 2);
        const int threads = 32 + static_cast<int>(std::min<long long>(480, (work + 31) / 32 * 32));
        e = launch(reinterpret_cast<const void *>(&append::latent_append_any_kernel), dim3(static_cast<unsigned>(T)),
                   dim3(static_cast<unsigned>(threads)), 0, cs, pdl, &p);
    }
    if (e != cudaSuccess) return SGEMM_ERR_CUDA;
    return SGEMM_OK;
}
