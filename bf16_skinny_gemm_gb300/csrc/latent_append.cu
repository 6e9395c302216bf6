// Append to a paged latent cache, with the position rotation on the way
// (declared in include/sgemm_decode.h).  For every token: the RMS norm of its
// latent vector (optional), the rotation of its E key elements, both written
// to the token's row of the cache, and the rotation of its queries' E elements
// per head.
//
// Every byte is read and written once and there are a few operations an
// element: bound by memory for many tokens, by latency for few.  One block
// takes one token: warp 0 the latent vector (R / 8 16-byte pieces, kept in
// registers over the reduction), the other warps the H + 1 rotated rows.
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
// at most 1024, and E / 2 a multiple of 8 (4 if interleaved).
__global__ void __launch_bounds__(512) latent_append_vec_kernel(const __grid_constant__ AppendParams p) {
    const sgemm_latent_append_t &a = p.a;
    if (a.flags & SGEMM_FLAG_PDL) {
        pdl_launch_dependents();
        pdl_wait();
    }
    const long long t = blockIdx.x;
    const int lane = threadIdx.x & 31;
    const uint16_t *kv = a.kv + t * a.ldkv;
    if (threadIdx.x < 32) {
        uint4 in[kMaxPieces];
        const int pieces = a.R / 8;
#pragma unroll
        for (int i = 0; i < kMaxPieces; ++i)
            if (lane + 32 * i < pieces) in[i] = *reinterpret_cast<const uint4 *>(kv + 8 * (lane + 32 * i));
        const long long slot = a.slots[t];
        if (lane == 0 && slot >= a.pages * a.page_size) atomicOr(p.err, kErrBadIndex);
        uint16_t *row = row_of(p, slot);
        if (!row) return;
        if (a.weight) {
            uint4 w[kMaxPieces];
#pragma unroll
            for (int i = 0; i < kMaxPieces; ++i)
                if (lane + 32 * i < pieces) w[i] = *reinterpret_cast<const uint4 *>(a.weight + 8 * (lane + 32 * i));
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < kMaxPieces; ++i)
                if (lane + 32 * i < pieces) {
                    float v[8];
                    unpack(in[i], v);
#pragma unroll
                    for (int j = 0; j < 8; ++j) ss = fmaf(v[j], v[j], ss);
                }
            const float rs = rsqrtf(warp_sum(ss) / static_cast<float>(a.R) + a.eps);
#pragma unroll
            for (int i = 0; i < kMaxPieces; ++i)
                if (lane + 32 * i < pieces) {
                    float v[8], g[8];
                    unpack(in[i], v);
                    unpack(w[i], g);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = v[j] * rs * g[j];
                    in[i] = pack(v);
                }
        }
#pragma unroll
        for (int i = 0; i < kMaxPieces; ++i)
            if (lane + 32 * i < pieces) *reinterpret_cast<uint4 *>(row + 8 * (lane + 32 * i)) = in[i];
        return;
    }
    // row 0 is the key's, row 1 + h head h's
    const int half = a.E / 2;
    const int per = a.interleaved ? a.E / 8 : a.E / 16;  // threads a row
    const long long pos = a.positions[t];
    const bool bad = pos < 0 || pos >= a.max_position;
    const float *cs = a.cos_sin + (bad ? 0 : pos) * a.ldcs;
    const float nan = __int_as_float(0x7fc00000);
    for (int i = static_cast<int>(threadIdx.x) - 32; i < (a.H + 1) * per; i += static_cast<int>(blockDim.x) - 32) {
        const int h = i / per - 1, u = i % per;
        const uint16_t *src = h < 0 ? kv + a.R : a.q + t * a.q_token + h * a.q_head;
        uint16_t *dst;
        if (h < 0) {
            const long long slot = a.slots[t];
            if (u == 0 && bad && slot >= 0) atomicOr(p.err, kErrBadIndex);
            dst = row_of(p, slot);
            if (!dst) continue;
            dst += a.R;
        } else {
            dst = a.q_out + t * a.qo_token + h * a.qo_head;
        }
        if (a.interleaved) {
            float v[8];
            unpack(*reinterpret_cast<const uint4 *>(src + 8 * u), v);
            const float4 c = *reinterpret_cast<const float4 *>(cs + 4 * u);
            const float4 s = *reinterpret_cast<const float4 *>(cs + half + 4 * u);
            const float cc[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float x = v[2 * j], y = v[2 * j + 1];
                v[2 * j] = bad ? nan : x * cc[j] - y * sn[j];
                v[2 * j + 1] = bad ? nan : y * cc[j] + x * sn[j];
            }
            *reinterpret_cast<uint4 *>(dst + 8 * u) = pack(v);
        } else {
            float x[8], y[8];
            unpack(*reinterpret_cast<const uint4 *>(src + 8 * u), x);
            unpack(*reinterpret_cast<const uint4 *>(src + half + 8 * u), y);
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const float4 c = *reinterpret_cast<const float4 *>(cs + 8 * u + 4 * g);
                const float4 s = *reinterpret_cast<const float4 *>(cs + half + 8 * u + 4 * g);
                const float cc[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float xv = x[4 * g + j], yv = y[4 * g + j];
                    x[4 * g + j] = bad ? nan : xv * cc[j] - yv * sn[j];
                    y[4 * g + j] = bad ? nan : yv * cc[j] + xv * sn[j];
                }
            }
            *reinterpret_cast<uint4 *>(dst + 8 * u) = pack(x);
            *reinterpret_cast<uint4 *>(dst + half + 8 * u) = pack(y);
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
    const bool vec = a->R % 8 == 0 && a->R <= 256 * append::kMaxPieces && (a->E / 2) % (a->interleaved ? 4 : 8) == 0 &&
                     rows16(a->kv, a->ldkv) && aligned(a->weight, 16) && aligned(a->cache, 16) &&
                     a->row_stride % 8 == 0 && a->page_stride % 8 == 0 && aligned(a->cos_sin, 16) && a->ldcs % 4 == 0 &&
                     (a->H == 0 || (rows16(a->q, a->q_token) && rows16(a->q_out, a->qo_token) && a->q_head % 8 == 0 &&
                                    a->qo_head % 8 == 0));
    const long long work = vec ? static_cast<long long>(a->H + 1) * (a->interleaved ? a->E / 8 : a->E / 16)
                               : static_cast<long long>(a->H + 1) * (a->E / 2);
    const int threads = 32 + static_cast<int>(std::min<long long>(480, (work + 31) / 32 * 32));
    const void *fn = vec ? reinterpret_cast<const void *>(&append::latent_append_vec_kernel)
                         : reinterpret_cast<const void *>(&append::latent_append_any_kernel);
    if (launch(fn, dim3(static_cast<unsigned>(T)), dim3(static_cast<unsigned>(threads)), 0,
               reinterpret_cast<cudaStream_t>(stream), (a->flags & SGEMM_FLAG_PDL) != 0, &p) != cudaSuccess)
        return SGEMM_ERR_CUDA;
    return SGEMM_OK;
}
