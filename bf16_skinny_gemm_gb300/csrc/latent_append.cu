// Append to a paged latent cache, with the position rotation on the way
// (declared in include/sgemm_decode.h).  For every token: the RMS norm of its
// latent vector (optional), the rotation of its E key elements, both written
// to the token's row of the cache, and the rotation of its queries' E elements
// per head.
//
// Every byte is read and written once and there are a few operations an
// element: bound by memory for many tokens, by latency for few.
//
// Measured on one GB300, calls one after the other: 16384 tokens with 32 heads'
// queries 33.1 us (176 MB, 5.3 TB/s, 0.78 of the measured copy rate: the queries'
// parts are 128 bytes every 1152, and a warp waits for a position, then its
// angles, then stores), with half-split pairs 37.1 us (a thread holds twice the
// elements and angles there, and an access covers 64 of a row's 128 bytes);
// 1 to 777 tokens 2.8 to 3.0 us, a launch and that chain.
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
    long long slots;    // rows of the cache
    int tokens, warps;  // tokens a block; warps for a token's queries
};

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
    if (slot < 0 || slot >= p.slots) return nullptr;
    // 32-bit division where it serves: the 64-bit one takes a few hundred instructions
    long long page, row;
    if (p.slots <= 0x7fffffffLL) {
        const unsigned s = static_cast<unsigned>(slot), ps = static_cast<unsigned>(p.a.page_size);
        page = s / ps;
        row = s % ps;
    } else {
        page = slot / p.a.page_size;
        row = slot % p.a.page_size;
    }
    return p.a.cache + page * p.a.page_stride + row * p.a.row_stride;
}

constexpr int kBatch = 4;  // pieces of queries a thread loads at once (16384 tokens: 4 35 us, 2 49, 6 42)

// Cosines and sines of the pairs of piece u (PAIRS of them) at a position; NaN where it is out
// of range.
template <int PAIRS>
struct Angles {
    float c[PAIRS], s[PAIRS];
    __device__ __forceinline__ void load(const sgemm_latent_append_t &a, long long pos, int u) {
        const bool bad = pos < 0 || pos >= a.max_position;
        const float *cs = a.cos_sin + (bad ? 0 : pos) * a.ldcs + PAIRS * u;
#pragma unroll
        for (int i = 0; i < PAIRS; i += 4) {
            const float4 x = *reinterpret_cast<const float4 *>(cs + i);
            const float4 y = *reinterpret_cast<const float4 *>(cs + a.E / 2 + i);
            c[i] = x.x, c[i + 1] = x.y, c[i + 2] = x.z, c[i + 3] = x.w;
            s[i] = y.x, s[i + 1] = y.y, s[i + 2] = y.z, s[i + 3] = y.w;
        }
        if (bad) {
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) c[i] = s[i] = __int_as_float(0x7fc00000);
        }
    }
};

// One piece of a rotated row: 16 bytes with 4 pairs (INTER), or 16 bytes of each half of the row
// with 8 pairs.
template <bool INTER>
struct Piece {
    uint4 v[INTER ? 1 : 2];
    __device__ __forceinline__ void load(const uint16_t *row, int u, int half) {
        v[0] = *reinterpret_cast<const uint4 *>(row + 8 * u);
        if constexpr (!INTER) v[1] = *reinterpret_cast<const uint4 *>(row + half + 8 * u);
    }
    __device__ __forceinline__ void store(uint16_t *row, int u, int half, const Angles<INTER ? 4 : 8> &t) const {
        float x[8];
        unpack(v[0], x);
        if constexpr (INTER) {
            float y[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                y[2 * j] = x[2 * j] * t.c[j] - x[2 * j + 1] * t.s[j];
                y[2 * j + 1] = x[2 * j + 1] * t.c[j] + x[2 * j] * t.s[j];
            }
            *reinterpret_cast<uint4 *>(row + 8 * u) = pack(y);
        } else {
            float y[8], z[8];
            unpack(v[1], y);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                z[j] = x[j] * t.c[j] - y[j] * t.s[j];
                y[j] = y[j] * t.c[j] + x[j] * t.s[j];
            }
            *reinterpret_cast<uint4 *>(row + 8 * u) = pack(z);
            *reinterpret_cast<uint4 *>(row + half + 8 * u) = pack(y);
        }
    }
};

// 16-byte accesses: every row of every array starts on 16 bytes, R is a multiple of 8 and at most
// 256 PIECES, and the pieces of a rotated row divide a warp, so that a thread meets the same
// elements, and angles, in every row.  A token is taken by one warp for its row of the cache and
// `p.warps` for its queries, which load kBatch pieces a thread before they wait for the token's
// position and then its angles, a chain of two loads.
template <bool INTER, int PIECES>
__global__ void __launch_bounds__(544) latent_append_vec_kernel(const __grid_constant__ AppendParams p) {
    const sgemm_latent_append_t &a = p.a;
    if (a.flags & SGEMM_FLAG_PDL) pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = p.warps + 1;
    const int which = warp / warps, w = warp % warps - 1;
    const long long t = static_cast<long long>(blockIdx.x) * p.tokens + which;
    if (t >= a.T) return;  // whole warps; no block barrier below
    const int half = a.E / 2, per = a.E / (INTER ? 8 : 16), u = lane & (per - 1);
    Angles<INTER ? 4 : 8> turn;
    if (w >= 0) {
        const int first = w * (32 / per) + lane / per, step = p.warps * (32 / per);  // heads
        const uint16_t *q = a.q + t * a.q_token;
        uint16_t *qo = a.q_out + t * a.qo_token;
        const long long pos = a.positions[t];
        for (int h0 = first; h0 < a.H; h0 += kBatch * step) {
            Piece<INTER> v[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; ++b)
                if (h0 + b * step < a.H) v[b].load(q + (h0 + b * step) * a.q_head, u, half);
            if (h0 == first) turn.load(a, pos, u);
#pragma unroll
            for (int b = 0; b < kBatch; ++b)
                if (h0 + b * step < a.H) v[b].store(qo + (h0 + b * step) * a.qo_head, u, half, turn);
        }
        return;
    }
    const long long pos = a.positions[t], slot = a.slots[t];
    const uint16_t *kv = a.kv + t * a.ldkv;
    uint4 latent[PIECES], g[PIECES];
    const int pieces = a.R / 8;
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
        if (lane + 32 * i < pieces) {
            latent[i] = *reinterpret_cast<const uint4 *>(kv + 8 * (lane + 32 * i));
            if (a.weight) g[i] = *reinterpret_cast<const uint4 *>(a.weight + 8 * (lane + 32 * i));
        }
    Piece<INTER> key;
    if (lane < per) key.load(kv + a.R, u, half);
    turn.load(a, pos, u);
    uint16_t *row = row_of(p, slot);
    if (lane == 0 && (slot >= p.slots || (slot >= 0 && (pos < 0 || pos >= a.max_position)))) atomicOr(p.err, kErrBadIndex);
    if (!row) return;
    if (lane < per) key.store(row + a.R, u, half, turn);
    if (a.weight) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
            if (lane + 32 * i < pieces) {
                float x[8];
                unpack(latent[i], x);
#pragma unroll
                for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
            }
        const float rs = rsqrtf(warp_sum(ss) / static_cast<float>(a.R) + a.eps);
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
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
    for (int i = 0; i < PIECES; ++i)
        if (lane + 32 * i < pieces) *reinterpret_cast<uint4 *>(row + 8 * (lane + 32 * i)) = latent[i];
}

// Any strides and alignment: element by element, the latent vector read once for its sum
// and once for its output.
__global__ void __launch_bounds__(512) latent_append_any_kernel(const __grid_constant__ AppendParams p) {
    const sgemm_latent_append_t &a = p.a;
    if (a.flags & SGEMM_FLAG_PDL) pdl_launch_dependents();
    pdl_wait();
    const long long t = blockIdx.x;
    const int lane = threadIdx.x & 31;
    const uint16_t *kv = a.kv + t * a.ldkv;
    const long long slot = a.slots[t];
    uint16_t *row = row_of(p, slot);
    if (threadIdx.x < 32) {
        if (lane == 0 && slot >= p.slots) atomicOr(p.err, kErrBadIndex);
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
    p.slots = a->pages * a->page_size;
    const sgemm_status_t st = device_ready(&sms, &p.err);
    if (st != SGEMM_OK) return st;

    const bool one = T == 1;
    auto rows16 = [&](const void *q, long long ld) { return aligned(q, 16) && (one || ld % 8 == 0); };
    const int per = a->interleaved ? a->E / 8 : a->E / 16;  // 16-byte pieces (pairs of them) of a rotated row
    const bool vec = a->R % 8 == 0 && a->R <= 1024 && a->E % (a->interleaved ? 8 : 16) == 0 &&
                     32 % per == 0 && rows16(a->kv, a->ldkv) && aligned(a->weight, 16) && aligned(a->cache, 16) &&
                     a->row_stride % 8 == 0 && a->page_stride % 8 == 0 && aligned(a->cos_sin, 16) && a->ldcs % 4 == 0 &&
                     (a->H == 0 || (rows16(a->q, a->q_token) && rows16(a->q_out, a->qo_token) && a->q_head % 8 == 0 &&
                                    a->qo_head % 8 == 0));
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (vec) {
        // Few tokens: a thread a piece (up to 16 warps a token), for the shortest chain.  More than
        // one for each SM: one warp for a token's queries where they fit, several loads in flight
        // in each, two tokens a block.  The one against the other, 128 heads: 8 tokens 2.68 us,
        // 2.8; 300 tokens 3.1, 2.85; 32 heads: 1200 tokens 5.1, 3.0; 16384 tokens with one token a
        // block in place of two 34.9 for 35.3, with four 36.9.
        const int full = (a->H * per + 31) / 32;
        const bool many = T > sms;
        p.warps = many ? std::min((full + append::kBatch - 1) / append::kBatch, 4) : std::min(full, 16);
        p.tokens = many ? 2 : 1;
        const bool narrow = a->R <= 512;
        const void *fn =
            a->interleaved
                ? (narrow ? reinterpret_cast<const void *>(&append::latent_append_vec_kernel<true, 2>)
                          : reinterpret_cast<const void *>(&append::latent_append_vec_kernel<true, 4>))
                : (narrow ? reinterpret_cast<const void *>(&append::latent_append_vec_kernel<false, 2>)
                          : reinterpret_cast<const void *>(&append::latent_append_vec_kernel<false, 4>));
        e = launch(fn, dim3(static_cast<unsigned>((T + p.tokens - 1) / p.tokens)),
                   dim3(static_cast<unsigned>(32 * p.tokens * (p.warps + 1))), 0, cs, &p);
    } else {
        const long long work = static_cast<long long>(a->H + 1) * (a->E / 2);
        const int threads = 32 + static_cast<int>(std::min<long long>(480, (work + 31) / 32 * 32));
        e = launch(reinterpret_cast<const void *>(&append::latent_append_any_kernel), dim3(static_cast<unsigned>(T)),
                   dim3(static_cast<unsigned>(threads)), 0, cs, &p);
    }
    if (e != cudaSuccess) return SGEMM_ERR_CUDA;
    return SGEMM_OK;
}
