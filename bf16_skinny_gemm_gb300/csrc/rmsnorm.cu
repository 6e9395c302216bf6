// Residual add and RMS norm in one pass, with a BF16 or an 8-bit output
// (declared in include/sgemm_decode.h):
//
//     h = x + residual,   y = h * rsqrt(mean(h^2) + eps) * weight
//
// One read of x and residual, one write of y and of the new residual: the
// operator moves 6 to 8 bytes an element and does about as many operations, so
// it is bound by memory for many rows and by latency for few.  A row stays in
// registers between the reduction and the output (FP32, the sum not rounded to
// BF16 in between), so nothing is read twice.
//
// Measured on one GB300, calls one after the other: 16384 x 4096 in 8 bits, a
// scale a row, 71.8 us (6.5 TB/s, 0.97 of the measured copy rate); 1003 x 1537
// (2 bytes an access) 3.9 us; 1 x 4096 2.5 us, of which the arithmetic is little:
// a launch, one load, two reductions' barriers and a store, one after the other.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "decode_common.h"
#include "skinny_ldg.cuh"

namespace sk {
namespace norm {

struct NormParams {
    const uint16_t *x, *residual, *weight;
    uint16_t *residual_out;
    void *y;
    float *scales;
    long long ldx, ldr, ldro, ldy, lds, T;
    int D;
    int tpr;  // threads per row, a multiple of 32
    float eps;
    int flags;
};

constexpr float kE4m3Max = 448.0f;
constexpr int kGroup = 128;
constexpr long long kMaxD = 1LL << 30;  // columns are counted in 32 bits, in steps of up to 4096
// y / s is worked out as y (1 / s), two roundings of 2^-24 beside e4m3's of 2^-4, which differ from
// one only where y / s is within 2^-23 of a tie; dividing each element is most of the kernel's
// arithmetic (16384 x 4096, a scale a row: 72.6 us, 90.9 by division).  Below this scale by division.
constexpr float kTinyScale = 1e-30f;

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// A scale too small to be a normal number is rounded up: never to 0, where the largest y would
// become infinite and a y of 0 NaN, nor so far down that the largest y / s passes e4m3's maximum.
__device__ __forceinline__ float scale_of(float top) {
    if (top == 0.0f) return 1.0f;
    const float s = top / kE4m3Max;
    return s < 1.17549435e-38f ? __fdiv_ru(top, kE4m3Max) : s;
}

__device__ __forceinline__ uint16_t pack_e4m3(float a, float b) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    return static_cast<uint32_t>(f32_to_bf16_rn(a)) | (static_cast<uint32_t>(f32_to_bf16_rn(b)) << 16);
}

// Sum (or NaN-propagating maximum) over the row's warps; every thread gets the
// same bits.  `part` holds one float a warp and is used once per call.
template <bool MAX>
__device__ __forceinline__ float row_reduce(float v, int wr, float *part) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        const float o = __shfl_xor_sync(0xffffffffu, v, off);
        v = MAX ? max_nan(v, o) : v + o;
    }
    if (wr == 1) return v;
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    v = lane < wr ? part[lane] : 0.0f;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        const float o = __shfl_xor_sync(0xffffffffu, v, off);
        v = MAX ? max_nan(v, o) : v + o;
    }
    return v;
}

// How the elements of a row are dealt to its threads.  A thread holds NV units.
// VEC 8: a unit is 8 consecutive elements (16-byte accesses), the units of one
// warp access 256 consecutive elements, so 16 lanes hold a group of 128.
// VEC 2 and 1 (rows that do not start on 16 bytes): a warp access covers 64 or
// 32 consecutive elements and a unit is the thread's 4 elements of a chunk of
// 128, so a warp holds a group of 128.
template <int VEC>
struct Deal {
    static constexpr int kUnit = VEC == 8 ? 8 : 4;
    static __device__ __forceinline__ int first(int u, int tpr, int t) {
        if (VEC == 8) return (u * tpr + t) * 8;
        return ((u * (tpr >> 5) + (t >> 5)) << 7) + VEC * (t & 31);
    }
    // column of the i-th element of a unit, from its first column
    static __device__ __forceinline__ int col(int c, int i) {
        if (VEC == 8) return c + i;
        if (VEC == 2) return c + (i >> 1) * 64 + (i & 1);
        return c + 32 * i;
    }
};

// A unit as it was read (BF16 bits), 0 past the row.
template <int VEC>
struct Raw {
    uint32_t w[VEC == 2 ? 2 : 4];
    __device__ __forceinline__ void load(const uint16_t *row, int c, int D) {
        if constexpr (VEC == 8) {
            uint4 q = make_uint4(0u, 0u, 0u, 0u);
            if (c < D) q = *reinterpret_cast<const uint4 *>(row + c);
            w[0] = q.x;
            w[1] = q.y;
            w[2] = q.z;
            w[3] = q.w;
        } else if constexpr (VEC == 2) {
#pragma unroll
            for (int i = 0; i < 2; ++i) w[i] = c + 64 * i < D ? *reinterpret_cast<const uint32_t *>(row + c + 64 * i) : 0u;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = c + 32 * i < D ? row[c + 32 * i] : 0u;
        }
    }
    // the i-th element (of Deal<VEC>::kUnit)
    __device__ __forceinline__ float get(int i) const {
        if constexpr (VEC == 1) return bf16_lo(w[i]);
        return i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
    }
};

template <int VEC>
__device__ __forceinline__ void store_unit(uint16_t *row, int c, int D, const float (&v)[Deal<VEC>::kUnit]) {
    if constexpr (VEC == 8) {
        if (c < D)
            *reinterpret_cast<uint4 *>(row + c) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                                             pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    } else if constexpr (VEC == 2) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (c + 64 * i < D) *reinterpret_cast<uint32_t *>(row + c + 64 * i) = pack_bf16(v[2 * i], v[2 * i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + 32 * i < D) row[c + 32 * i] = f32_to_bf16_rn(v[i]);
    }
}

template <int VEC>
__device__ __forceinline__ void store_unit_e4m3(uint8_t *row, int c, int D, const float (&v)[Deal<VEC>::kUnit]) {
    if constexpr (VEC == 8) {
        if (c < D) {
            uint2 q;
            q.x = pack_e4m3(v[0], v[1]) | (static_cast<uint32_t>(pack_e4m3(v[2], v[3])) << 16);
            q.y = pack_e4m3(v[4], v[5]) | (static_cast<uint32_t>(pack_e4m3(v[6], v[7])) << 16);
            *reinterpret_cast<uint2 *>(row + c) = q;
        }
    } else if constexpr (VEC == 2) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (c + 64 * i < D) *reinterpret_cast<uint16_t *>(row + c + 64 * i) = pack_e4m3(v[2 * i], v[2 * i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + 32 * i < D) row[c + 32 * i] = static_cast<uint8_t>(pack_e4m3(v[i], 0.0f));
    }
}

// A block takes blockDim.x / tpr rows (more than one only where tpr is 32, so
// that the block barriers below are reached by a block of one row, or by none).
// Threads a row at most, by the units a thread holds: 64 registers for 1024, 128 for 512.
constexpr int most_threads(int nv) { return nv <= 2 ? 1024 : 512; }

template <int VEC, int NV, int FORM>
__global__ void __launch_bounds__(most_threads(NV)) add_rmsnorm_kernel(const __grid_constant__ NormParams p) {
    using DL = Deal<VEC>;
    constexpr int E = DL::kUnit;
    __shared__ float part[2][32];
    if (p.flags & kFlagPdl) pdl_launch_dependents();
    const int tpr = p.tpr, wr = tpr >> 5;
    const int t = threadIdx.x % tpr;
    const long long row = static_cast<long long>(blockIdx.x) * (blockDim.x / tpr) + threadIdx.x / tpr;
    pdl_wait();
    if (row >= p.T) return;  // whole warps, and no block barrier is used where a block has several rows

    float h[NV][E];
    Raw<VEC> in[NV], add[NV];
#pragma unroll
    for (int u = 0; u < NV; ++u) in[u].load(p.x + row * p.ldx, DL::first(u, tpr, t), p.D);
    if (p.residual) {
#pragma unroll
        for (int u = 0; u < NV; ++u) add[u].load(p.residual + row * p.ldr, DL::first(u, tpr, t), p.D);
#pragma unroll
        for (int u = 0; u < NV; ++u)
#pragma unroll
            for (int i = 0; i < E; ++i) h[u][i] = in[u].get(i) + add[u].get(i);
    } else {
#pragma unroll
        for (int u = 0; u < NV; ++u)
#pragma unroll
            for (int i = 0; i < E; ++i) h[u][i] = in[u].get(i);
    }
    Raw<VEC> w[NV];
#pragma unroll
    for (int u = 0; u < NV; ++u) w[u].load(p.weight, DL::first(u, tpr, t), p.D);
    if (p.residual_out) {
#pragma unroll
        for (int u = 0; u < NV; ++u) store_unit<VEC>(p.residual_out + row * p.ldro, DL::first(u, tpr, t), p.D, h[u]);
    }
    float ss = 0.0f;
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
        for (int i = 0; i < E; ++i) ss = fmaf(h[u][i], h[u][i], ss);
    ss = row_reduce<false>(ss, wr, part[0]);
    const float rs = rsqrtf(ss / static_cast<float>(p.D) + p.eps);
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
        for (int i = 0; i < E; ++i) h[u][i] = h[u][i] * rs * w[u].get(i);

    if constexpr (FORM == SGEMM_NORM_BF16) {
        uint16_t *y = static_cast<uint16_t *>(p.y) + row * p.ldy;
#pragma unroll
        for (int u = 0; u < NV; ++u) store_unit<VEC>(y, DL::first(u, tpr, t), p.D, h[u]);
    } else {
        // elements past the row are 0 (their x, residual and weight were read as 0)
        uint8_t *y = static_cast<uint8_t *>(p.y) + row * p.ldy;
        float *scales = p.scales + row * p.lds;
        float s = 1.0f;
        if constexpr (FORM == SGEMM_NORM_E4M3_ROW) {
            float top = 0.0f;
#pragma unroll
            for (int u = 0; u < NV; ++u)
#pragma unroll
                for (int i = 0; i < E; ++i) top = max_nan(top, fabsf(h[u][i]));
            s = scale_of(row_reduce<true>(top, wr, part[1]));
            if (t == 0) scales[0] = s;
        }
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int c = DL::first(u, tpr, t);
            if constexpr (FORM == SGEMM_NORM_E4M3_GROUP128) {
                float top = 0.0f;
#pragma unroll
                for (int i = 0; i < E; ++i) top = max_nan(top, fabsf(h[u][i]));
#pragma unroll
                for (int off = VEC == 8 ? 8 : 16; off >= 1; off >>= 1)
                    top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, off));
                s = scale_of(top);
                if (c % kGroup == 0 && c < p.D) scales[c / kGroup] = s;
            }
            float q[E];
            const float inv = 1.0f / s;
#pragma unroll
            for (int i = 0; i < E; ++i) q[i] = h[u][i] * inv;
            if (s < kTinyScale) {  // 1 / s would overflow
#pragma unroll
                for (int i = 0; i < E; ++i) q[i] = h[u][i] / s;
            }
            store_unit_e4m3<VEC>(y, c, p.D, q);
        }
    }
}

// Rows too long for a block's registers (more than 16384 columns): the row is read
// again for each pass (sum, maximum, output) by one block, element by element, 2
// bytes an access.  4000 rows of 16392 columns 228 us (16384, by the other kernel:
// 94.7, 0.82 of the measured copy rate), one such row 8.3 us (3.3).
template <int FORM>
__global__ void __launch_bounds__(1024) add_rmsnorm_long_kernel(const __grid_constant__ NormParams p) {
    __shared__ float part[2][32];
    if (p.flags & kFlagPdl) pdl_launch_dependents();
    pdl_wait();
    const long long row = blockIdx.x;
    const int wr = blockDim.x >> 5;
    const uint16_t *x = p.x + row * p.ldx;
    const uint16_t *r = p.residual ? p.residual + row * p.ldr : nullptr;
    auto sum = [&](int c) { return bf16_lo(x[c]) + (r ? bf16_lo(r[c]) : 0.0f); };
    float ss = 0.0f;
    for (int c = threadIdx.x; c < p.D; c += blockDim.x) ss = fmaf(sum(c), sum(c), ss);
    ss = row_reduce<false>(ss, wr, part[0]);
    const float rs = rsqrtf(ss / static_cast<float>(p.D) + p.eps);
    auto value = [&](float h, int c) { return h * rs * bf16_lo(p.weight[c]); };
    float s = 1.0f;
    if constexpr (FORM == SGEMM_NORM_E4M3_ROW) {
        float top = 0.0f;
        for (int c = threadIdx.x; c < p.D; c += blockDim.x) top = max_nan(top, fabsf(value(sum(c), c)));
        s = scale_of(row_reduce<true>(top, wr, part[1]));
        if (threadIdx.x == 0) p.scales[row * p.lds] = s;
    }
    // blockDim.x is a multiple of 128 and a warp takes a whole group of 128 columns a turn
    const int lane = threadIdx.x & 31;
    for (int c0 = (threadIdx.x >> 5) * kGroup; c0 < p.D; c0 += wr * kGroup) {
        float h[4], v[4], top = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = c0 + 32 * i + lane;
            h[i] = c < p.D ? sum(c) : 0.0f;
            v[i] = c < p.D ? value(h[i], c) : 0.0f;
            top = max_nan(top, fabsf(v[i]));
        }
        if constexpr (FORM == SGEMM_NORM_E4M3_GROUP128) {
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, off));
            s = scale_of(top);
            if (lane == 0) p.scales[row * p.lds + c0 / kGroup] = s;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = c0 + 32 * i + lane;
            if (c < p.D) {
                if (p.residual_out) p.residual_out[row * p.ldro + c] = f32_to_bf16_rn(h[i]);
                if constexpr (FORM == SGEMM_NORM_BF16) {
                    static_cast<uint16_t *>(p.y)[row * p.ldy + c] = f32_to_bf16_rn(v[i]);
                } else {
                    static_cast<uint8_t *>(p.y)[row * p.ldy + c] = static_cast<uint8_t>(pack_e4m3(v[i] / s, 0.0f));
                }
            }
        }
    }
}

template <int VEC, int NV>
const void *kernel_of(int form) {
    switch (form) {
        case SGEMM_NORM_BF16: return reinterpret_cast<const void *>(&add_rmsnorm_kernel<VEC, NV, SGEMM_NORM_BF16>);
        case SGEMM_NORM_E4M3_ROW: return reinterpret_cast<const void *>(&add_rmsnorm_kernel<VEC, NV, SGEMM_NORM_E4M3_ROW>);
        default: return reinterpret_cast<const void *>(&add_rmsnorm_kernel<VEC, NV, SGEMM_NORM_E4M3_GROUP128>);
    }
}

template <int VEC>
const void *kernel_of(int nv, int form) {
    if (nv == 1) return kernel_of<VEC, 1>(form);
    if (nv == 2) return kernel_of<VEC, 2>(form);
    if (nv == 4) return kernel_of<VEC, 4>(form);
    if constexpr (VEC != 8) return kernel_of<VEC, 8>(form);
    return nullptr;
}

const void *long_kernel_of(int form) {
    switch (form) {
        case SGEMM_NORM_BF16: return reinterpret_cast<const void *>(&add_rmsnorm_long_kernel<SGEMM_NORM_BF16>);
        case SGEMM_NORM_E4M3_ROW: return reinterpret_cast<const void *>(&add_rmsnorm_long_kernel<SGEMM_NORM_E4M3_ROW>);
        default: return reinterpret_cast<const void *>(&add_rmsnorm_long_kernel<SGEMM_NORM_E4M3_GROUP128>);
    }
}

}  // namespace norm
}  // namespace sk

extern "C" sgemm_status_t sgemm_bf16_add_rmsnorm(const sgemm_add_rmsnorm_t *a, sgemm_stream_t stream) {
    using namespace sk;
    if (!a || !valid_flags(a->flags)) return SGEMM_ERR_INVALID_ARG;
    if (a->form < SGEMM_NORM_BF16 || a->form > SGEMM_NORM_E4M3_GROUP128) return SGEMM_ERR_INVALID_ARG;
    const bool bf16 = a->form == SGEMM_NORM_BF16;
    const long long T = a->T, D = a->D;
    if (T < 0 || T > 0x7fffffffLL || D < 1 || !(a->eps >= 0.0f) || std::isinf(a->eps)) return SGEMM_ERR_INVALID_ARG;
    if (D > norm::kMaxD) return SGEMM_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return SGEMM_OK;
    if (!a->x || !a->weight || !a->y || (!bf16 && !a->scales)) return SGEMM_ERR_INVALID_ARG;
    const long long groups = a->form == SGEMM_NORM_E4M3_GROUP128 ? (D + norm::kGroup - 1) / norm::kGroup : 1;
    if (a->ldx < D || a->ldy < D || (a->residual && a->ldr < D) || (a->residual_out && a->ldro < D) ||
        (!bf16 && a->lds < groups))
        return SGEMM_ERR_INVALID_ARG;
    if (!aligned(a->x, 2) || !aligned(a->residual, 2) || !aligned(a->weight, 2) || !aligned(a->residual_out, 2) ||
        (bf16 && !aligned(a->y, 2)) || (!bf16 && !aligned(a->scales, 4)))
        return SGEMM_ERR_MISALIGNED;
    // outputs: x or residual itself, or apart from every input and from each other
    struct Arr {
        const void *p;
        long long w, s;
    };
    const Arr ins[2] = {{a->x, 2 * D, 2 * a->ldx}, {a->residual, 2 * D, 2 * a->ldr}};
    const Arr outs[3] = {{a->y, (bf16 ? 2 : 1) * D, (bf16 ? 2 : 1) * a->ldy},
                         {a->residual_out, 2 * D, 2 * a->ldro},
                         {bf16 ? nullptr : a->scales, 4 * groups, 4 * a->lds}};
    for (int i = 0; i < 3; ++i) {
        const Arr &o = outs[i];
        if (rows_overlap(o.p, (T - 1) * o.s + o.w, 0, a->weight, 2 * D, 0, 1)) return SGEMM_ERR_INVALID_ARG;
        for (const Arr &in : ins) {
            const bool same = o.p == in.p && (o.s == in.s || T == 1) && (i == 1 || (i == 0 && bf16));
            if (!same && rows_overlap(o.p, o.w, o.s, in.p, in.w, in.s, T)) return SGEMM_ERR_INVALID_ARG;
        }
        for (int j = 0; j < i; ++j)
            if (rows_overlap(o.p, o.w, o.s, outs[j].p, outs[j].w, outs[j].s, T)) return SGEMM_ERR_INVALID_ARG;
    }
    int sms = 0, *err = nullptr;
    const sgemm_status_t st = device_ready(&sms, &err);
    if (st != SGEMM_OK) return st;

    norm::NormParams p;
    std::memset(&p, 0, sizeof(p));
    p.x = a->x;
    p.residual = a->residual;
    p.weight = a->weight;
    p.residual_out = a->residual_out;
    p.y = a->y;
    p.scales = a->scales;
    p.ldx = a->ldx;
    p.ldr = a->ldr;
    p.ldro = a->ldro;
    p.ldy = a->ldy;
    p.lds = a->lds;
    p.T = T;
    p.D = a->D;
    p.eps = a->eps;
    p.flags = static_cast<int>(a->flags);

    // the widest access every row of every array allows (strides do not matter for one row)
    auto fits = [&](int vec) {
        auto row = [&](const void *q, long long ld, int bytes) {
            return !q || (aligned(q, vec * bytes) && (T == 1 || ld % vec == 0));
        };
        return D % vec == 0 && row(a->x, a->ldx, 2) && row(a->residual, a->ldr, 2) && row(a->weight, 0, 2) &&
               row(a->residual_out, a->ldro, 2) && row(a->y, a->ldy, bf16 ? 2 : 1);
    };
    const int vec = fits(8) ? 8 : fits(2) ? 2 : 1;
    // a unit covers a whole chunk of 128 columns a warp where it is not 8 consecutive elements
    const int units = vec == 8 ? (a->D + 7) / 8 : (a->D + 127) / 128 * 32;
    const int most = vec == 8 ? 4 : 8;
    // Few rows: one unit a thread, for the shortest chain.  More than two for each SM: up to four, so
    // that a thread has as many loads in flight and fewer threads meet at the barriers.  One against
    // four: 8 x 8192 (8 bits, a scale per 128) 2.75 us, 3.1; 200 x 4096 (BF16) 2.65, 2.63;
    // 320 x 4096 3.13, 2.94; 320 x 8192 (8 bits) 5.7, 4.8; 16384 x 4096 (8 bits) 90 (two: 78), 75.
    const bool many = T > 2LL * sms;
    int nv = 1;
    if (many)
        while (nv < 4 && units >= 64 * nv) nv *= 2;
    while (nv < most && units > norm::most_threads(nv) * nv) nv *= 2;
    const void *fn;
    dim3 grid, block;
    if (units > norm::most_threads(nv) * nv) {
        fn = norm::long_kernel_of(a->form);
        p.tpr = 1024;
        block = dim3(1024);
        grid = dim3(static_cast<unsigned>(T));
    } else {
        fn = vec == 8 ? norm::kernel_of<8>(nv, a->form) : vec == 2 ? norm::kernel_of<2>(nv, a->form)
                                                                   : norm::kernel_of<1>(nv, a->form);
        p.tpr = ((units + nv - 1) / nv + 31) / 32 * 32;
        const int rows = p.tpr == 32 && many ? 4 : 1;
        block = dim3(static_cast<unsigned>(p.tpr * rows));
        grid = dim3(static_cast<unsigned>((T + rows - 1) / rows));
    }
    if (launch(fn, grid, block, 0, reinterpret_cast<cudaStream_t>(stream), &p) !=
        cudaSuccess)
        return SGEMM_ERR_CUDA;
    return SGEMM_OK;
}
