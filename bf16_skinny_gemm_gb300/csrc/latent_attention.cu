// Attention of new tokens over a paged latent cache, absorbed form (declared
// in include/sgemm_decode.h).  All heads of a token share one cached row of
// R + E elements, whose first R are also its value:
//
//     s_j = scale q . row_j,   out = sum_j exp(s_j - m) row_j[:R] / sum_j exp(s_j - m)
//
// What bounds it.  A row of 576 elements (1152 bytes) is used for
// 2 (2R + E) = 2176 operations per head, 2 per byte and head: with up to about
// 140 (head, token) rows a sequence the cache's bytes bound it, above that the
// tensor cores.  So every cached byte is to be read from memory once, for all
// rows of its sequence, and enough of them have to be in flight all the time.
//
// Layout.  A CTA takes NT = 16, 32 or 64 query rows ((token, head) pairs of one
// sequence) and walks its keys in tiles of 64:
//
//  * The transposed products keep the keys (then the latent elements) on the
//    M side of tcgen05.mma and the few query rows on the N side, so that few
//    rows cost few columns, not an idle tile:
//        S^T[64 keys, NT]  = K[64, R+E] Q^T        K and Q K-major
//        O^T[R, NT]       += K[:, :R]^T P^T        both MN-major, M = 128 a time
//    One copy of the tile in shared memory (64 rows x 128 bytes per chunk of 64
//    elements, 128-byte swizzle) serves as A of both products.
//  * Warp 0 streams the tiles with TMA into a ring of slots (two chunks, 128
//    latent elements, a slot; the E elements in a ring of their own).  Slots
//    rather than tiles: a slot is free again as soon as its part of O^T is
//    done, and what is left of shared memory beside Q holds 1.75 to 2.5 tiles.
//  * One thread of warp 1 issues the products.  It takes whichever is ready:
//    O^T of tile t as soon as its weights are there, else the next slot of
//    S^T of tile t + 1; waiting for the latter first would hold tile t's slots.
//  * Warps 2..5 do the softmax: S^T is read in the 16 x 256-bit form, so that
//    all lanes hold scores though M = 64 fills half of the lanes.  The running
//    maximum of a row is over keys, which lie across lanes and warps; it is
//    exchanged only in tiles where some score exceeds the maximum in use by
//    more than 2^8 (in units of the result), else the old one stands: one
//    barrier with a vote a tile.  The weights are then at most 2^8, and neither
//    their rounding to BF16 nor the FP32 sums care about that factor.
//  * Warps 6 and 7 copy the queries of the next piece of work (any strides).
//
// Work split.  The tiles of all sequences form one line, cut into equal shares,
// one for each group of CTAs (a group has a CTA for each NT rows of a sequence
// with max_q tokens, so that these read a tile at about the same time and the
// L2 cache serves all but the first).  The lengths are on the device, so each
// CTA finds its share itself.  A sequence that a share ends in leaves partial
// results (FP32 O, m and l), which a second kernel joins in the order of the
// shares: the result does not depend on timing.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>

#include "decode_common.h"
#include "skinny_tc05.cuh"

namespace sk {
namespace latent {

constexpr int kTile = 64;                // keys per tile (M of the first product)
constexpr int kChunk = kTile * 64 * 2;   // 64 keys x 64 elements
constexpr int kSlot = 2 * kChunk;        // 128 latent elements (M of the second product)
constexpr int kMaxSlots = 12;
constexpr int kMaxRopeSlots = 3;
constexpr int kThreads = 256;            // producer, MMA, 4 softmax and 2 query-loading warps
constexpr int kStaticSmem = 4096;        // bound on the static shared memory below

struct LatentParams {
    CUtensorMap tv;  // the latent part: {64, page rows, R / 64, pages}
    CUtensorMap tr;  // the rotated part: {E, page rows, pages}
    const uint16_t *q;
    const int *table;
    const int *lens;
    const int *cu_q;
    uint16_t *out;
    float *lse;
    float *ws;
    int *err;
    long long q_token, q_head, ldt, out_token, out_head, lse_token, total_q;
    int pages, page_size, width;
    int B, H, R, E, max_q;
    int nt, rt, groups;     // rows a CTA, CTAs a group, groups
    int slots, rope_slots;  // rings
    float scale_log2;       // scale * log2(e)
    int flags;
    int nseg, by_seq, cw, pw;  // the joining kernel's grid
};

// ------------------------------------------------------------------ the work's line of tiles
struct Seq {
    int q0, n, n_all, len;  // first query row, tokens computed, tokens, cached rows
    bool bad;               // an entry was out of range and was cut
};

__device__ __forceinline__ Seq seq_of(const LatentParams &p, int b) {
    Seq s;
    s.bad = false;
    if (p.cu_q) {
        s.q0 = p.cu_q[b];
        s.n_all = p.cu_q[b + 1] - s.q0;
        if (s.q0 < 0 || s.n_all < 0 || static_cast<long long>(s.q0) + s.n_all > p.total_q) {
            s.bad = true;
            s.n_all = 0;
            s.q0 = 0;
        }
    } else {
        s.q0 = b * p.max_q;
        s.n_all = p.max_q;
    }
    s.n = min(s.n_all, p.max_q);
    s.bad |= s.n_all > p.max_q;
    const long long most = static_cast<long long>(p.width) * p.page_size;
    const int len = p.lens[b];
    s.bad |= len > most || len < 0;
    s.len = static_cast<int>(max(0LL, min(static_cast<long long>(len), most)));
    return s;
}

// Tiles of a sequence on the line: at least one where it has tokens (their results are
// written though they see nothing).
__device__ __forceinline__ int tiles_of(const Seq &s) {
    return s.n > 0 ? max(1, (s.len + kTile - 1) / kTile) : 0;
}

// Exclusive prefix sum over the block's threads, and the total.  `part`: 32 ints.
__device__ __forceinline__ int block_prefix(int v, int *part, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    if (lane == 31) part[warp] = x;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < warps; ++w) {
        const int y = part[w];
        if (w < warp) before += y;
        all += y;
    }
    __syncthreads();
    *total = all;
    return before + x - v;
}

__device__ __forceinline__ int share_begin(int units, int g, int groups) {
    return static_cast<int>(static_cast<long long>(units) * g / groups);
}

// One piece of a share: rows row0 .. row0 + nrows of sequence b, its tiles k0 .. k1 - 1 (none
// where the rows see no key of the piece).
struct Piece {
    Seq s;
    int b, row0, nrows, k0, k1;
    bool first, last;  // holds the sequence's first / last tile
};

struct Walk {
    int b, k, left;
    __device__ __forceinline__ bool next(const LatentParams &p, int r, Piece &o) {
        while (left > 0) {
            o.s = seq_of(p, b);
            const int kt = tiles_of(o.s);
            const int take = min(kt - k, left);
            o.b = b;
            o.k0 = k;
            o.first = k == 0;
            o.last = k + take == kt;
            o.row0 = r * p.nt;
            const int rows = o.s.n * p.H;
            ++b;
            k = 0;
            left -= take;
            if (take == 0 || o.row0 >= rows) continue;
            o.nrows = min(p.nt, rows - o.row0);
            // keys that the piece's last row sees
            const int seen = o.s.len - o.s.n_all + (o.row0 + o.nrows - 1) / p.H + 1;
            o.k1 = max(o.k0, min(o.k0 + take, (max(seen, 0) + kTile - 1) / kTile));
            return true;
        }
        return false;
    }
};

// ------------------------------------------------------------------------------- primitives
using tc05::bar_arrive;
using tc05::bar_try;
using tc05::mma_commit;
using tc05::prefetch_tmap;
using tc05::tc_fence_after;
using tc05::tc_fence_before;
using tc05::tmem_ld16;

__device__ __forceinline__ bool bar_test(uint32_t b, unsigned parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(b), "r"(parity)
        : "memory");
    return ok != 0;
}

// Wait for a phase, at most kWaitLimitNs, and not past another role's giving up.
__device__ __forceinline__ bool wait_or_stop(uint32_t b, unsigned parity, int *stop) {
    if (bar_try(b, parity)) return true;
    const unsigned long long t0 = global_ns();
    while (!bar_try(b, parity)) {
        if (*reinterpret_cast<volatile int *>(stop)) return false;
        if (static_cast<long long>(global_ns() - t0) > kWaitLimitNs) {
            atomicExch(stop, 1);
            return false;
        }
    }
    return true;
}

// Barrier of the 128 softmax threads, alone or with the OR of a predicate.
__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool soft_any(bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %1, 0;\n\t"
        "bar.red.or.pred q, 1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(v ? 1u : 0u)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u)
        : "memory");
}

// Descriptor of an MN-major operand in 128-byte swizzle atoms (64 elements x 8 k): atoms of
// the next 64 elements 8 KiB on (leading byte offset), of the next 8 k 1 KiB on (stride).
__device__ __forceinline__ uint64_t mn_desc(uint32_t addr) {
    return tc05::kDescHi | (static_cast<uint64_t>(kChunk >> 4) << 16) | static_cast<uint64_t>((addr & 0x3FFFFu) >> 4);
}

// 16 bytes global -> shared, asynchronously; zeros where `bytes` is 0.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, int c3,
                                       uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
}

// S^T of 64 keys x NT rows: lane l of the warp gets keys l / 4 and l / 4 + 8 of the warp's 16,
// and of each 8 rows the pair 2 (l % 4): s[4i], s[4i+1] of the first key, s[4i+2], s[4i+3] of
// the second.
__device__ __forceinline__ void tmem_ld_s(uint32_t addr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(addr));
}
__device__ __forceinline__ void tmem_ld_s(uint32_t addr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_ld_s(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// BF16 pairs with infinities and NaN set to 0.
__device__ __forceinline__ uint32_t finite_or_zero(uint32_t w) {
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0x0000ffffu;
    return w;
}

// ----------------------------------------------------------------------------- the kernel
template <int NT>
__global__ void __launch_bounds__(kThreads, 1) latent_attention_kernel(const __grid_constant__ LatentParams p) {
    constexpr int kSCols = NT;                    // tensor-memory columns of one S^T
    constexpr int kTmem = NT == 64 ? 512 : NT == 32 ? 256 : 128;
    constexpr int NC = NT / 4;                    // rows a softmax thread holds scores of
    constexpr uint32_t kIdescS = (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(NT >> 3) << 17) |
                                 (static_cast<uint32_t>(kTile >> 4) << 24);
    constexpr uint32_t kIdescO = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (1u << 16) |
                                 (static_cast<uint32_t>(NT >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[2 * kMaxSlots + 2 * kMaxRopeSlots + 11];
    __shared__ __align__(16) float ex[2][4][NT];   // a warp's maxima (or sums) of each row
    __shared__ __align__(16) float fs[NT], ms[NT];  // a row's factor for O^T; its maximum
    __shared__ long long off[NT];    // a row's place in out
    __shared__ int part[32], plan[3];
    __shared__ uint32_t tmem_slot;
    __shared__ int stop;

    uint8_t *base = smem_raw + ((1024u - (saddr(smem_raw) & 1023u)) & 1023u);
    const int pairs = p.R / 128;            // slots a tile
    const int qchunk = NT * 128;            // bytes of a chunk of Q
    const uint32_t s_q = saddr(base);
    const uint32_t s_p = s_q + (2 * pairs + 1) * qchunk;
    const uint32_t s_r = s_p + 2 * kChunk;
    const uint32_t s_v = s_r + p.rope_slots * kChunk;
    const int S = p.slots, RS = p.rope_slots;

    const uint32_t vfull = saddr(bars), vempty = vfull + 8 * kMaxSlots;
    const uint32_t rfull = vempty + 8 * kMaxSlots, rempty = rfull + 8 * kMaxRopeSlots;
    const uint32_t qfull = rempty + 8 * kMaxRopeSlots, qempty = qfull + 8;
    const uint32_t sfull = qempty + 8, sempty = sfull + 16, pfull = sempty + 16, pvd = pfull + 16, fin = pvd + 16;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = static_cast<int>(blockIdx.x) / p.rt, r = static_cast<int>(blockIdx.x) % p.rt;

    if (warp == 0) {
        if (lane == 0) {
            prefetch_tmap(&p.tv);
            prefetch_tmap(&p.tr);
            stop = 0;
            plan[2] = 0;
            for (int i = 0; i < kMaxSlots; ++i) {
                bar_init(vfull + 8 * i, 1);
                bar_init(vempty + 8 * i, 1);
            }
            for (int i = 0; i < kMaxRopeSlots; ++i) {
                bar_init(rfull + 8 * i, 1);
                bar_init(rempty + 8 * i, 1);
            }
            bar_init(qfull, 2);
            bar_init(qempty, 1);
            for (int i = 0; i < 2; ++i) {
                bar_init(sfull + 8 * i, 1);
                bar_init(sempty + 8 * i, 4);
                bar_init(pfull + 8 * i, 4);
                bar_init(pvd + 8 * i, 1);
            }
            bar_init(fin, 1);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        __syncwarp();
    }
    if (p.flags & kFlagPdl) pdl_wait();
    // Tensor memory is taken after the wait: a CTA of the previous kernel may still want its
    // own, and this one holds its columns until that kernel is done.
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&tmem_slot)),
                     "r"(kTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    __syncthreads();
    // this CTA's share of the line
    {
        const int per = (p.B + kThreads - 1) / kThreads;
        const int b0 = min(p.B, static_cast<int>(threadIdx.x) * per), b1 = min(p.B, b0 + per);
        int sum = 0, units;
        for (int b = b0; b < b1; ++b) {
            const Seq s = seq_of(p, b);
            if (s.bad && blockIdx.x == 0) atomicOr(p.err, kErrBadIndex);
            sum += tiles_of(s);
        }
        int at = block_prefix(sum, part, &units);
        const int ge = min(p.groups, max(units, 1));
        if (g < ge) {
            const int u0 = share_begin(units, g, ge), u1 = share_begin(units, g + 1, ge);
            if (u0 < u1 && u0 >= at && u0 < at + sum) {
                for (int b = b0; b < b1; ++b) {
                    const int kt = tiles_of(seq_of(p, b));
                    if (u0 < at + kt) {
                        plan[0] = b;
                        plan[1] = u0 - at;
                        plan[2] = u1 - u0;
                        break;
                    }
                    at += kt;
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_launch_dependents();
    const uint32_t tmem = tmem_slot;
    const uint32_t t_o = tmem + 2 * kSCols;
    Walk walk{plan[0], plan[1], plan[2]};
    const bool stall = (p.flags & kFlagTestStall) != 0;
    Piece o;
    int issued = 0, rissued = 0;  // slots of each ring that the producer filled

    if (warp == 0) {
        // ------------------------------------------------------------------- producer
        const int rows = min(kTile, p.page_size);       // rows of one copy
        const bool whole = rows == kTile;
        int n = 0;
        bool ok = true;
        while (ok && walk.next(p, r, o)) {
            const int *table = p.table + static_cast<long long>(o.b) * p.ldt;
            auto page_of = [&](int k) {
                // lane f: the page of the f-th copy of tile k (or the page past the last one,
                // which reads as zeros)
                const int key = k * kTile + (whole ? 0 : lane * rows);
                const bool in = whole ? key < o.s.len : lane < kTile / rows && key < o.s.len;
                if (!in || k >= o.k1) return p.pages;
                const int page = table[key / p.page_size];
                if (page < 0 || page >= p.pages) {
                    if (lane == 0 || !whole) atomicOr(p.err, kErrBadIndex);
                    return p.pages;
                }
                return page;
            };
            int next = o.k0 < o.k1 ? page_of(o.k0) : 0;
            for (int k = o.k0; ok && k < o.k1; ++k, ++n) {
                const int page = next;
                if (k + 1 < o.k1) next = page_of(k + 1);
                const int keys = min(kTile, o.s.len - k * kTile);
                const int nf = (keys + rows - 1) / rows;  // copies of each chunk
                const int row = whole ? (k * kTile) % p.page_size : 0;
                for (int j = 0; j < pairs; ++j) {
                    const int at = n * pairs + j, slot = at % S;
                    if (lane == 0) {
                        ok = at < S || wait_or_stop(vempty + 8 * slot, ((at / S) - 1) & 1, &stop);
                        if (ok) bar_expect_tx(vfull + 8 * slot, static_cast<unsigned>(2 * nf * rows * 128));
                    }
                    ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
                    if (!ok) break;
                    issued = stall ? 0 : at + 1;
                    if (stall) continue;
                    const uint32_t dst = s_v + slot * kSlot;
                    if (whole) {
                        if (lane == 0) tma_4d(dst, &p.tv, 0, row, 2 * j, page, vfull + 8 * slot);
                    } else {
                        const int f = lane % nf, c = lane / nf;
                        const int pg = __shfl_sync(0xffffffffu, page, f);
                        if (c < 2) tma_4d(dst + c * kChunk + f * rows * 128, &p.tv, 0, 0, 2 * j + c, pg, vfull + 8 * slot);
                    }
                }
                if (!ok) break;
                const int slot = n % RS;
                if (lane == 0) {
                    ok = n < RS || wait_or_stop(rempty + 8 * slot, ((n / RS) - 1) & 1, &stop);
                    if (ok) bar_expect_tx(rfull + 8 * slot, static_cast<unsigned>(nf * rows * 128));
                }
                ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
                if (!ok) break;
                rissued = stall ? 0 : n + 1;
                if (!stall && lane < (whole ? 1 : nf))
                    tma_3d(s_r + slot * kChunk + lane * rows * 128, &p.tr, 0, row, page, rfull + 8 * slot);
            }
        }
    } else if (warp == 1) {
        // --------------------------------------------------------------- the products
        if (lane == 0) {
            int ns = 0, no = 0;  // tiles whose S^T, whose O^T is issued
            int step = 0, tile = 0, piece = -1;
            unsigned opens = 0;  // bit (tile & 3): the first tile of its piece, O^T starts anew
            bool have = false, more = true, idle = false;
            unsigned long long t0 = 0;
            while (more || have || no < ns) {
                bool did = false;
                if (no < ns && bar_test(pfull + 8 * (no & 1), (no >> 1) & 1)) {
                    tc_fence_after();
                    const uint32_t pb = s_p + (no & 1) * kChunk;
                    const bool open = (opens >> (no & 3)) & 1;
                    for (int j = 0; j < pairs; ++j) {
                        const int slot = (no * pairs + j) % S;
                        const uint32_t a = s_v + slot * kSlot;
#pragma unroll
                        for (int kk = 0; kk < kTile / 16; ++kk)
                            mma(t_o + j * NT, mn_desc(a + kk * 2048), mn_desc(pb + kk * 2048), kIdescO, !(open && kk == 0));
                        mma_commit(vempty + 8 * slot);
                    }
                    mma_commit(pvd + 8 * (no & 1));
                    ++no;
                    did = true;
                }
                if (more && !have) {
                    more = walk.next(p, r, o);
                    if (more && o.k0 < o.k1) {
                        have = true;
                        tile = o.k0;
                        ++piece;
                    }
                    did = true;
                }
                if (have) {
                    bool ready = true;
                    if (step == 0)
                        ready = (ns < 2 || bar_test(sempty + 8 * (ns & 1), ((ns >> 1) - 1) & 1)) &&
                                (tile != o.k0 || bar_test(qfull, piece & 1));
                    const int at = ns * pairs + step;
                    if (ready)
                        ready = step < pairs ? bar_test(vfull + 8 * (at % S), (at / S) & 1)
                                             : bar_test(rfull + 8 * (ns % RS), (ns / RS) & 1);
                    if (ready) {
                        tc_fence_after();
                        const uint32_t d = tmem + (ns & 1) * kSCols;
                        const uint32_t a = step < pairs ? s_v + (at % S) * kSlot : s_r + (ns % RS) * kChunk;
                        const uint32_t b = s_q + 2 * step * qchunk;
                        const int chunks = step < pairs ? 2 : 1;
                        for (int c = 0; c < chunks; ++c)
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                mma(d, tc05::sw128_desc(a + c * kChunk + 32 * kk), tc05::sw128_desc(b + c * qchunk + 32 * kk),
                                    kIdescS, (step | c | kk) != 0);
                        if (++step > pairs) {
                            mma_commit(rempty + 8 * (ns % RS));
                            mma_commit(sfull + 8 * (ns & 1));
                            if (tile + 1 == o.k1) mma_commit(qempty);
                            opens = (opens & ~(1u << (ns & 3))) | (tile == o.k0 ? 1u << (ns & 3) : 0u);
                            ++ns;
                            step = 0;
                            if (++tile == o.k1) have = false;
                        }
                        did = true;
                    }
                }
                if (did) {
                    idle = false;
                } else if (!idle) {
                    idle = true;
                    t0 = global_ns();
                } else if (*reinterpret_cast<volatile int *>(&stop)) {
                    break;
                } else if (static_cast<long long>(global_ns() - t0) > kWaitLimitNs) {
                    atomicExch(&stop, 1);
                    break;
                }
            }
            // every product issued is complete before the tensor memory is given back
            mma_commit(fin);
            const unsigned long long w0 = global_ns();
            while (!bar_try(fin, 0))
                if (static_cast<long long>(global_ns() - w0) > kWaitLimitNs) {
                    atomicExch(&stop, 1);
                    break;
                }
        }
    } else if (warp < 6) {
        // ------------------------------------------------------------------- softmax
        const int sw = warp & 3;  // tensor-memory lanes 32 sw .. and keys 16 sw .. of a tile
        const int tid = threadIdx.x - 64;
        const int c0 = 2 * (lane & 3);
        const uint32_t quarter = static_cast<uint32_t>(32 * sw) << 16;
        const float inf = __int_as_float(0x7f800000), nan = __int_as_float(0x7fc00000);
        int n = 0;
        bool ok = true, dead = false;
        while (walk.next(p, r, o)) {
            float m[NC], l[NC];
            int lim[NC];  // keys a row sees
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int col = 8 * (c >> 1) + c0 + (c & 1);
                m[c] = -inf;
                l[c] = 0.0f;
                lim[c] = col < o.nrows ? o.s.len - o.s.n_all + (o.row0 + col) / p.H + 1 : 0;
            }
            const int lim_min = max(0, o.s.len - o.s.n_all + o.row0 / p.H + 1);
            for (int k = o.k0; k < o.k1 && !dead; ++k, ++n) {
                ok = wait_or_stop(sfull + 8 * (n & 1), (n >> 1) & 1, &stop) && ok;
                ok = __all_sync(0xffffffffu, ok);
                uint32_t sr[4 * (NT / 8)];
                float s[4 * (NT / 8)];
                if (ok) {
                    tc_fence_after();
                    tmem_ld_s(tmem + quarter + (n & 1) * kSCols, sr);
                    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) bar_arrive(sempty + 8 * (n & 1));
                const int key = k * kTile + 16 * sw + (lane >> 2);
                const bool edge = (k + 1) * kTile > lim_min || o.nrows < NT;
                bool over = !ok;
#pragma unroll
                for (int i = 0; i < NT / 8; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int c = 2 * i + (e & 1);
                        float v = ok ? __uint_as_float(sr[4 * i + e]) * p.scale_log2 : 0.0f;
                        if (edge && key + 8 * (e >> 1) >= lim[c]) v = -inf;
                        s[4 * i + e] = v;
                        over |= v > m[c] + 8.0f;
                    }
                if (soft_any(over)) {
                    if (soft_any(!ok)) {
                        dead = true;
                        break;
                    }
                    float f[NC];
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        const int i = c >> 1, e = c & 1;
                        float v = fmaxf(s[4 * i + e], s[4 * i + 2 + e]);
#pragma unroll
                        for (int d = 4; d <= 16; d <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
                        f[c] = v;
                    }
                    if (lane < 4)
#pragma unroll
                        for (int i = 0; i < NT / 8; ++i)
                            *reinterpret_cast<float2 *>(&ex[n & 1][sw][8 * i + c0]) = make_float2(f[2 * i], f[2 * i + 1]);
                    soft_sync();
#pragma unroll
                    for (int i = 0; i < NT / 8; ++i) {
                        float2 v = make_float2(m[2 * i], m[2 * i + 1]);
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            const float2 x = *reinterpret_cast<const float2 *>(&ex[n & 1][w][8 * i + c0]);
                            v.x = fmaxf(v.x, x.x);
                            v.y = fmaxf(v.y, x.y);
                        }
                        const float nm[2] = {v.x, v.y};
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int c = 2 * i + e;
                            f[c] = nm[e] == m[c] ? 1.0f : ex2(m[c] - nm[e]);  // 0 from -inf
                            l[c] *= f[c];
                            m[c] = nm[e];
                        }
                    }
                    if (k > o.k0) {
                        // O^T of the tiles before: complete, then scaled in place
                        if (sw == 0 && lane < 4)
#pragma unroll
                            for (int i = 0; i < NT / 8; ++i)
                                *reinterpret_cast<float2 *>(&fs[8 * i + c0]) = make_float2(f[2 * i], f[2 * i + 1]);
                        ok = wait_or_stop(pvd + 8 * ((n - 1) & 1), ((n - 1) >> 1) & 1, &stop) && ok;
                        soft_sync();
                        tc_fence_after();
                        for (int c = 0; c < pairs * NT; c += 16) {
                            uint32_t v[16];
                            tmem_ld16(t_o + quarter + c, v);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                v[i] = __float_as_uint(__uint_as_float(v[i]) * fs[(c + i) % NT]);
                            tmem_st16(t_o + quarter + c, v);
                        }
                        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                        tc_fence_before();
                    }
                }
                if ((k + 1) * kTile > lim_min) {
                    // Rows of the tile that some query row does not see get weight 0; what they
                    // hold must not turn that into NaN: rows past the sequence's end (never
                    // copied, or left over in the page) become 0, infinities and NaN of others 0.
                    const int r0 = max(0, lim_min - k * kTile), end = o.s.len - k * kTile;
                    const int units = 2 * pairs * 8;
                    for (int i = tid; i < (kTile - r0) * units; i += 128) {
                        const int row = r0 + i / units, u = i % units, c = u >> 3;
                        uint8_t *at = base + (s_v - s_q) + ((n * pairs + (c >> 1)) % S) * kSlot + (c & 1) * kChunk +
                                      row * 128 + (u & 7) * 16;
                        uint4 v = make_uint4(0u, 0u, 0u, 0u);
                        if (row < end) {
                            v = *reinterpret_cast<const uint4 *>(at);
                            v.x = finite_or_zero(v.x);
                            v.y = finite_or_zero(v.y);
                            v.z = finite_or_zero(v.z);
                            v.w = finite_or_zero(v.w);
                        }
                        *reinterpret_cast<uint4 *>(at) = v;
                    }
                }
                // the weights, BF16 (their sum keeps FP32), into the buffer that tile n - 2 used
                if (n >= 2) ok = wait_or_stop(pvd + 8 * (n & 1), ((n >> 1) - 1) & 1, &stop) && ok;
                {
                    const int key_in = 16 * sw + (lane >> 2);
                    uint8_t *row = base + (s_p - s_q) + (n & 1) * kChunk + key_in * 128;
#pragma unroll
                    for (int i = 0; i < NT / 8; ++i) {
                        float w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int c = 2 * i + (e & 1);
                            w[e] = ex2(s[4 * i + e] - (m[c] == -inf ? 0.0f : m[c]));
                            l[c] += w[e];
                        }
                        const int at = ((i ^ (lane >> 2)) << 4) + 2 * c0;  // key_in % 8 = lane / 4
                        *reinterpret_cast<uint32_t *>(row + at) = bf16x2(w[0], w[1]);
                        *reinterpret_cast<uint32_t *>(row + 8 * 128 + at) = bf16x2(w[2], w[3]);
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) bar_arrive(pfull + 8 * (n & 1));
            }
            // ---------------------------------------------------------- the piece's result
            if (!dead && o.k0 < o.k1) {
                ok = wait_or_stop(pvd + 8 * ((n - 1) & 1), ((n - 1) >> 1) & 1, &stop) && ok;
                tc_fence_after();
            }
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int d = 4; d <= 16; d <<= 1) l[c] += __shfl_xor_sync(0xffffffffu, l[c], d);
            if (lane < 4)
#pragma unroll
                for (int i = 0; i < NT / 8; ++i) {
                    *reinterpret_cast<float2 *>(&ex[n & 1][sw][8 * i + c0]) = make_float2(l[2 * i], l[2 * i + 1]);
                    if (sw == 0) *reinterpret_cast<float2 *>(&ms[8 * i + c0]) = make_float2(m[2 * i], m[2 * i + 1]);
                }
            dead = soft_any(!ok || dead);
            const bool direct = o.first && o.last;
            float *ws = p.ws + (static_cast<long long>(blockIdx.x) * 2 + (o.first ? 1 : 0)) * NT * (p.R + 2);
            if (tid < NT) {
                const float sum = (ex[n & 1][0][tid] + ex[n & 1][1][tid]) + (ex[n & 1][2][tid] + ex[n & 1][3][tid]);
                const int row = o.row0 + tid, tok = o.s.q0 + row / p.H, head = row % p.H;
                if (direct) {
                    fs[tid] = dead ? nan : sum == 0.0f ? 0.0f : 1.0f / sum;
                    off[tid] = tok * p.out_token + head * p.out_head;
                    if (p.lse && tid < o.nrows)
                        p.lse[tok * p.lse_token + head] =
                            dead ? nan : sum == 0.0f ? -inf : (ms[tid] + log2f(sum)) * 0.69314718056f;
                } else {
                    // a NaN score leaves the maximum alone: the piece's is then NaN itself, so
                    // that joining keeps it whatever the maximum
                    ws[NT * p.R + tid] = dead || sum != sum ? nan : ms[tid];
                    ws[NT * p.R + NT + tid] = dead ? nan : sum;
                }
            }
            soft_sync();
            const bool empty = o.k0 >= o.k1;
            if (direct || !(empty || dead)) {
                for (int c = 0; c < pairs * NT; c += 16) {
                    uint32_t v[16];
                    if (empty || dead) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(dead ? nan : 0.0f);
                    } else {
                        tmem_ld16(t_o + quarter + c, v);
                    }
                    const int d = (c / NT) * 128 + 32 * sw + lane, col = c % NT;
                    if (direct) {
                        // two lanes exchange, so that each stores a pair of elements of one row
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            const float a = __uint_as_float(v[i]) * fs[col + i], b = __uint_as_float(v[i + 1]) * fs[col + i + 1];
                            const bool odd = lane & 1;
                            const float got = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
                            const int row = col + i + (odd ? 1 : 0);
                            if (row < o.nrows)
                                *reinterpret_cast<uint32_t *>(p.out + off[row] + (d & ~1)) = odd ? bf16x2(got, b) : bf16x2(a, got);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (col + i < o.nrows) ws[static_cast<long long>(col + i) * p.R + d] = __uint_as_float(v[i]);
                    }
                }
                tc_fence_before();
            }
            soft_sync();  // fs, off and ex are used again
        }
    } else {
        // ------------------------------------------------------------------ queries
        const int tid = threadIdx.x - 192;
        const int units = (2 * pairs + 1) * 8, width = p.R + p.E;
        int piece = 0;
        while (walk.next(p, r, o)) {
            if (o.k0 >= o.k1) continue;
            if (!__all_sync(0xffffffffu, piece == 0 || wait_or_stop(qempty, (piece - 1) & 1, &stop))) break;
            for (int i = tid; i < NT * units; i += 64) {
                const int row = i / units, u = i % units;
                // rows past the piece and elements past the width are 0
                const bool in = row < o.nrows && 8 * u < width;
                const int rr = in ? o.row0 + row : o.row0;
                const uint16_t *src = p.q + (o.s.q0 + rr / p.H) * p.q_token + (rr % p.H) * p.q_head + (in ? 8 * u : 0);
                copy16(s_q + (u >> 3) * qchunk + row * 128 + (((u & 7) ^ (row & 7)) << 4), src, in ? 16 : 0);
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) bar_arrive(qfull);
            ++piece;
        }
    }
    __syncwarp();
    // a producer that was stopped: its copies have landed before the shared memory goes
    if (warp == 0 && lane == 0 && *reinterpret_cast<volatile int *>(&stop)) {
        const unsigned long long w0 = global_ns();
        for (int i = max(0, issued - S); i < issued; ++i)
            while (!bar_try(vfull + 8 * (i % S), (i / S) & 1))
                if (static_cast<long long>(global_ns() - w0) > kWaitLimitNs) break;
        for (int i = max(0, rissued - RS); i < rissued; ++i)
            while (!bar_try(rfull + 8 * (i % RS), (i / RS) & 1))
                if (static_cast<long long>(global_ns() - w0) > kWaitLimitNs) break;
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && stop) atomicOr(p.err, 1);
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmem) : "memory");
    }
}

// ------------------------------------------------------------------ joining partial results
// One block takes one row of one sequence that several shares hold a piece of: cw warps wide
// (128 elements each), pw warps taking every pw-th piece, added in that order.
__global__ void __launch_bounds__(512) latent_join_kernel(const __grid_constant__ LatentParams p) {
    __shared__ int part[32], found[3];
    __shared__ __align__(16) float acc[16][128];
    __shared__ float lsum[16];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) found[0] = -1;
    __syncthreads();
    pdl_launch_dependents();
    const int per = (p.B + static_cast<int>(blockDim.x) - 1) / static_cast<int>(blockDim.x);
    const int b0 = min(p.B, static_cast<int>(threadIdx.x) * per), b1 = min(p.B, b0 + per);
    int sum = 0, units;
    for (int b = b0; b < b1; ++b) sum += tiles_of(seq_of(p, b));
    int at = block_prefix(sum, part, &units);
    const int ge = min(p.groups, max(units, 1));
    const int seg = blockIdx.x;
    // by sequence: the seg-th sequence; else the one that share seg + 1 begins inside of, if it
    // is the first share to do so
    const int u = p.by_seq ? 0 : (seg + 1 < ge ? share_begin(units, seg + 1, ge) : units);
    for (int b = b0; b < b1; ++b) {
        const int kt = tiles_of(seq_of(p, b));
        if (p.by_seq ? b == seg : (u > at && u < at + kt && share_begin(units, seg, ge) <= at)) {
            found[0] = b;
            found[1] = at;
            found[2] = kt;
        }
        at += kt;
    }
    __syncthreads();
    pdl_wait();
    if (found[0] < 0 || found[2] == 0) return;
    const int begin = found[1], end = found[1] + found[2];
    // first and last share that hold a tile of it
    int g0 = static_cast<int>(static_cast<long long>(begin) * ge / units);
    while (g0 + 1 < ge && share_begin(units, g0 + 1, ge) <= begin) ++g0;
    while (share_begin(units, g0, ge) > begin) --g0;
    int g1 = static_cast<int>(static_cast<long long>(end - 1) * ge / units);
    while (g1 + 1 < ge && share_begin(units, g1 + 1, ge) <= end - 1) ++g1;
    while (share_begin(units, g1, ge) > end - 1) --g1;
    if (g0 == g1) return;
    const Seq s = seq_of(p, found[0]);
    const int rr = blockIdx.y, r = rr / p.nt, i = rr % p.nt;
    if (rr >= s.n * p.H) return;

    const long long size = static_cast<long long>(p.nt) * (p.R + 2);
    auto slot = [&](int g) { return p.ws + ((static_cast<long long>(g) * p.rt + r) * 2 + (g == g0 ? 1 : 0)) * size; };
    const float inf = __int_as_float(0x7f800000);
    float top = -inf;
    for (int g = g0 + lane; g <= g1; g += 32) top = fmaxf(top, slot(g)[p.nt * p.R + i]);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    if (top == -inf) top = 0.0f;
    const int wp = warp / p.cw, col = (blockIdx.z * p.cw + warp % p.cw) * 128 + 4 * lane;
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float l = 0.0f;
#pragma unroll 4
    for (int g = g0 + wp; g <= g1; g += p.pw) {
        const float *w = slot(g);
        const float f = ex2(w[p.nt * p.R + i] - top);  // 0 for a piece without a key
        const float4 v = *reinterpret_cast<const float4 *>(w + static_cast<long long>(i) * p.R + col);
        if (f != 0.0f) {
            l = fmaf(f, w[p.nt * p.R + p.nt + i], l);
            a.x = fmaf(f, v.x, a.x);
            a.y = fmaf(f, v.y, a.y);
            a.z = fmaf(f, v.z, a.z);
            a.w = fmaf(f, v.w, a.w);
        }
    }
    *reinterpret_cast<float4 *>(&acc[warp][4 * lane]) = a;
    if (lane == 0) lsum[warp] = l;
    __syncthreads();
    if (wp > 0) return;
    for (int w = 1; w < p.pw; ++w) {
        const float4 v = *reinterpret_cast<const float4 *>(&acc[w * p.cw + warp][4 * lane]);
        a.x += v.x;
        a.y += v.y;
        a.z += v.z;
        a.w += v.w;
        l += lsum[w * p.cw + warp];
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const long long tok = s.q0 + rr / p.H, head = rr % p.H;
    uint32_t *out = reinterpret_cast<uint32_t *>(p.out + tok * p.out_token + head * p.out_head + col);
    out[0] = bf16x2(a.x * inv, a.y * inv);
    out[1] = bf16x2(a.z * inv, a.w * inv);
    if (p.lse && col == 0) p.lse[tok * p.lse_token + head] = l == 0.0f ? -inf : (top + log2f(l)) * 0.69314718056f;
}

const void *kernel_of(int nt) {
    return nt == 64   ? reinterpret_cast<const void *>(&latent_attention_kernel<64>)
           : nt == 32 ? reinterpret_cast<const void *>(&latent_attention_kernel<32>)
                      : reinterpret_cast<const void *>(&latent_attention_kernel<16>);
}

// The sizes of a call: rows a CTA, CTAs a group, groups.
struct Split {
    int nt, rt, groups;
    long long ws_bytes;
};

Split split_of(const sgemm_latent_attention_t &a, int sms) {
    Split s;
    const long long rows = static_cast<long long>(a.max_q) * a.H;
    s.nt = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
    s.rt = static_cast<int>((rows + s.nt - 1) / s.nt);
    const long long tiles = std::max(1LL, (static_cast<long long>(a.table_width) * a.page_size + kTile - 1) / kTile);
    s.groups = static_cast<int>(std::max(1LL, std::min<long long>(sms / s.rt, tiles * a.B)));
    s.ws_bytes = s.groups > 1 ? static_cast<long long>(s.groups) * s.rt * 2 * s.nt * (a.R + 2) * 4 : 0;
    return s;
}

sgemm_status_t check_sizes(const sgemm_latent_attention_t &a) {
    if (a.flags & ~(kDecodeFlags | SGEMM_FLAG_TEST_STALL)) return SGEMM_ERR_INVALID_ARG;
    if (a.B < 0 || a.total_q < 0 || a.H < 1 || a.H > 1024 || a.max_q < 1 || a.table_width < 0 || a.pages < 1 ||
        a.page_size < 1 || a.R < 1 || a.E < 1)
        return SGEMM_ERR_INVALID_ARG;
    if (a.R % 128 || a.R > 512 || a.E % 8 || a.E > 64) return SGEMM_ERR_UNSUPPORTED_SHAPE;
    if (a.page_size != 8 && a.page_size != 16 && a.page_size != 32 && a.page_size % 64) return SGEMM_ERR_UNSUPPORTED_SHAPE;
    // counts that the kernel keeps in 32 bits
    const long long big = 1LL << 30;
    if (a.pages >= big || a.total_q >= big || static_cast<long long>(a.max_q) * a.H >= big ||
        static_cast<long long>(a.max_q) * a.B >= big || static_cast<long long>(a.table_width) * a.page_size >= big ||
        (static_cast<long long>(a.table_width) * a.page_size / kTile + 2) * a.B >= big)
        return SGEMM_ERR_UNSUPPORTED_SHAPE;
    return SGEMM_OK;
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *q = nullptr;
        cudaDriverEntryPointQueryResult res;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &q, 12000, cudaEnableDefault, &res) !=
                cudaSuccess ||
            res != cudaDriverEntryPointSuccess)
            q = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(q);
    }();
    return fn;
}

bool encode_maps(LatentParams &p, const sgemm_latent_attention_t &a) {
    auto enc = encoder();
    if (!enc) return false;
    const cuuint32_t rows = static_cast<cuuint32_t>(std::min(kTile, a.page_size));
    const cuuint64_t ps = static_cast<cuuint64_t>(a.page_size), pages = static_cast<cuuint64_t>(a.pages);
    const cuuint64_t rs = static_cast<cuuint64_t>(a.row_stride) * 2, pg = static_cast<cuuint64_t>(a.page_stride) * 2;
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    {
        const cuuint64_t dims[4] = {64, ps, static_cast<cuuint64_t>(a.R / 64), pages};
        const cuuint64_t strides[3] = {rs, 128, pg};
        const cuuint32_t box[4] = {64, rows, rows == kTile ? 2u : 1u, 1};
        if (enc(&p.tv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t *>(a.cache), dims, strides, box, ones,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return false;
    }
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(a.E), ps, pages};
    const cuuint64_t strides[2] = {rs, pg};
    const cuuint32_t box[3] = {64, rows, 1};
    return enc(&p.tr, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t *>(a.cache) + a.R, dims, strides, box, ones,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace latent
}  // namespace sk

extern "C" sgemm_status_t sgemm_latent_attention_workspace(const sgemm_latent_attention_t *a, long long *bytes) {
    using namespace sk;
    if (!a || !bytes) return SGEMM_ERR_INVALID_ARG;
    *bytes = 0;
    sgemm_status_t st = latent::check_sizes(*a);
    if (st != SGEMM_OK) return st;
    if (a->B == 0 || a->total_q == 0) return SGEMM_OK;
    int sms = 0, *err = nullptr;
    st = device_ready(&sms, &err);
    if (st != SGEMM_OK) return st;
    *bytes = latent::split_of(*a, sms).ws_bytes;
    return SGEMM_OK;
}

extern "C" sgemm_status_t sgemm_bf16_latent_attention(const sgemm_latent_attention_t *a, sgemm_stream_t stream) {
    using namespace sk;
    using namespace sk::latent;
    if (!a) return SGEMM_ERR_INVALID_ARG;
    sgemm_status_t st = check_sizes(*a);
    if (st != SGEMM_OK) return st;
    if (a->B == 0 || a->total_q == 0) return SGEMM_OK;
    const long long W = a->R + a->E;
    if (!a->q || !a->cache || !a->block_table || !a->seq_lens || !a->out) return SGEMM_ERR_INVALID_ARG;
    if (!a->cu_q && a->total_q != static_cast<long long>(a->B) * a->max_q) return SGEMM_ERR_INVALID_ARG;
    if (a->ldt < a->table_width || a->row_stride < W || a->page_stride < (a->page_size - 1) * a->row_stride + W ||
        a->q_token < 0 || a->q_head < 0 || a->workspace_bytes < 0 || std::isnan(a->scale) || std::isinf(a->scale))
        return SGEMM_ERR_INVALID_ARG;
    {
        // no two rows of out may share elements
        const long long none = 1LL << 62;
        const long long tok = a->total_q == 1 ? none : a->out_token, head = a->H == 1 ? none : a->out_head;
        const long long lo = std::min(tok, head), hi = std::max(tok, head), n = tok <= head ? a->total_q : a->H;
        if (lo < a->R || (hi != none && hi < (n - 1) * lo + a->R)) return SGEMM_ERR_INVALID_ARG;
        if (a->lse && a->total_q > 1 && a->lse_token < a->H) return SGEMM_ERR_INVALID_ARG;
    }
    if (!aligned(a->q, 16) || a->q_token % 8 || a->q_head % 8 || !aligned(a->cache, 16) || a->row_stride % 8 ||
        a->page_stride % 8 || !aligned(a->out, 4) || a->out_token % 2 || a->out_head % 2 || !aligned(a->lse, 4) ||
        !aligned(a->block_table, 4) || !aligned(a->seq_lens, 4) || !aligned(a->cu_q, 4) || !aligned(a->workspace, 16))
        return SGEMM_ERR_MISALIGNED;
    // strides that a tensor map can hold
    if (a->row_stride >= (1LL << 38) || a->page_stride >= (1LL << 38)) return SGEMM_ERR_UNSUPPORTED_SHAPE;

    LatentParams p;
    std::memset(&p, 0, sizeof(p));
    int sms = 0;
    st = device_ready(&sms, &p.err);
    if (st != SGEMM_OK) return st;
    const Split sp = split_of(*a, sms);
    if (sp.ws_bytes > 0 && (!a->workspace || a->workspace_bytes < sp.ws_bytes)) return SGEMM_ERR_NO_WORKSPACE;
    if (!encode_maps(p, *a)) return SGEMM_ERR_CUDA;
    p.q = a->q;
    p.table = a->block_table;
    p.lens = a->seq_lens;
    p.cu_q = a->cu_q;
    p.out = a->out;
    p.lse = a->lse;
    p.ws = static_cast<float *>(a->workspace);
    p.q_token = a->q_token;
    p.q_head = a->q_head;
    p.ldt = a->ldt;
    p.out_token = a->out_token;
    p.out_head = a->out_head;
    p.lse_token = a->lse_token;
    p.total_q = a->total_q;
    p.pages = static_cast<int>(a->pages);
    p.page_size = a->page_size;
    p.width = a->table_width;
    p.B = a->B;
    p.H = a->H;
    p.R = a->R;
    p.E = a->E;
    p.max_q = a->max_q;
    p.nt = sp.nt;
    p.rt = sp.rt;
    p.groups = sp.groups;
    p.scale_log2 = static_cast<float>(static_cast<double>(a->scale) * 1.4426950408889634);
    p.flags = static_cast<int>(a->flags);

    const int fixed = (a->R / 64 + 1) * sp.nt * 128 + 2 * kChunk + 1024;
    p.rope_slots = sp.nt == 64 ? 2 : 3;
    const int room = static_cast<int>(kMaxSmemOptin) - kStaticSmem - fixed - p.rope_slots * kChunk;
    p.slots = std::min(kMaxSlots, room / kSlot);
    const int smem = fixed + p.rope_slots * kChunk + p.slots * kSlot;
    const void *fn = kernel_of(sp.nt);
    {
        // once per kernel and device: allow the shared memory
        static std::atomic<unsigned long long> done[3];
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return SGEMM_ERR_CUDA;
        std::atomic<unsigned long long> &d = done[sp.nt == 64 ? 2 : sp.nt == 32 ? 1 : 0];
        const unsigned long long bit = dev < 64 ? 1ULL << dev : 0ULL;
        if (!(d.load(std::memory_order_acquire) & bit)) {
            if (allow_max_dynamic_smem(fn) != cudaSuccess) return SGEMM_ERR_CUDA;
            d.fetch_or(bit, std::memory_order_release);
        }
    }
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (launch(fn, dim3(static_cast<unsigned>(sp.groups * sp.rt)), dim3(kThreads), static_cast<size_t>(smem), cs,
               (a->flags & SGEMM_FLAG_PDL) != 0, &p) != cudaSuccess)
        return SGEMM_ERR_CUDA;
    if (sp.groups == 1) return SGEMM_OK;
    // sequences that may be split: each at most once by sequence, or by the shares' beginnings
    p.by_seq = a->B < sp.groups ? 1 : 0;
    p.nseg = p.by_seq ? a->B : sp.groups - 1;
    const int parts = p.by_seq ? (sp.groups + a->B - 1) / a->B + 1 : 2;
    const int blocks = a->R / 128;
    p.cw = parts > 16 ? 1 : blocks;
    p.pw = parts > 16 ? 16 : parts > 4 ? 4 : parts > 2 ? 2 : 1;
    const dim3 grid(static_cast<unsigned>(p.nseg),
                    static_cast<unsigned>(std::min<long long>(static_cast<long long>(sp.rt) * sp.nt,
                                                              static_cast<long long>(a->max_q) * a->H)),
                    static_cast<unsigned>(blocks / p.cw));
    if (launch(reinterpret_cast<const void *>(&latent_join_kernel), grid, dim3(static_cast<unsigned>(32 * p.cw * p.pw)), 0,
               cs, true, &p) != cudaSuccess)
        return SGEMM_ERR_CUDA;
    return SGEMM_OK;
}
