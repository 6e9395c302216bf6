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
//  * Warp 0 and the last one stream the tiles with TMA into a ring of slots (two
//    chunks, 128 latent elements, a slot; the E elements in a ring of their
//    own).  Slots rather than tiles: a slot is free again as soon as its part of O^T is
//    done, and what is left of shared memory beside Q holds 2 to 2.5 tiles.
//  * Warp 1 issues the first product (and copies the queries), the last but one
//    the second.  Two warps, because neither may wait for the other's operands:
//    O^T of tile t is issued as soon as its weights are there, which frees the
//    tile's slots, and S^T of tile t + 1 as its slots arrive.  (In an early
//    form, 64 sequences of up to 8192: 115 us, 127 with one warp for both.)
//  * Warps 2..5 (2..9 with 64 rows) do the softmax: S^T is read in the 16 x
//    256-bit form, so that all lanes hold scores though M = 64 fills half of the
//    lanes.  The running
//    maximum of a row is over keys, which lie across lanes and warps; it is
//    exchanged only in tiles where some score exceeds the maximum in use by
//    more than 2^8 (in units of the result), else the old one stands: one
//    barrier with a vote a tile.  The weights are then at most 2^8, and neither
//    their rounding to BF16 nor the FP32 sums care about that factor.
//
// Work split.  The tiles of all sequences form one line, cut into equal shares,
// one for each group of CTAs (a group has a CTA for each NT rows of a sequence
// with max_q tokens, so that these read a tile at about the same time and the
// L2 cache serves all but the first).  The lengths are on the device, so each
// CTA finds its share itself.  A sequence that a share ends in leaves partial
// results (FP32 O, m and l), which a second kernel joins in the order of the
// shares: the result does not depend on timing.
// The CTAs of a group are those of the sequence with the most new tokens, and the
// groups what the SMs then hold: sequences with fewer tokens leave CTAs of their
// groups idle, and where a group needs more than half of the SMs there is one, which
// walks every sequence whole.  128 heads, 64 sequences of 8192: 194 us; with 8 new
// tokens in one of them 1.4 ms, with 39 12.6 ms.
//
// Measured on one GB300, calls one after the other, 512 + 64 elements:
//   32 heads, 64 sequences of up to 8192 (378 MB)    74.0 us  5.1 TB/s
//   32 heads, one sequence of 131072 (151 MB)        36.7 us  4.1 TB/s
//   128 heads, 32 sequences of 8192 (73 GFLOP)      105.6 us  0.69 PFLOP/s
//   20 heads, 8 x 8 tokens, up to 4099 rows          24.7 us
//   32 heads, one sequence of 1000                   10.8 us
// A tile more a CTA costs 1.76 us with 32 heads, 0.94 of the measured copy rate
// for all SMs; with 128 heads 1.59 us (1.55 from the L2 cache), of which the
// MMAs are 1.0: there the ring's turn (copy, S^T, softmax, O^T, with two tiles in
// flight) bounds it.  Beside the tiles a call costs 10 to 20 us: the start until
// the first copies land, the pieces' results, the joining kernel.
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
constexpr int kRopeSlots = 2;  // (3: the same times)
// Warps: copies, first product, 4 soft_parts of softmax, second product, copies.
__host__ __device__ constexpr int soft_parts(int nt) { return nt == 64 ? 2 : 1; }
// Buffers of weights, 8 KiB each.  With 64 rows one: it is read long before it is written again,
// and what it frees holds a second slot of rotated elements beside two whole tiles of latent ones.
__host__ __device__ constexpr int weight_buffers(int nt) { return nt == 64 ? 1 : 2; }
__host__ __device__ constexpr int threads_of(int nt) { return 128 + 128 * soft_parts(nt); }
constexpr int kPieceCost = 1;            // see tiles_of (1: verification of 8 sequences 25.0 us; 0: 26.6; 2: 25.2)
constexpr float kLazy = 8.0f;            // log2 of the largest weight before a maximum moves
constexpr float kNoMax = -3.4028234e38f;  // no score is smaller: the maximum of none
constexpr int kMaxCopies = 8;            // copies of a chunk of a tile: pages of at least 8 rows
constexpr int kBarBytes = 384;           // the mbarriers

// Division by a number of the call, exact for 0 <= n < 2^30: n m / 2^s with m = ceil(2^s / d),
// s = 30 + ceil(log2 d).  (A division by a number the compiler does not know takes 100 cycles and
// more, and the warps here wait for a chain of them before the first copy.)
struct Divisor {
    unsigned m;
    int s, d;
    static Divisor of(int d) {
        int l = 0;
        while ((1LL << l) < d) ++l;
        return {static_cast<unsigned>(((1ULL << (30 + l)) + d - 1) / d), 30 + l, d};
    }
    __device__ __forceinline__ int div(int n) const {
        return static_cast<int>((static_cast<unsigned long long>(static_cast<unsigned>(n)) * m) >> s);
    }
    __device__ __forceinline__ int mod(int n) const { return n - div(n) * d; }
};

struct LatentParams {
    CUtensorMap tv;  // the latent part: {64, page rows, R / 64, pages}
    CUtensorMap tr;  // the rotated part: {E, page rows, pages}
    CUtensorMap qv, qr;  // the same parts of the queries, where (token, head) rows are evenly spaced
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
    int cost;               // kPieceCost, or 0 for a short line
    int slots;    // of latent elements in the ring
    Divisor heads, ctas, shares;  // by H, by rt, by groups
    Divisor page_tiles;     // by the tiles of a page (pages of whole tiles)
    int row_shift;          // log2 of the rows of one copy: of a tile, or of a page where that is smaller
    float scale_log2;       // scale * log2(e)
    int flags;
    int q_even;   // the queries' rows are evenly spaced: copied with TMA
    int out16;    // out's rows start on 16 bytes
    int by_seq;   // descriptors of split sequences: one a sequence, else one a group
    int pw;       // warps of the joining kernel that share a sequence's pieces
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

// Length of a sequence on the line: its tiles, and before them what turning to it costs a CTA
// (its queries, the last piece's result), in tiles.  At least one where it has tokens (their
// results are written though they see nothing).
__device__ __forceinline__ int tiles_of(const LatentParams &p, const Seq &s) {
    return s.n > 0 ? max(1, (s.len + kTile - 1) / kTile + p.cost) : 0;
}

// Where the g-th of `groups` equal shares of a line of `units` tiles begins: floor(units g / groups).
// A line shorter than p.groups is cut into shares of one tile (groups = units).
__device__ __forceinline__ int share_begin(const LatentParams &p, int units, int g, int groups) {
    if (units <= groups) return g;
    if (units < (1 << 19)) return p.shares.div(units * g);  // groups = p.groups < 2^11
    return static_cast<int>(static_cast<long long>(units) * g / groups);
}

// A group's share of the line.
struct Share {
    int units, groups;  // tiles on the line, shares it is cut into
    int u0, u1;         // this share's tiles
    int b, k;           // sequence and tile of the first
    Seq s;              // that sequence
};

// Found by each warp by itself (no block barrier before the first copies): a pass over the
// sequences for the line's length, one for the place of the share's beginning.
__device__ __forceinline__ Share share_of(const LatentParams &p, int g, bool report) {
    const int lane = threadIdx.x & 31;
    Share s;
    s.units = 0;
    Seq mine;  // the lane's sequence of the last 32 read
    mine.n = 0;
    int c = 0;
    for (;;) {
        if (c + lane < p.B) {
            mine = seq_of(p, c + lane);
            if (mine.bad && report) atomicOr(p.err, kErrBadIndex);
        } else {
            mine.n = 0;
        }
        s.units += static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(tiles_of(p, mine))));
        if (c + 32 >= p.B) break;
        c += 32;
    }
    s.groups = min(p.groups, max(s.units, 1));
    s.u0 = s.u1 = s.b = s.k = 0;
    if (g >= min(s.groups, s.units)) return s;
    s.u0 = share_begin(p, s.units, g, s.groups);
    s.u1 = share_begin(p, s.units, g + 1, s.groups);
    if (c > 0) mine = seq_of(p, lane);
    for (int at = 0, b0 = 0;;) {
        const int t = b0 + lane < p.B ? tiles_of(p, mine) : 0;
        int x = t;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, off);
            if (lane >= off) x += y;
        }
        const unsigned past = __ballot_sync(0xffffffffu, s.u0 < at + x);
        if (past) {
            const int w = __ffs(past) - 1;
            s.b = b0 + w;
            s.k = s.u0 - at - __shfl_sync(0xffffffffu, x - t, w);
            s.s.q0 = __shfl_sync(0xffffffffu, mine.q0, w);
            s.s.n = __shfl_sync(0xffffffffu, mine.n, w);
            s.s.n_all = __shfl_sync(0xffffffffu, mine.n_all, w);
            s.s.len = __shfl_sync(0xffffffffu, mine.len, w);
            return s;
        }
        at += __shfl_sync(0xffffffffu, x, 31);
        b0 += 32;
        if (b0 + lane < p.B) mine = seq_of(p, b0 + lane);
    }
}

// Scratch: descriptors, then two slots a CTA, each O (NT x R), m and l of a piece.  Slot 1 holds
// a sequence's first piece, slot 0 a later one.
__device__ __forceinline__ float *slot_of(const LatentParams &p, int cta, int which, int nt) {
    return p.ws + 4 * ((p.groups + 3) / 4 * 4) + (static_cast<long long>(cta) * 2 + which) * nt * (p.R + 2);
}

// One piece of a share: rows row0 .. row0 + nrows of sequence b, its tiles k0 .. k1 - 1 (none
// where the rows see no key of the piece).
struct Piece {
    Seq s;
    int b, row0, nrows, k0, k1;
    bool first, last;  // holds the sequence's first / last tile
    int left;          // tiles of the share from the piece's first on
};

struct Walk {
    int b, k, left;
    Seq s;       // sequence b, where it is known
    bool known;
    __device__ __forceinline__ explicit Walk(const Share &sh)
        : b(sh.b), k(sh.k), left(sh.u1 - sh.u0), s(sh.s), known(true) {}
    __device__ __forceinline__ bool next(const LatentParams &p, int r, Piece &o) {
        while (left > 0) {
            o.s = s;
            if (!known) o.s = seq_of(p, b);
            known = false;
            const int kt = tiles_of(p, o.s);
            const int take = min(kt - k, left);
            o.b = b;
            o.left = left;
            o.k0 = max(0, k - p.cost);
            const int end = max(0, k + take - p.cost);
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
            const int seen = o.s.len - o.s.n_all + p.heads.div(o.row0 + o.nrows - 1) + 1;
            o.k1 = max(o.k0, min(end, (max(seen, 0) + kTile - 1) / kTile));
            return true;
        }
        return false;
    }
};

// The pages of a piece's tiles, read 32 table entries at a time (one load a warp for 4 to 32
// tiles).  A tile is copied in `copies` pieces of `rows` rows of a page each.
struct Pages {
    const int *table;
    int rows, shift, per;  // rows a copy, log2 of the copies of a whole tile, their number
    int limit;             // rows the sequence has, as far as the piece goes
    int first;             // the first tile of the batch in `now`
    int now;
    int k, copies, row;    // the current tile, its copies, the first one's row in its page
    int pages;             // (the page past the last one reads as zeros)
    bool whole;            // a tile lies in one page

    // the table's entry for copy f of a tile, -1 past the piece's end
    __device__ __forceinline__ int look(const LatentParams &p, int tile, int f) const {
        if (tile * kTile + f * rows >= limit) return -1;
        return table[whole ? p.page_tiles.div(tile) : (tile << shift) + f];
    }
    __device__ __forceinline__ int look(const LatentParams &p, int tile) const {
        const int lane = threadIdx.x & 31;
        return look(p, tile + (lane >> shift), lane & (per - 1));
    }
    __device__ __forceinline__ Pages(const LatentParams &p, const Piece &o) {
        table = p.table + static_cast<long long>(o.b) * p.ldt;
        rows = 1 << p.row_shift;
        shift = 6 - p.row_shift;
        per = 1 << shift;
        whole = p.page_size >= kTile;
        limit = min(o.s.len, o.k1 * kTile);
        pages = p.pages;
        first = o.k0;
        now = look(p, first);
        row = whole ? p.page_tiles.mod(first) * kTile - kTile : 0;
    }
    // on to a tile: the first one, then one by one
    __device__ __forceinline__ void step(const LatentParams &p, int tile) {
        k = tile;
        if (k == first + (32 >> shift)) {
            first = k;
            now = look(p, k);
        }
        copies = (min(kTile, limit - k * kTile) + rows - 1) >> p.row_shift;
        if (whole) {
            row += kTile;
            if (row == p.page_size) row = 0;
        }
    }
    // the page of copy f of the current tile; an entry out of range is reported
    __device__ __forceinline__ int page(const LatentParams &p, int f) const {
        const int v = __shfl_sync(0xffffffffu, now, ((k - first) << shift) + f);
        if (v >= 0 && v < pages) return v;
        if ((threadIdx.x & 31) == 0) atomicOr(p.err, kErrBadIndex);
        return pages;
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

// The same for a whole warp, which goes on together.
__device__ __forceinline__ bool all_wait(uint32_t b, unsigned parity, int *stop) {
    if (__all_sync(0xffffffffu, bar_try(b, parity))) return true;
    return __all_sync(0xffffffffu, wait_or_stop(b, parity, stop));
}

// A value that all lanes of the warp have alike, by an instruction whose result the compiler
// knows to be: the issuing warps' loops and descriptors then stay in uniform registers, where
// tcgen05.mma and the copies want them.
__device__ __forceinline__ int alike(int v) { return static_cast<int>(__reduce_or_sync(0xffffffffu, static_cast<unsigned>(v))); }

// Barrier of the N softmax threads, alone or with the OR of a predicate.
template <int N>
__device__ __forceinline__ void soft_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(N) : "memory");
}
template <int N>
__device__ __forceinline__ bool soft_any(bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %1, 0;\n\t"
        "bar.red.or.pred q, 1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(v ? 1u : 0u), "n"(N)
        : "memory");
    return r != 0;
}

// One lane of a converged warp, the same each time.
__device__ __forceinline__ bool elect() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)::"memory");
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
                                       uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
        "[%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar), "l"(policy)
        : "memory");
}

// How the L2 cache keeps what is copied: evicted first where this CTA is its only reader (one
// sequence of 131072: 36.7 us, 38.3 without; where two CTAs read a tile, 128 heads, 110 became 132).
__device__ __forceinline__ uint64_t policy_of(bool once) {
    uint64_t r;
    if (once)
        asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(r));
    else
        asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(r));
    return r;
}

// Four 8 x 8 BF16 fragments, each stored turned: lane l gives the address of row l % 8 (its
// column in the fragment) of fragment l / 8.
__device__ __forceinline__ void stmatrix_turned(uint32_t addr, const uint32_t (&q)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(q[0]),
                 "r"(q[1]), "r"(q[2]), "r"(q[3])
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

// Wait (bounded) for a copy in flight.
__device__ __forceinline__ void landed(uint32_t bar, unsigned parity) {
    const unsigned long long t0 = global_ns();
    while (!bar_try(bar, parity))
        if (static_cast<long long>(global_ns() - t0) > kWaitLimitNs) break;
}

// Wait (bounded) until every product this warp issued is complete.
__device__ __forceinline__ void finish(uint32_t bar, int *stop) {
    if (elect()) mma_commit(bar);
    __syncwarp();
    const unsigned long long t0 = global_ns();
    while (!bar_try(bar, 0))
        if (static_cast<long long>(global_ns() - t0) > kWaitLimitNs) {
            atomicExch(stop, 1);
            break;
        }
    __syncwarp();
}

// BF16 pairs with infinities and NaN set to 0.
__device__ __forceinline__ uint32_t finite_or_zero(uint32_t w) {
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0x0000ffffu;
    return w;
}

// ----------------------------------------------------------------------------- the kernel
template <int NT>
__global__ void __launch_bounds__(threads_of(NT), 1) latent_attention_kernel(const __grid_constant__ LatentParams p) {
    constexpr int kSCols = NT;                    // tensor-memory columns of one S^T
    constexpr int kTmem = NT == 64 ? 512 : NT == 32 ? 256 : 128;
    constexpr int NP = weight_buffers(NT);
    constexpr int W = soft_parts(NT), CT = NT / W;  // softmax warps per quarter, their rows
    constexpr int kSoft = 128 * W;                // softmax threads
    constexpr int kLast = 3 + 4 * W;              // the last warp
    constexpr int NC = CT / 4;                    // rows a softmax thread holds scores of
    constexpr uint32_t kIdescS = (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(NT >> 3) << 17) |
                                 (static_cast<uint32_t>(kTile >> 4) << 24);
    constexpr uint32_t kIdescO = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (1u << 16) |
                                 (static_cast<uint32_t>(NT >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
    extern __shared__ __align__(1024) uint8_t base[];  // the only shared memory: it starts on 1 KiB
    const int pairs = p.R / 128;            // slots a tile
    const int qchunk = NT * 128;            // bytes of a chunk of Q
    const int S = p.slots;
    constexpr int RS = kRopeSlots;
    const uint32_t s_q = saddr(base);
    const uint32_t s_p = s_q + (2 * pairs + 1) * qchunk;
    const uint32_t s_r = s_p + NP * kChunk;
    const uint32_t s_v = s_r + RS * kChunk;
    uint8_t *misc = base + (s_v - s_q) + S * kSlot;
    uint64_t *bars = reinterpret_cast<uint64_t *>(misc);
    float(*ex)[4][NT] = reinterpret_cast<float(*)[4][NT]>(misc + kBarBytes);  // [2] a warp's maxima (or sums) of each row
    float *fs = reinterpret_cast<float *>(misc + kBarBytes + 32 * NT), *ms = fs + NT;  // a row's factor for O^T, its maximum
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(ms + NT);
    int &stop = *reinterpret_cast<int *>(tmem_slot + 1);

    const uint32_t vfull = saddr(bars), vempty = vfull + 8 * kMaxSlots;
    const uint32_t rfull = vempty + 8 * kMaxSlots, rempty = rfull + 8 * kRopeSlots;
    const uint32_t qfull = rempty + 8 * kRopeSlots, qempty = qfull + 8;
    const uint32_t sfull = qempty + 8, sempty = sfull + 16, pfull = sempty + 16, pvd = pfull + 16, fin = pvd + 16;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = p.ctas.div(static_cast<int>(blockIdx.x)), r = static_cast<int>(blockIdx.x) - g * p.rt;

    if (warp == 0) {
        if (lane == 0) {
            prefetch_tmap(&p.tv);
            prefetch_tmap(&p.tr);
            if (p.q_even) {
                prefetch_tmap(&p.qv);
                prefetch_tmap(&p.qr);
            }
            stop = 0;
        }
        // in the order of their addresses: the softmax warps arrive one by one on sempty, pfull
        for (int i = lane; i < (static_cast<int>(fin - vfull) >> 3) + 2; i += 32) {
            const uint32_t bar = vfull + 8 * i;
            bar_init(bar, bar >= sempty && bar < pvd ? 4 * W : 1);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
    }
    pdl_wait();
    uint32_t tmem = 0;
    if (warp == 0) {
        // the producer goes on: it needs the mbarriers only, which are its own work
        asm volatile("bar.arrive 2, %0;" ::"n"(threads_of(NT)) : "memory");
    } else if (warp == 1) {
        // Tensor memory is taken after the wait: a CTA of the previous kernel may still want its
        // own, and this one holds its columns until that kernel is done.
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(tmem_slot)),
                     "r"(kTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    const Share sh = share_of(p, g, blockIdx.x == 0 && warp == 2);  // while the tensor memory is taken
    if (warp != 0) {
        tc_fence_before();
        asm volatile("bar.sync 2, %0;" ::"n"(threads_of(NT)) : "memory");
        tc_fence_after();
        tmem = *tmem_slot;
    }
    const uint32_t t_o = tmem + 2 * kSCols;
    Walk walk(sh);
    const bool stall = (p.flags & kFlagTestStall) != 0;
    Piece o;
    int issued = 0, rissued = 0;  // slots of each ring that the producer filled
    int pieces = 0;               // pieces whose queries were copied

    if (warp == 0 || warp == kLast) {
        // ------------------------------------------------------------------ the copies
        // Two warps, every other slot of latent elements each, the second the rotated elements
        // too: one warp's wait, expect and copy take 630 cycles a slot, two warps 370.
        const uint64_t policy = policy_of(p.rt == 1);
        int at = 0, slot = 0, n = 0, rslot = 0;  // slots and tiles done; the rings' next slots
        unsigned ph = 0, rph = 0;                // parities of the rings' rounds
        bool ok = true;
        while (ok && walk.next(p, r, o)) {
            if (o.k0 >= o.k1) continue;
            Pages pages(p, o);
            for (int k = o.k0; ok && k < o.k1; ++k, ++n) {
                pages.step(p, k);
                const int copies = alike(pages.copies), step = pages.rows * 128;
                const int row = alike(pages.row);
                int page[kMaxCopies];
                page[0] = alike(pages.page(p, 0));
                if (copies > 1)
#pragma unroll
                    for (int f = 1; f < kMaxCopies; ++f)
                        if (f < copies) page[f] = alike(pages.page(p, f));
                for (int j = 0; j < pairs; ++j) {
                    if ((at & 1) == (warp == 0 ? 0 : 1)) {
                        if (!(ok = at < S || all_wait(vempty + 8 * slot, ph ^ 1, &stop))) break;
                        if (!stall) issued = at + 1;
                        const uint32_t dst = s_v + slot * kSlot, bar = vfull + 8 * slot;
                        if (elect()) {
                            bar_expect_tx(bar, static_cast<unsigned>(2 * copies * step));
                            if (!stall) {
                                if (pages.whole) {
                                    tma_4d(dst, &p.tv, 0, row, 2 * j, page[0], bar, policy);
                                } else {
#pragma unroll
                                    for (int f = 0; f < kMaxCopies; ++f)
                                        if (f < copies) {
                                            tma_4d(dst + f * step, &p.tv, 0, 0, 2 * j, page[f], bar, policy);
                                            tma_4d(dst + f * step + kChunk, &p.tv, 0, 0, 2 * j + 1, page[f], bar, policy);
                                        }
                                }
                            }
                        }
                        __syncwarp();
                    }
                    ++at;
                    if (++slot == S) {
                        slot = 0;
                        ph ^= 1;
                    }
                }
                if (warp == 0 || !ok) continue;
                if (!(ok = n < RS || all_wait(rempty + 8 * rslot, rph ^ 1, &stop))) break;
                if (!stall) rissued = n + 1;
                const uint32_t dst = s_r + rslot * kChunk, bar = rfull + 8 * rslot;
                if (elect()) {
                    bar_expect_tx(bar, static_cast<unsigned>(copies * step));
                    if (!stall) {
                        tma_3d(dst, &p.tr, 0, row, page[0], bar);
                        if (copies > 1)
#pragma unroll
                            for (int f = 1; f < kMaxCopies; ++f)
                                if (f < copies) tma_3d(dst + f * step, &p.tr, 0, row, page[f], bar);
                    }
                }
                __syncwarp();
                if (++rslot == RS) {
                    rslot = 0;
                    rph ^= 1;
                }
            }
        }
    } else if (warp == 1) {
        // --------------------------------------------------- the first product, S^T = K Q^T
        // The whole warp follows the loop, one elected lane issues: a branch on the lane's
        // number in its place made every tcgen05.mma take 100 to 250 cycles to issue.
        const int units = (2 * pairs + 1) * 8, width = p.R + p.E;
        int n = 0, slot = 0, rslot = 0;
        unsigned ph = 0, rph = 0;  // parities of the rings' rounds
        bool ok = true;
        const uint32_t base_d = alike(static_cast<int>(tmem));
        while (ok && alike(walk.next(p, r, o) ? 1 : 0)) {
            const int tiles = alike(o.k1 - o.k0);
            if (tiles == 0) continue;
            // the queries, when the last piece's products have read the ones before
            if (!(ok = pieces == 0 || all_wait(qempty, (pieces - 1) & 1, &stop))) break;
            ++pieces;
            if (p.q_even) {
                // rows past the sequence's are the next one's (or zeros past the last): their
                // products are columns of S^T that nothing reads
                if (elect()) {
                    const int row = o.s.q0 * p.H + o.row0;
                    bar_expect_tx(qfull, static_cast<unsigned>((2 * pairs + 1) * qchunk));
                    tma_3d(s_q, &p.qv, 0, row, 0, qfull);
                    tc05::tma_load_2d(s_q + 2 * pairs * qchunk, &p.qr, 0, row, qfull);
                }
                __syncwarp();
            } else {
                int tok = o.s.q0 + p.heads.div(o.row0), head = p.heads.mod(o.row0);
                for (int row = 0; row < NT; ++row) {
                    // rows past the piece and elements past the width are 0
                    const bool in = row < o.nrows;
                    const uint16_t *src = in ? p.q + tok * p.q_token + head * p.q_head : p.q;
#pragma unroll 3
                    for (int u = lane; u < units; u += 32)
                        copy16(s_q + (u >> 3) * qchunk + row * 128 + (((u & 7) ^ (row & 7)) << 4),
                               in && 8 * u < width ? src + 8 * u : p.q, in && 8 * u < width ? 16 : 0);
                    if (++head == p.H) {
                        head = 0;
                        ++tok;
                    }
                }
                asm volatile("cp.async.wait_all;" ::: "memory");
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) bar_arrive(qfull);
            }
            ok = all_wait(qfull, (pieces - 1) & 1, &stop);
            for (int k = 0; ok && k < tiles; ++k, ++n) {
                ok = n < 2 || all_wait(sempty + 8 * (n & 1), ((n >> 1) - 1) & 1, &stop);
                const uint32_t d = base_d + (n & 1) * kSCols;
                for (int j = 0; ok && j < pairs; ++j) {
                    if (!(ok = all_wait(vfull + 8 * slot, ph, &stop))) break;
                    tc_fence_after();
                    if (elect()) {
                        const uint64_t a = tc05::sw128_desc(s_v + slot * kSlot), b = tc05::sw128_desc(s_q + j * (2 * NT * 128));
#pragma unroll
                        for (int c = 0; c < 2; ++c)
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                mma(d, a + ((c * kChunk + 32 * kk) >> 4), b + ((c * NT * 128 + 32 * kk) >> 4), kIdescS,
                                    (c | kk) != 0 || j != 0);
                    }
                    __syncwarp();
                    if (++slot == S) {
                        slot = 0;
                        ph ^= 1;
                    }
                }
                if (!ok || !(ok = all_wait(rfull + 8 * rslot, rph, &stop))) break;
                tc_fence_after();
                if (elect()) {
                    const uint64_t a = tc05::sw128_desc(s_r + rslot * kChunk), b = tc05::sw128_desc(s_q + pairs * (2 * NT * 128));
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) mma(d, a + ((32 * kk) >> 4), b + ((32 * kk) >> 4), kIdescS, true);
                    mma_commit(sfull + 8 * (n & 1));
                    mma_commit(rempty + 8 * rslot);
                    if (k + 1 == tiles) mma_commit(qempty);
                }
                __syncwarp();
                if (++rslot == RS) {
                    rslot = 0;
                    rph ^= 1;
                }
            }
        }
        finish(fin, &stop);
    } else if (warp == 2 + 4 * W) {
        // ----------------------------------------------- the second product, O^T += V^T P^T
        int n = 0, slot = 0;
        bool ok = true;
        const uint32_t base_d = alike(static_cast<int>(t_o));
        while (ok && alike(walk.next(p, r, o) ? 1 : 0)) {
            const int tiles = alike(o.k1 - o.k0);
            for (int k = 0; k < tiles; ++k, ++n) {
                if (!(ok = all_wait(pfull + 8 * (n & 1), (n >> 1) & 1, &stop))) break;
                tc_fence_after();
                for (int j = 0; j < pairs; ++j) {
                    if (elect()) {
                        const uint64_t a = mn_desc(s_v + slot * kSlot), b = mn_desc(s_p + n % NP * kChunk);
#pragma unroll
                        for (int kk = 0; kk < kTile / 16; ++kk)
                            mma(base_d + j * NT, a + kk * (2048 >> 4), b + kk * (2048 >> 4), kIdescO, kk != 0 || k != 0);
                        mma_commit(vempty + 8 * slot);
                        if (j == pairs - 1) mma_commit(pvd + 8 * (n & 1));
                    }
                    __syncwarp();
                    if (++slot == S) slot = 0;
                }
            }
        }
        finish(fin + 8, &stop);
    } else if (warp < 2 + 4 * W) {
        // ------------------------------------------------------------------- softmax
        const int sw = warp & 3;  // tensor-memory lanes 32 sw .. and keys 16 sw .. of a tile
        const int tid = threadIdx.x - 64, part = (warp - 2) >> 2, col0 = part * CT;  // this warp's rows (columns of S^T)
        const int c0 = 2 * (lane & 3);
        const uint32_t quarter = static_cast<uint32_t>(32 * sw) << 16;
        const float inf = __int_as_float(0x7f800000), nan = __int_as_float(0x7fc00000);
        int n = 0, vslot = 0;  // tiles done; the next one's first slot
        bool ok = true, dead = false;
        // descriptors for the joining kernel: {q0, tokens, first, last group} of a split sequence
        int4 *desc = reinterpret_cast<int4 *>(p.ws);
        const bool tell = r == 0 && tid == 0 && p.groups > 1;
        if (tell && !p.by_seq) desc[g] = make_int4(0, 0, 0, -1);
        while (walk.next(p, r, o)) {
            if (tell && o.first) {
                const int u_last = sh.u0 + (sh.u1 - sh.u0 - o.left) + tiles_of(p, o.s) - 1;
                // the last share that begins at or before u_last: ceil((u_last + 1) groups / units) - 1
                const int g1 = static_cast<int>((static_cast<long long>(u_last + 1) * sh.groups - 1) / sh.units);
                if (p.by_seq || !o.last) desc[p.by_seq ? o.b : g] = make_int4(o.s.q0, o.s.n, g, o.last ? -1 : g1);
            }
            float m[NC], l[NC];
            int lim[NC];  // keys a row sees
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int col = col0 + 8 * (c >> 1) + c0 + (c & 1);
                m[c] = kNoMax;
                l[c] = 0.0f;
                lim[c] = col < o.nrows ? o.s.len - o.s.n_all + p.heads.div(o.row0 + col) + 1 : 0;
            }
            const int lim_min = max(0, o.s.len - o.s.n_all + p.heads.div(o.row0) + 1);
            for (int k = o.k0; k < o.k1 && !dead; ++k, ++n) {
                ok = wait_or_stop(sfull + 8 * (n & 1), (n >> 1) & 1, &stop) && ok;
                ok = __all_sync(0xffffffffu, ok);
                uint32_t sr[4 * (CT / 8)] = {};
                if (ok) {
                    tc_fence_after();
                    tmem_ld_s(tmem + quarter + (n & 1) * kSCols + col0, sr);
                    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) bar_arrive(sempty + 8 * (n & 1));
                // exponents: scores in base 2 less the maximum in use; over a lazy threshold some
                // maximum has to move
                const int key = k * kTile + 16 * sw + (lane >> 2);
                const bool edge = (k + 1) * kTile > lim_min || o.nrows < NT;
                float x[4 * (CT / 8)];
                auto hide = [&]() {
#pragma unroll
                    for (int i = 0; i < CT / 8; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (key + 8 * (e >> 1) >= lim[2 * i + (e & 1)]) x[4 * i + e] = -inf;
                };
#pragma unroll
                for (int i = 0; i < CT / 8; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        x[4 * i + e] = fmaf(__uint_as_float(sr[4 * i + e]), p.scale_log2, -m[2 * i + (e & 1)]);
                if (edge) hide();
                float most = -inf;
#pragma unroll
                for (int i = 0; i < 4 * (CT / 8); ++i) most = fmaxf(most, x[i]);
                if (soft_any<kSoft>(most > kLazy || !ok)) {
                    if (soft_any<kSoft>(!ok)) {
                        dead = true;
                        break;
                    }
                    float f[NC];
#pragma unroll
                    for (int i = 0; i < 4 * (CT / 8); ++i) x[i] = __uint_as_float(sr[i]) * p.scale_log2;
                    if (edge) hide();
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        const int i = c >> 1, e = c & 1;
                        float v = fmaxf(x[4 * i + e], x[4 * i + 2 + e]);
#pragma unroll
                        for (int d = 4; d <= 16; d <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
                        f[c] = v;
                    }
                    if (lane < 4)
#pragma unroll
                        for (int i = 0; i < CT / 8; ++i)
                            *reinterpret_cast<float2 *>(&ex[n & 1][sw][col0 + 8 * i + c0]) = make_float2(f[2 * i], f[2 * i + 1]);
                    soft_sync<kSoft>();
#pragma unroll
                    for (int i = 0; i < CT / 8; ++i) {
                        float2 v = make_float2(m[2 * i], m[2 * i + 1]);
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            const float2 y = *reinterpret_cast<const float2 *>(&ex[n & 1][w][col0 + 8 * i + c0]);
                            v.x = fmaxf(v.x, y.x);
                            v.y = fmaxf(v.y, y.y);
                        }
                        const float nm[2] = {v.x, v.y};
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int c = 2 * i + e;
                            f[c] = ex2(m[c] - nm[e]);
                            l[c] *= f[c];
                            m[c] = nm[e];
                            x[4 * i + e] -= nm[e];
                            x[4 * i + 2 + e] -= nm[e];
                        }
                    }
                    if (k > o.k0) {
                        // O^T of the tiles before: complete, then scaled in place
                        if (sw == 0 && lane < 4)
#pragma unroll
                            for (int i = 0; i < CT / 8; ++i)
                                *reinterpret_cast<float2 *>(&fs[col0 + 8 * i + c0]) = make_float2(f[2 * i], f[2 * i + 1]);
                        ok = wait_or_stop(pvd + 8 * ((n - 1) & 1), ((n - 1) >> 1) & 1, &stop) && ok;
                        soft_sync<kSoft>();
                        tc_fence_after();
                        for (int j = 0; j < pairs; ++j)
#pragma unroll
                            for (int c = col0; c < col0 + CT; c += 16) {
                                uint32_t v[16];
                                tmem_ld16(t_o + quarter + j * NT + c, v);
#pragma unroll
                                for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * fs[c + i]);
                                tmem_st16(t_o + quarter + j * NT + c, v);
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
                    for (int row = r0 + (warp - 2); row < kTile; row += 4 * W)
#pragma unroll 2
                        for (int u = lane; u < 16 * pairs; u += 32) {
                            int slot = vslot + (u >> 4);
                            slot = slot >= S ? slot - S : slot;
                            uint4 *at = reinterpret_cast<uint4 *>(base + (s_v - s_q) + slot * kSlot + ((u >> 3) & 1) * kChunk +
                                                                  row * 128 + (u & 7) * 16);
                            uint4 v = make_uint4(0u, 0u, 0u, 0u);
                            if (row < end) {
                                v = *at;
                                v.x = finite_or_zero(v.x);
                                v.y = finite_or_zero(v.y);
                                v.z = finite_or_zero(v.z);
                                v.w = finite_or_zero(v.w);
                            }
                            *at = v;
                        }
                }
                // The weights, into the buffer that tile n - NP used.  BF16, as the values are: both
                // operands of an MMA have one type.  Their rounding adds up to 1.2e-3 of the result
                // (root mean square) to the 1.7e-3 of the result's own; their sum keeps FP32.
                if (n >= NP) ok = wait_or_stop(pvd + 8 * ((n - NP) & 1), ((n - NP) >> 1) & 1, &stop) && ok;
                {
                    const int key_in = 16 * sw + (lane >> 2);
                    uint8_t *row = base + (s_p - s_q) + n % NP * kChunk + key_in * 128;
#pragma unroll
                    for (int i = 0; i < CT / 8; ++i) {
                        float w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int c = 2 * i + (e & 1);
                            w[e] = ex2(x[4 * i + e]);
                            l[c] += w[e];
                        }
                        const int at = (((i + col0 / 8) ^ (lane >> 2)) << 4) + 2 * c0;  // key_in % 8 = lane / 4
                        *reinterpret_cast<uint32_t *>(row + at) = bf16x2(w[0], w[1]);
                        *reinterpret_cast<uint32_t *>(row + 8 * 128 + at) = bf16x2(w[2], w[3]);
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) bar_arrive(pfull + 8 * (n & 1));
                vslot += pairs;
                if (vslot >= S) vslot -= S;
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
                for (int i = 0; i < CT / 8; ++i) {
                    *reinterpret_cast<float2 *>(&ex[n & 1][sw][col0 + 8 * i + c0]) = make_float2(l[2 * i], l[2 * i + 1]);
                    if (sw == 0) *reinterpret_cast<float2 *>(&ms[col0 + 8 * i + c0]) = make_float2(m[2 * i], m[2 * i + 1]);
                }
            dead = soft_any<kSoft>(!ok || dead);
            const bool empty = o.k0 >= o.k1;
            auto total = [&](int col) {
                return (ex[n & 1][0][col] + ex[n & 1][1][col]) + (ex[n & 1][2][col] + ex[n & 1][3][col]);
            };
            if (o.first && o.last) {
                // The whole sequence: O / l, BF16, turned in shared memory (where the weights
                // were) so that rows of out are written 16 bytes a thread.  The tensor memory is
                // read in the 16 x 256-bit form again, whose fragments stmatrix stores turned.
                long long *off = reinterpret_cast<long long *>(&ex[(n & 1) ^ 1][0][0]);
                if (tid < NT) {
                    const int row = o.row0 + tid, tok = o.s.q0 + p.heads.div(row), head = p.heads.mod(row);
                    off[tid] = tok * p.out_token + head * p.out_head;
                    const float sum = total(tid);
                    if (p.lse && tid < o.nrows)
                        p.lse[tok * p.lse_token + head] =
                            dead ? nan : sum == 0.0f ? -inf : (ms[tid] + log2f(sum)) * 0.69314718056f;
                }
                float inv[NC];
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const float sum = total(col0 + 8 * (c >> 1) + c0 + (c & 1));
                    inv[c] = dead ? nan : sum == 0.0f ? 0.0f : 1.0f / sum;
                }
                // 32 rows at a time (of 128 elements, 16-byte units swizzled), alternating where
                // there are two buffers
                for (int turn = 0; turn < pairs * (NT > 32 ? 2 : 1); ++turn) {
                    const int j = NT > 32 ? turn >> 1 : turn, rows0 = NT > 32 ? 32 * (turn & 1) : 0;
                    const uint32_t stage = s_p + (NP == 2 ? (turn & 1) * kChunk : 0);
                    if (NP == 1 && turn > 0) soft_sync<kSoft>();
                    if (NT <= 32 || rows0 == col0)
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            uint32_t v[4 * (CT / 8)];
                            if (empty || dead) {
#pragma unroll
                                for (int i = 0; i < 4 * (CT / 8); ++i) v[i] = 0u;
                            } else {
                                tmem_ld_s(t_o + quarter + (static_cast<uint32_t>(16 * half) << 16) + j * NT + col0, v);
                                asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
                            }
#pragma unroll
                            for (int i = 0; i < CT / 8; i += 2) {
                                uint32_t q[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const int c = 2 * (i + (e >> 1)), at = 4 * (i + (e >> 1)) + 2 * (e & 1);
                                    q[e] = bf16x2(__uint_as_float(v[at]) * inv[c], __uint_as_float(v[at + 1]) * inv[c + 1]);
                                }
                                const int col = col0 - rows0 + 8 * (i + (lane >> 4)) + (lane & 7);
                                const int unit = 4 * sw + 2 * half + ((lane >> 3) & 1);
                                stmatrix_turned(stage + col * 256 + ((unit ^ (col & 7)) << 4), q);
                            }
                        }
                    soft_sync<kSoft>();
                    for (int i = tid; i < min(32, o.nrows - rows0) * 16; i += kSoft) {
                        const int row = i >> 4, u = i & 15;
                        const uint4 v = *reinterpret_cast<const uint4 *>(base + (stage - s_q) + row * 256 + ((u ^ (row & 7)) << 4));
                        uint16_t *dst = p.out + off[rows0 + row] + 128 * j + 8 * u;
                        if (p.out16) {
                            *reinterpret_cast<uint4 *>(dst) = v;
                        } else {
                            uint32_t *d4 = reinterpret_cast<uint32_t *>(dst);
                            d4[0] = v.x;
                            d4[1] = v.y;
                            d4[2] = v.z;
                            d4[3] = v.w;
                        }
                    }
                }
            } else {
                // A piece: O, m and l as they are, FP32.  O in groups of four rows, [group][element][4]:
                // a thread holds one element of all rows and stores 16 bytes a group.
                float *ws = slot_of(p, static_cast<int>(blockIdx.x), o.first ? 1 : 0, NT);
                if (tid < NT) {
                    const float sum = total(tid);
                    // a NaN score leaves the maximum alone: the piece's is then NaN itself, so
                    // that joining keeps it whatever the maximum
                    ws[NT * p.R + tid] = dead || sum != sum ? nan : sum == 0.0f ? -inf : ms[tid];
                    ws[NT * p.R + NT + tid] = dead ? nan : sum;
                }
                if (!empty && !dead) {
                    float4 *o4 = reinterpret_cast<float4 *>(ws) + 32 * sw + lane;
                    const int groups = (o.nrows + 3) / 4;
                    for (int j = 0; j < pairs; ++j)
#pragma unroll
                    for (int c = col0; c < col0 + CT; c += 16) {
                        uint32_t v[16];
                        tmem_ld16(t_o + quarter + j * NT + c, v);
#pragma unroll
                        for (int i = 0; i < 16; i += 4)
                            if ((c + i) / 4 < groups)
                                o4[(j * NT + c + i) / 4 * 128] = make_float4(__uint_as_float(v[i]), __uint_as_float(v[i + 1]),
                                                                    __uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]));
                    }
                }
            }
            tc_fence_before();
            soft_sync<kSoft>();  // the shared buffers are used again
        }
    }
    __syncwarp();
    // after a stop: the copies issued have landed before the shared memory goes
    if (lane == 0 && *reinterpret_cast<volatile int *>(&stop)) {
        if (warp == 0 || warp == kLast) {
            for (int i = max(0, issued - S); i < issued; ++i)
                if ((i & 1) == (warp == 0 ? 0 : 1)) landed(vfull + 8 * (i % S), (i / S) & 1);
            for (int i = max(0, rissued - RS); i < rissued; ++i) landed(rfull + 8 * (i % RS), (i / RS) & 1);
        }
        if (warp == 1 && pieces > 0) landed(qfull, (pieces - 1) & 1);
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 32 && stop) atomicOr(p.err, 1);
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmem) : "memory");
    }
}

// ------------------------------------------------------------------ joining partial results
// A warp takes ES slabs of 32 elements of four rows of a split sequence, PB pieces at a time; the
// pw warps of a block with the same elements take every pw-th PB pieces and are added in their
// order.  Lane 4 q + e works out the weight of piece q for row e.  Where there are many rows (a
// batch of sequences): 4 at a time and 128 elements, so that a weight serves 16 products.  Where
// there are few (one long sequence over all groups): 8 at a time, up to 32 warps, so that all are
// read at once.
template <int PB, int ES>
__global__ void __launch_bounds__(PB == 8 ? 1024 : 128) latent_join_kernel(const __grid_constant__ LatentParams p) {
    constexpr int kWarps = PB == 8 ? 32 : 1;  // warps that share elements
    __shared__ __align__(16) float4 acc[kWarps][32];
    __shared__ float tacc[kWarps][4], lacc[kWarps][4];
    if (p.flags & kFlagPdl) pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row0 = 4 * static_cast<int>(blockIdx.y), i = row0 & (p.nt - 1), r = row0 / p.nt;
    // many: the block's warps share one slab; few: each has its own ES slabs
    const int wp = PB == 8 ? warp : 0;
    const int slab = PB == 8 ? static_cast<int>(blockIdx.z) : warp * ES;
    const int at = ((slab >> 2) * (p.nt / 4) + i / 4) * 128 + (slab & 3) * 32 + lane;
    const float inf = __int_as_float(0x7f800000);
    // a sequence without tokens has no pieces, and no descriptor
    const bool none = p.by_seq && seq_of(p, blockIdx.x).n == 0;
    pdl_wait();
    if (none) return;
    const int4 d = reinterpret_cast<const int4 *>(p.ws)[blockIdx.x];
    const int g0 = d.z, g1 = d.w, rows = d.y * p.H;
    if (g1 < 0 || row0 >= rows) return;
    auto slot = [&](int g) { return slot_of(p, g * p.rt + r, g == g0 ? 1 : 0, p.nt); };

    const int e = lane & 3, mine_at = (lane >> 2) & (PB - 1);
    float top = -inf, l = 0.0f;  // of row e, the same in all its lanes
    float4 a[ES];
#pragma unroll
    for (int c = 0; c < ES; ++c) a[c] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int g = g0 + PB * wp; g <= g1; g += PB * p.pw) {
        const int mine = g + mine_at;
        const float *ml = slot(min(mine, g1)) + p.nt * p.R + i + e;
        float m = ml[0], lm = ml[p.nt];
        float4 v[PB][ES];
#pragma unroll
        for (int q = 0; q < PB; ++q)
            if (g + q <= g1) {
                const float4 *o4 = reinterpret_cast<const float4 *>(slot(g + q)) + at;
#pragma unroll
                for (int c = 0; c < ES; ++c) v[q][c] = o4[32 * c];
            }
        if (mine > g1) m = -inf;
        float t = m;
#pragma unroll
        for (int o = 4; o < 4 * PB; o <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
        t = fmaxf(t, top);
        const float base = t == -inf ? 0.0f : t;
        const float f = ex2(top - base);
        // a piece that has no key for the row (m = -inf) holds nothing: its O was not written
        const float w = m == -inf ? 0.0f : ex2(m - base);
        float lw = m == -inf ? 0.0f : w * lm;
#pragma unroll
        for (int o = 4; o < 4 * PB; o <<= 1) lw += __shfl_xor_sync(0xffffffffu, lw, o);
        l = l * f + lw;
        top = t;
        const float f0 = __shfl_sync(0xffffffffu, f, 0), f1 = __shfl_sync(0xffffffffu, f, 1);
        const float f2 = __shfl_sync(0xffffffffu, f, 2), f3 = __shfl_sync(0xffffffffu, f, 3);
#pragma unroll
        for (int c = 0; c < ES; ++c) a[c] = make_float4(a[c].x * f0, a[c].y * f1, a[c].z * f2, a[c].w * f3);
#pragma unroll
        for (int q = 0; q < PB; ++q) {
            const float w0 = __shfl_sync(0xffffffffu, w, 4 * q), w1 = __shfl_sync(0xffffffffu, w, 4 * q + 1);
            const float w2 = __shfl_sync(0xffffffffu, w, 4 * q + 2), w3 = __shfl_sync(0xffffffffu, w, 4 * q + 3);
#pragma unroll
            for (int c = 0; c < ES; ++c) {
                a[c].x = w0 == 0.0f ? a[c].x : fmaf(w0, v[q][c].x, a[c].x);
                a[c].y = w1 == 0.0f ? a[c].y : fmaf(w1, v[q][c].y, a[c].y);
                a[c].z = w2 == 0.0f ? a[c].z : fmaf(w2, v[q][c].z, a[c].z);
                a[c].w = w3 == 0.0f ? a[c].w : fmaf(w3, v[q][c].w, a[c].w);
            }
        }
    }
    if constexpr (PB == 8) {
        if (p.pw > 1) {
            acc[warp][lane] = a[0];
            if (lane < 4) {
                tacc[warp][e] = top;
                lacc[warp][e] = l;
            }
            __syncthreads();
            if (wp > 0) return;
            // the same once more, over the warps: lane 4 q + e has row e of warps q, q + 8, ...
            float m[4], f[4], t = -inf;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int w = mine_at + 8 * c;
                m[c] = w < p.pw ? tacc[w][e] : -inf;
                t = fmaxf(t, m[c]);
            }
#pragma unroll
            for (int o = 4; o <= 16; o <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
            const float base = t == -inf ? 0.0f : t;
            l = 0.0f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int w = mine_at + 8 * c;
                f[c] = ex2(m[c] - base);
                // the sum of a warp whose scores were NaN is NaN though its maximum may be -inf
                const float x = w < p.pw ? lacc[w][e] : 0.0f;
                l += f[c] == 0.0f && x == x ? 0.0f : f[c] * x;
            }
#pragma unroll
            for (int o = 4; o <= 16; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            top = t;
            float4 s4 = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int c = 0; c < 4; ++c)
                for (int q = 0; q < 8 && 8 * c + q < p.pw; ++q) {
                    const float4 v = acc[8 * c + q][lane];
                    s4.x = fmaf(__shfl_sync(0xffffffffu, f[c], 4 * q), v.x, s4.x);
                    s4.y = fmaf(__shfl_sync(0xffffffffu, f[c], 4 * q + 1), v.y, s4.y);
                    s4.z = fmaf(__shfl_sync(0xffffffffu, f[c], 4 * q + 2), v.z, s4.z);
                    s4.w = fmaf(__shfl_sync(0xffffffffu, f[c], 4 * q + 3), v.w, s4.w);
                }
            a[0] = s4;
        }
    }
    const float inv_e = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int row = row0 + c;
        const float inv = __shfl_sync(0xffffffffu, inv_e, c);
        const long long tok = d.x + p.heads.div(row), head = p.heads.mod(row);
        uint16_t *out = p.out + tok * p.out_token + head * p.out_head + 32 * slab + lane;
#pragma unroll
        for (int z = 0; z < ES; ++z) {
            const float v = (c == 0 ? a[z].x : c == 1 ? a[z].y : c == 2 ? a[z].z : a[z].w) * inv;
            const float other = __shfl_xor_sync(0xffffffffu, v, 1);
            if (row < rows && !(lane & 1)) *reinterpret_cast<uint32_t *>(out + 32 * z) = bf16x2(v, other);
        }
    }
    if (p.lse && slab == 0 && lane < 4 && row0 + lane < rows) {
        const long long tok = d.x + p.heads.div(row0 + lane), head = p.heads.mod(row0 + lane);
        p.lse[tok * p.lse_token + head] = l == 0.0f ? -inf : (top + log2f(l)) * 0.69314718056f;
    }
}

const void *kernel_of(int nt) {
    return nt == 64   ? reinterpret_cast<const void *>(&latent_attention_kernel<64>)
           : nt == 32 ? reinterpret_cast<const void *>(&latent_attention_kernel<32>)
                      : reinterpret_cast<const void *>(&latent_attention_kernel<16>);
}

// The sizes of a call: rows a CTA, CTAs a group, groups, a sequence's cost in tiles.
struct Split {
    int nt, rt, groups, cost;
    long long ws_bytes;
};

Split split_of(const sgemm_latent_attention_t &a, int sms) {
    Split s;
    const long long rows = static_cast<long long>(a.max_q) * a.H;
    // The fewest that hold a sequence's rows, for the room they leave to the ring and the softmax's
    // registers (16 sequences of 8192, 16 heads: 16 rows 33.7 us, 32 34.5, 64 36.9; 32 heads: 32 rows
    // 38.6, 64 40.6); more than 64 would leave room for one tile.
    s.nt = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
    s.rt = static_cast<int>((rows + s.nt - 1) / s.nt);
    const long long tiles = std::max(1LL, (static_cast<long long>(a.table_width) * a.page_size + kTile - 1) / kTile);
    // A line that is short whatever the lengths has a share for each tile.  Nothing else is counted
    // then: with a sequence's cost some share has two tiles (one sequence of 1000 rows: 11.9 us,
    // without it 10.8), or, with a share more for it, one has none (11.0).
    s.cost = tiles * a.B <= sms / s.rt ? 0 : kPieceCost;
    s.groups = static_cast<int>(std::max(1LL, std::min<long long>(sms / s.rt, tiles * a.B)));
    s.ws_bytes = s.groups > 1 ? (s.groups + 3) / 4 * 64 + static_cast<long long>(s.groups) * s.rt * 2 * s.nt * (a.R + 2) * 4 : 0;
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
    if (a.pages >= big || a.total_q >= big || a.total_q * a.H >= 2 * big || static_cast<long long>(a.max_q) * a.H >= big ||
        static_cast<long long>(a.max_q) * a.B >= big || static_cast<long long>(a.table_width) * a.page_size >= big ||
        (static_cast<long long>(a.table_width) * a.page_size / kTile + 2 + kPieceCost) * a.B >= big)
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
    if (p.q_even) {
        const cuuint64_t n = static_cast<cuuint64_t>(a.total_q) * static_cast<cuuint64_t>(a.H);
        const cuuint64_t step = static_cast<cuuint64_t>(a.H > 1 ? a.q_head : a.q_token) * 2;
        const cuuint32_t ones[3] = {1, 1, 1}, nt = static_cast<cuuint32_t>(p.nt), chunks = static_cast<cuuint32_t>(a.R / 64);
        const cuuint64_t dims[3] = {64, n, chunks}, strides[2] = {step, 128};
        const cuuint32_t box[3] = {64, nt, chunks};
        const cuuint64_t rdims[2] = {static_cast<cuuint64_t>(a.E), n}, rstrides[1] = {step};
        const cuuint32_t rbox[2] = {64, nt};
        if (enc(&p.qv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t *>(a.q), dims, strides, box, ones,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS ||
            enc(&p.qr, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t *>(a.q) + a.R, rdims, rstrides, rbox, ones,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return false;
    }
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

// Whether `n` bytes at `b` (the scratch) or the array `h` (an output of T x H rows) lie in what the
// call reads beside the queries.
bool in_inputs(const sgemm_latent_attention_t &a, const Heads *h, const void *b, long long n) {
    if (h) {
        b = h->p;
        n = h->extent(a.total_q, a.H);
    }
    const long long page = 2 * ((a.page_size - 1) * a.row_stride + a.R + a.E);
    return block_touches(b, n, a.cache, page, 2 * a.page_stride, a.pages) ||
           block_touches(b, n, a.block_table, 4LL * a.table_width, 4 * a.ldt, a.B) ||
           block_touches(b, n, a.seq_lens, 4LL * a.B, 0, 1) || block_touches(b, n, a.cu_q, 4LL * a.B + 4, 0, 1);
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
    // out and lse lie apart from what is read and from each other
    const Heads q{a->q, 2 * W, 2 * a->q_token, 2 * a->q_head}, out{a->out, 2LL * a->R, 2 * a->out_token, 2 * a->out_head};
    const Heads lse{a->lse, 4, 4 * a->lse_token, 4};
    if (heads_overlap(out, q, a->total_q, a->H) || heads_overlap(lse, q, a->total_q, a->H) ||
        heads_overlap(out, lse, a->total_q, a->H) || in_inputs(*a, &out, nullptr, 0) ||
        (a->lse && in_inputs(*a, &lse, nullptr, 0)))
        return SGEMM_ERR_INVALID_ARG;
    // strides that a tensor map can hold
    if (a->row_stride >= (1LL << 38) || a->page_stride >= (1LL << 38)) return SGEMM_ERR_UNSUPPORTED_SHAPE;

    LatentParams p;
    std::memset(&p, 0, sizeof(p));
    int sms = 0;
    st = device_ready(&sms, &p.err);
    if (st != SGEMM_OK) return st;
    const Split sp = split_of(*a, sms);
    if (sp.ws_bytes > 0 && (!a->workspace || a->workspace_bytes < sp.ws_bytes)) return SGEMM_ERR_NO_WORKSPACE;
    // and so does the scratch that the call uses
    auto in_scratch = [&](const Heads &h) {
        return rows_overlap(a->workspace, sp.ws_bytes, 0, h.p, h.extent(a->total_q, a->H), 0, 1);
    };
    if (sp.ws_bytes > 0 && (in_scratch(q) || in_scratch(out) || in_scratch(lse) || in_inputs(*a, nullptr, a->workspace, sp.ws_bytes)))
        return SGEMM_ERR_INVALID_ARG;
    p.nt = sp.nt;
    // one stride from each (token, head) row to the next, wide enough that rows are apart (a
    // tensor map's strides are)
    const long long step = a->H > 1 ? a->q_head : a->q_token;
    p.q_even = (a->H == 1 || a->total_q == 1 || a->q_token == a->H * a->q_head) && step >= W && step < (1LL << 38) ? 1 : 0;
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
    p.rt = sp.rt;
    p.groups = sp.groups;
    p.cost = sp.cost;
    p.scale_log2 = static_cast<float>(static_cast<double>(a->scale) * 1.4426950408889634);
    p.flags = static_cast<int>(a->flags);

    p.heads = Divisor::of(a->H);
    p.ctas = Divisor::of(sp.rt);
    p.shares = Divisor::of(sp.groups);
    p.page_tiles = Divisor::of(std::max(1, a->page_size / kTile));
    p.row_shift = a->page_size >= kTile ? 6 : a->page_size == 32 ? 5 : a->page_size == 16 ? 4 : 3;
    p.out16 = aligned(a->out, 16) && a->out_token % 8 == 0 && a->out_head % 8 == 0 ? 1 : 0;
    p.by_seq = a->B < sp.groups ? 1 : 0;
    // Shared memory: Q, the weights, the rotated elements' ring, then as many slots of latent
    // elements as there is room for
    const int fixed = (a->R / 64 + 1) * sp.nt * 128 + weight_buffers(sp.nt) * kChunk + kRopeSlots * kChunk + kBarBytes +
                      40 * sp.nt + 16;
    p.slots = std::min(kMaxSlots, (static_cast<int>(kMaxSmemOptin) - fixed) / kSlot);
    const int smem = fixed + p.slots * kSlot;
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
    if (launch(fn, dim3(static_cast<unsigned>(sp.groups * sp.rt)), dim3(static_cast<unsigned>(threads_of(sp.nt))), static_cast<size_t>(smem), cs, &p) != cudaSuccess)
        return SGEMM_ERR_CUDA;
    if (sp.groups == 1) return SGEMM_OK;
    // Joining: one warp for 128 elements of four rows of a sequence, where these warps are enough to
    // keep the loads coming (2.5 for each SM); else warps that share a sequence's pieces (as many as
    // it would have if all were as long as the table allows), for 32 elements.  The one against the
    // other, 8192 rows with 32 heads: 9 sequences (288 warps) 26.4 us, 25.3; 12 (384) 30.9, 31.0;
    // 16 (512) 36.6, 38.6; 64 (2048) 74.2, 79.6; one of 131072 (32) 57.5, 36.7.
    const long long rows = static_cast<long long>(a->max_q) * a->H;
    const int n = p.by_seq ? a->B : sp.groups, parts = p.by_seq ? (sp.groups + a->B - 1) / a->B + 1 : 2;
    const bool few = (rows + 3) / 4 * (a->R / 128) * n * 2 >= 5LL * sms;
    p.pw = few ? 1 : std::min(32, (parts + 7) / 8);
    const dim3 grid(static_cast<unsigned>(n), static_cast<unsigned>((rows + 3) / 4),
                    static_cast<unsigned>(few ? 1 : a->R / 32));
    const void *join = few ? reinterpret_cast<const void *>(&latent_join_kernel<4, 4>)
                           : reinterpret_cast<const void *>(&latent_join_kernel<8, 1>);
    // The first kernel never lets this one come early: blocks that came were in the way of CTAs
    // still running (verification of 8 sequences: 28.8 us, against 26.7).
    if (launch(join, grid, dim3(static_cast<unsigned>(32 * (few ? a->R / 128 : p.pw))), 0, cs, &p) != cudaSuccess)
        return SGEMM_ERR_CUDA;
    return SGEMM_OK;
}
