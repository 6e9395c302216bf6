// Linear attention with a decay for each head, whole sequences (declared in
// include/sgemm_layers.h).  In chunks of 64 tokens, with G_i the sum of g over a chunk's tokens up to i:
//
//     o_i = scale (exp(G_i) q_i^T S + sum_{j <= i} exp(G_i - G_j) (q_i . k_j) v_j)
//     S'  = exp(G) S + sum_j exp(G - G_j) k_j v_j^T
//
// What bounds it.  A token and head's q, k, v, out are 4 x 128 elements, 1 KiB, for about 10^5
// operations: 100 a byte, below what the tensor cores do for each byte of memory.  So memory bounds it,
// if the chain of the chunks' states does not: that chain has to be short, and there have to be
// enough of them.
//
// Work split.  Either an SM takes whole sequences of a head (the longest first, dealt out forwards and backwards in
// turn), or the chunks of all (sequence, head) pairs form one line, cut into equal shares, one
// for each SM; a share ends anywhere inside a sequence (see share_of).  Three launches:
//   (With few tokens there is nothing to cut, and the third is the only one.)
//   1. states: for every share that ends inside a sequence, what its part of that sequence adds to
//      the state, U = sum_j exp(sum of g from j to the share's end) k_j v_j^T, and the sum of its g.  The
//      chunks are taken from the last to the first, so that the factor of a key is known at once
//      and the sum stays in tensor memory untouched.
//   2. joining: along each cut sequence, S' = exp(G) S + U from share to share, element by element.
//   3. outputs: every share from the state it begins with.
// Keys and values of cut sequences are read twice.
//
// The state kernel: U = K'^T V.  Its warps read the keys turned (ldmatrix), scale them and put them into tensor
// memory as the first operand, element of the key a lane; the second are the values as they came.
//
// The output kernel, a CTA an SM, all products but A turned so that the value's elements are the 128
// rows (lanes of tensor memory) and tokens or the key's elements the columns:
//     A    = Q K^T         64 x 64          both from shared memory
//     S^T += V^T K'        128 x Dk         V^T from tensor memory, K' = exp(G - G_j) k_j, three BF16 numbers each
//     O1   = Sb^T Q^T      128 x 64         Sb, the state rounded to BF16, from tensor memory
//     O2   = V^T P^T       128 x 64         P = A with its decays, BF16, through shared memory
// The state stays in tensor memory, FP32, for the whole sequence; a lane holds a value element's row, so that
// scaling it and rounding it for the next O1 needs no exchange.  out = scale (exp(G_i) O1 + O2) is put
// together in FP32.  Why K' in three numbers (cut off after 8 bits each: 24 bits): its rounding would be the
// state's only error above FP32's, 2^-8 of every summand (in two numbers 2^-16), and it goes on to all later
// tokens.  P and Sb are rounded once: what they make is rounded to BF16 right after.
// Roles: a warp copies (TMA, a ring of chunks), two issue the products, a warp sums the decays, and
// eight turn the values and scale the keys, and four each carry the state, apply the decays to A, and write the outputs.
// Exponents' sums are kept as pairs of FP32 numbers where states are made of them: differences of long sums
// keep their digits.
// The roles' loops are short on purpose: unrolled, their code did not fit the instruction cache, and a chunk
// took 9600 cycles (4500 without any other change).
//
// Measured on one GB300, calls one after the other:
//   16384 tokens, 32 heads, 128 x 128 (541 MB)                         167 us
//     states 50 us (235 MB, 4.7 TB/s), joining 4, outputs 114 (529 MB, 4.6 TB/s; alone, from a cold cache)
//   8 ragged prompts of up to 2049, 8 key and 32 value heads, 64 x 128  72 us (whole sequences)
//   one prompt of 500, 16 heads                                         20 us (the third kernel alone)
// What bounds the output kernel: a chunk takes 3200 to 3500 cycles, and three chains of about that length wait for one
// another: the state's (product 1300, pass 1100, hand-overs 900), A's (decays 1600, two products and their hand-overs
// 1700) and the outputs' (2000, and 1500 until the next).  Issue slots are taken to 54%, the tensor pipe to 36%.  The states'
// kernel is bound by memory, 41 GB/s an SM while it runs.  Around them: 2.4 us until the first copies are
// issued, 3 us for a state's first load, 3 for the last store.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>

#include "linear_common.h"
#include "tc05_roles.cuh"
#include "tensor_map.h"

namespace sk {
namespace linear {

using namespace roles;

constexpr int kC = 64;                 // tokens a chunk
constexpr int kPart = kC * 128;        // 64 tokens x 64 elements, bytes
constexpr int kStages = 6;             // of chunks in a ring, at most
constexpr int kFew = 8;                // chunks a share has at least, where sequences differ
constexpr int kLeastCut = 4;           // and where they are alike
constexpr int kOutThreads = 24 * 32;   // copies, products, sums, products, state, decays, outputs (4 each), values and keys (8)
constexpr int kSums = 8;               // chunks whose sums of g are kept
constexpr int kStateThreads = 12 * 32;  // copies, products, keys (4 + 4), sums (2)
// A decay's exponent (base 2) is cut here: 2^-200 is 0.  The sum of a chunk's is then 12800 at most, one
// FP32 number of it off by 2^-11, and a factor exp2 of a difference by 2^-10.5: below BF16's rounding.
constexpr float kLeast = -200.0f;

struct LinearParams {
    CUtensorMap tq, tk, tv, to;  // {64, N, D / 64, heads}, boxes of 64 tokens: a chunk's operand is one copy
    const float *g;
    float *state;
    const long long *slots;
    const int *cu, *fresh;
    uint16_t *out;
    float *ws;
    int *err;
    long long g_token, g_head, s_slot, s_head, o_token, o_head, pool, N;
    int B, Hv, share;  // sequences, value heads, value heads a key head
    int Dk, Dv;
    int groups;        // shares at most
    int whole;         // no sequence is cut, whatever the lengths, and the third kernel is the only one
    int stages;
    int out16;         // out's rows start on 16 bytes: whole chunks are stored as one copy
    int flags;
    float scale;
};

// ------------------------------------------------------------------ the line of chunks
struct Seq {
    int t0, len, chunks;  // first token, tokens, chunks (at least one; 0: the offsets are no sequence's)
    long long slot;       // negative: none
    bool bad;
};

__device__ __forceinline__ Seq seq_of(const LinearParams &p, int b) {
    Seq s;
    const int a = p.cu[b], e = p.cu[b + 1];
    s.slot = p.slots[b];
    s.bad = s.slot >= p.pool;
    if (s.bad) s.slot = -1;
    s.t0 = a;
    s.len = e - a;
    if (a < 0 || e < a || e > p.N) {
        s.bad = true;
        s.t0 = s.len = s.chunks = 0;
    } else {
        s.chunks = max(1, (s.len + kC - 1) / kC);
    }
    return s;
}

// Chunks that a line has at most.  Offsets that rise keep far below it (checked on the host); offsets that fall and rise
// again over the same tokens may not, and their sum may pass 32 bits: nothing is computed then.
constexpr long long kMostUnits = 1LL << 30;

struct Share {
    int units, groups, u0, u1;
    bool whole;  // u1 chunks, of whole sequences, the first of which is
    int b, h;
};

__device__ __forceinline__ int begin_of(int units, int g, int groups) {
    return static_cast<int>(static_cast<long long>(units) * g / groups);
}

// Chunks on the line of the kEachLane sequences from b on: a lane's (their loads are in flight together: batches of
// many short sequences spend their time here); the least and the most that one of them has.
constexpr int kEachLane = 8;
__device__ __forceinline__ int units_of(const LinearParams &p, int b, bool report, int &least, int &most, int *keep = nullptr) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < kEachLane; ++i)
        if (b + i < p.B) {
            const Seq q = seq_of(p, b + i);
            n += q.chunks * p.Hv;
            least = min(least, q.chunks);
            most = max(most, q.chunks);
            if (keep) keep[b + i] = q.chunks;
            if (q.bad && report) atomicOr(p.err, kErrBadIndex);
        }
    return n;
}

// Whole sequences, for the SMs: the pairs of a sequence and a head in the order of their chunks, the longest first, are
// dealt out forwards and backwards in turn.
// Calls with more of either are cut, which takes longer (prompts of 200, 16 heads: 256 of them 338 us, 257 365, 400 545; 64
// heads: 152 of them 759, 153 816).
constexpr int kMostSorted = 256, kMostRounds = 64;
__device__ __forceinline__ int dealt(int round, int g, int groups) { return round & 1 ? (round + 1) * groups - 1 - g : round * groups + g; }

// Sorts the sequences (room: their chunks): the chunks of the SM that has the most, if whole ones are dealt out.  A
// function by itself, for shares that do not call it start 2 us later with it in their midst.
__device__ __noinline__ int deal(const LinearParams &p, int bins, int *room, uint8_t *order) {
    int *sorted = room + kMostSorted, *span = sorted + kMostSorted;
    const int pairs = p.B * p.Hv;
    if (threadIdx.x == 0) *span = 0;
    __syncthreads();
    for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
        const int mine = room[b];
        int rank = 0;
        for (int i = 0; i < p.B; ++i) rank += room[i] > mine || (room[i] == mine && i < b);
        sorted[rank] = mine;
        order[rank] = static_cast<uint8_t>(b);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < bins; i += blockDim.x) {
        int n = 0;
        for (int r = 0; r * bins < pairs; ++r) {
            const int j = dealt(r, i, bins);
            if (j < pairs) n += sorted[j / p.Hv];
        }
        atomicMax(span, n);
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // (copies come to where this was)
    __syncthreads();
    return *span;
}

// The chunks of an SM's whole sequences (by a whole warp).
__device__ __noinline__ int dealt_chunks(const LinearParams &p, int g, int bins, const int *sorted) {
    unsigned n = 0;
    for (int r = threadIdx.x & 31; r * bins < p.B * p.Hv; r += 32) {
        const int j = dealt(r, g, bins);
        if (j < p.B * p.Hv) n += static_cast<unsigned>(sorted[j / p.Hv]);
    }
    return static_cast<int>(__reduce_add_sync(0xffffffffu, n));
}

constexpr int kChunkCost = 185, kLineCost = 1700, kStarts = 340;  // 10 ns
// The line's length and share g of it (by all threads; `room` is shared memory).  order: the sequences, the longest first.
// How many shares.  A share's chunk takes 1.85 us, and 0.95 more if its sequence is cut; cutting costs 7 us and half a
// one a part, and 10 more where shares end inside one sequence and begin inside another.  So sequences are left whole, those
// that are alike are cut into equal parts, or the line of all of them is cut into shares of kFew chunks or more (one for each
// sequence and head where those are fewer), whichever takes the least.
// Whole, and on the line (us, ragged prompts): 4 up to 2324, 32 heads 77.4, 84.0; 3 of 3000 93.6, 85.5; 8 of 2000, 16
// heads 68.9, 78.4; 8 of 1500, 8 heads 52.7, 48.5; 16 of 900, 8 heads 38.7, 53.6; 32 of 500, 32 heads 116, 162; 200 of 200,
// 16 heads (21 rounds) 234, 312; 3 of 1000, 32 heads of 64 x 128 33.4, 37.2; 3 of 4000 102.5, 84.8.
// Alike (us, 128 x 128; shares of 4, of 8, of 16 chunks or whole): 500 tokens, 16 heads 28.1, 25.1 (whole); 1000, 8:
// 28.7, 37.1, 38.8 (whole); 2000, 4: 30.4, 37.8, 55.7; 4000, 2: 34.1, 39.6, 56.5; 2000, 32 heads, of 6.7, 8, 16: 46.9,
// 42.8, 58.9.  Equal parts, and shares of kFew with no regard to where sequences end: 750 tokens, 16 heads 30.4, 40.8;
// 640, 8: 28.8, 39.9; 3000, 16: 44.0, 50.0; 16384, 32: 170.6, 169.9.  Parts of 2 or 3 chunks gained nothing, and
// 8000 tokens of one head took 54.4 for 43.7.
// COUNTS: the sequences may come to kMostUnits chunks, whatever their offsets, and are counted in 64 bits (a template
// argument: with the test in the other kernels' midst ragged prompts took 72.1 us for 70.3, prompts of 500 20.5 for 20.3).
template <bool COUNTS>
__device__ __forceinline__ Share share_of(const LinearParams &p, int g, bool report, int *room, uint8_t *order) {
    const int lane = threadIdx.x & 31, pairs = p.B * p.Hv, bins = min(pairs, p.groups);
    const bool few = p.B <= kMostSorted && pairs <= kMostRounds * bins;
    int *keep = few && pairs > bins && threadIdx.x < 32 ? room : nullptr;
    Share s;
    s.units = 0;
    int least = 1 << 30, most = 0;
    if (COUNTS) {
        long long sum = 0;
        for (int c = 0; c < p.B; c += 32 * kEachLane) {
            const unsigned n = static_cast<unsigned>(units_of(p, c + kEachLane * lane, report, least, most, keep));  // (below 2^29)
            sum += __reduce_add_sync(0xffffffffu, n & 0xffffu) + (static_cast<long long>(__reduce_add_sync(0xffffffffu, n >> 16)) << 16);
        }
        s.units = static_cast<int>(sum);
        if (sum >= kMostUnits) {
            if (report && lane == 0) atomicOr(p.err, kErrBadIndex);
            s.units = s.u0 = s.u1 = s.b = s.h = 0;
            s.groups = 1;
            s.whole = false;
            return s;
        }
    } else {
        for (int c = 0; c < p.B; c += 32 * kEachLane)
            s.units += static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(units_of(p, c + kEachLane * lane, report, least, most, keep))));
    }
    least = __reduce_min_sync(0xffffffffu, least);
    most = __reduce_max_sync(0xffffffffu, most);
    const bool packs = few && most > 1, sorts = packs && pairs > bins;  // (a line of single chunks cuts nothing)
    int busiest = most;
    if (sorts) busiest = deal(p, bins, room, order);
    s.groups = max(1, min(p.groups, max((s.units + kFew - 1) / kFew, min(s.units, pairs))));
    const long long each = (s.units + s.groups - 1) / s.groups, whole = kChunkCost * static_cast<long long>(busiest);
    const long long line = kLineCost + kChunkCost * each + 95 * min(each, static_cast<long long>(most));
    const bool alike = least == most && pairs <= p.groups;
    const int parts = alike ? max(1, min(p.groups / pairs, most / kLeastCut)) : 1;
    const long long cut = parts > 1 ? 700 + 50 * parts + 280LL * ((most + parts - 1) / parts) : line;
    s.whole = p.whole || (packs && whole <= cut && whole <= line);
    if (!s.whole && parts > 1 && cut <= line) s.groups = pairs * parts;
    s.u0 = s.u1 = s.b = s.h = 0;
    if (s.whole) {
        s.groups = bins;
        if (g < bins) {
            const int at = g / p.Hv;
            s.b = sorts ? order[at] : at;
            s.h = g - at * p.Hv;
            s.u1 = sorts ? dealt_chunks(p, g, bins, room + kMostSorted) : seq_of(p, s.b).chunks;
        }
    } else if (g < s.groups) {
        s.u0 = begin_of(s.units, g, s.groups);
        s.u1 = begin_of(s.units, g + 1, s.groups);
    }
    return s;
}

// A place on the line: chunk k of head h of sequence b.
struct Place {
    int b, h, k;
    Seq s;
};

// Where unit u is (there is such a unit).
__device__ __forceinline__ Place place_of(const LinearParams &p, int u) {
    const int lane = threadIdx.x & 31;
    Place o;
    for (int c = 0, at = 0;; c += 32 * kEachLane) {
        int least, most;  // (not asked for)
        const int mine = units_of(p, c + kEachLane * lane, false, least, most);
        int x = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, off);
            if (lane >= off) x += y;
        }
        const unsigned past = __ballot_sync(0xffffffffu, u < at + x);
        if (past || c + 32 * kEachLane >= p.B) {
            const int w = past ? __ffs(past) - 1 : 0;
            int left = u - at - __shfl_sync(0xffffffffu, x - mine, w);
            o.b = c + kEachLane * w;
            o.s = seq_of(p, o.b);
            while (left >= o.s.chunks * p.Hv && o.b + 1 < p.B) {
                left -= o.s.chunks * p.Hv;
                o.s = seq_of(p, ++o.b);
            }
            o.h = left / max(1, o.s.chunks);
            o.k = left - o.h * o.s.chunks;
            return o;
        }
        at += __shfl_sync(0xffffffffu, x, 31);
    }
}

constexpr int kHead = 256, kTail = 512, kFirst = 1024;  // flags beside a chunk's tokens

// The chunks of a share one by one.
struct Chunk {
    int b, h, t0, valid;  // first token, tokens
    bool head, tail;      // the first of its piece of a sequence, the sequence's last
    bool first;           // the sequence's first
    long long slot;       // the sequence's
};
// The place after sequence b of head h: the next head's, or the next sequence's; or the next of the whole
// sequences (one function for all roles: the instruction cache).
__device__ __noinline__ Place after(const LinearParams &p, int b, int h, int round, const uint8_t *order) {
    Place o;
    o.k = 0;
    if (order) {
        const int j = dealt(round, static_cast<int>(blockIdx.x), min(p.B * p.Hv, p.groups)), i = j / p.Hv;
        o.b = order[i];
        o.h = j - i * p.Hv;
        o.s = seq_of(p, o.b);
        return o;
    }
    o.b = b;
    o.h = h + 1;
    if (o.h == p.Hv) {
        o.h = 0;
        do o.s = seq_of(p, ++o.b);
        while (o.s.chunks == 0);
    } else {
        o.s = seq_of(p, b);
    }
    return o;
}
struct Cursor {
    Place at;
    int left;
    bool head;
    int round;             // of whole sequences
    const uint8_t *order;  // of those, or none
    __device__ __forceinline__ Cursor(const Place &o, int n, const uint8_t *f) : at(o), left(n), head(true), round(0), order(f) {}
    __device__ __forceinline__ bool next(const LinearParams &p, Chunk &c) {
        if (left <= 0) return false;
        --left;
        c.b = at.b;
        c.h = at.h;
        c.t0 = at.s.t0 + at.k * kC;
        c.valid = max(0, min(kC, at.s.len - at.k * kC));
        c.first = at.k == 0;
        c.slot = at.s.slot;
        c.head = head || c.first;
        c.tail = at.k + 1 == at.s.chunks;
        head = false;
        if (++at.k == at.s.chunks && left > 0) at = after(p, at.b, at.h, ++round, order);
        return true;
    }
};

// A wait of a whole warp, as all_wait; what it does when the phase is not there yet is one function for all
// roles (the instruction cache).
__device__ __noinline__ bool long_wait(uint32_t b, unsigned parity, int *stop) {
    return __all_sync(0xffffffffu, wait_or_stop(b, parity, stop));
}
__device__ __forceinline__ bool phase(uint32_t b, int parity, int *stop) {
    return __all_sync(0xffffffffu, bar_try(b, static_cast<unsigned>(parity & 1))) || long_wait(b, static_cast<unsigned>(parity & 1), stop);
}

// Whether a predicate holds for all of the 128 threads that meet at barrier 1.
__device__ __forceinline__ bool all_of(bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %1, 0;\n\t"
        "bar.red.and.pred q, 1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(v ? 1u : 0u)
        : "memory");
    return r != 0;
}

// The copy of a chunk's outputs to memory; its thread's copies so far have read shared memory, or are done.
__device__ __forceinline__ void tma_store_4d(uint32_t src, const CUtensorMap *map, int c0, int c1, int c2, int c3) {
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(src)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void copies_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Scratch: exp of the sum of g of each share's cut piece; what the joining is to do from each share on;
// the pieces' states (what the next share begins with, after the joining); what cut sequences begin with.
__device__ __forceinline__ int4 *joins_of(const LinearParams &p) { return reinterpret_cast<int4 *>(p.ws + (p.groups + 3) / 4 * 4); }
__device__ __forceinline__ float *state_of(const LinearParams &p, int g) {
    return p.ws + (p.groups + 3) / 4 * 4 + 4 * p.groups + static_cast<long long>(g) * p.Dk * p.Dv;
}
__device__ __forceinline__ float *begin_state(const LinearParams &p, int g) { return state_of(p, p.groups + g); }

// ------------------------------------------------------------------------- sums of exponents
struct Pair {
    float hi, lo;
};
__device__ __forceinline__ Pair add(Pair a, Pair b) {
    const float s = a.hi + b.hi, bb = s - a.hi;
    const float e = (a.hi - (s - bb)) + (b.hi - bb) + (a.lo + b.lo);
    Pair r;
    r.hi = s + e;
    r.lo = e - (r.hi - s);
    return r;
}
__device__ __forceinline__ float less(Pair a, Pair b) { return (a.hi - b.hi) + (a.lo - b.lo); }
__device__ __forceinline__ Pair shfl(Pair a, int from) {
    return Pair{__shfl_sync(0xffffffffu, a.hi, from), __shfl_sync(0xffffffffu, a.lo, from)};
}

// g of tokens 2 lane and 2 lane + 1 of a chunk (0 behind its tokens), in base 2.
struct Decays {
    float a, b;
};
__device__ __forceinline__ Decays load_g(const LinearParams &p, const Chunk &c) {
    const int i = 2 * (threadIdx.x & 31);
    const float *at = p.g + (c.t0 + static_cast<long long>(i)) * p.g_token + c.h * p.g_head;
    Decays d;
    d.a = i < c.valid ? at[0] : 0.0f;
    d.b = i + 1 < c.valid ? at[p.g_token] : 0.0f;
    return d;
}
// Sums up to the lane's two tokens (inclusive), and the chunk's.
__device__ __forceinline__ void sums_of(Decays d, Pair &a, Pair &b, Pair &all) {
    constexpr float kLog2e = 1.4426950408889634f;
    const int lane = threadIdx.x & 31;
    d.a *= kLog2e;
    d.b *= kLog2e;
    d.a = d.a < kLeast ? kLeast : d.a;  // (NaN stays)
    d.b = d.b < kLeast ? kLeast : d.b;
    const Pair pa{d.a, 0.0f}, pb{d.b, 0.0f};
    Pair x = add(pa, pb);
#pragma unroll 1
    for (int off = 1; off < 32; off <<= 1) {
        const Pair y{__shfl_up_sync(0xffffffffu, x.hi, off), __shfl_up_sync(0xffffffffu, x.lo, off)};
        if (lane >= off) x = add(y, x);
    }
    b = x;
    all = shfl(x, 31);
    Pair before{__shfl_up_sync(0xffffffffu, x.hi, 1), __shfl_up_sync(0xffffffffu, x.lo, 1)};
    if (lane == 0) before = Pair{0.0f, 0.0f};
    a = add(before, pa);
}

// The product with A in tensor memory.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u)
        : "memory");
}

// An operand whose rows are not along k: 64 elements x 8 k an atom, the next 64 elements kPart on.
__device__ __forceinline__ uint64_t mn_desc(uint32_t addr) {
    return tc05::kDescHi | (static_cast<uint64_t>(kPart >> 4) << 16) | static_cast<uint64_t>((addr & 0x3FFFFu) >> 4);
}
__host__ __device__ constexpr uint32_t idesc_of(int m, int n, bool a_mn, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
           (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// 16 lanes x 4 N columns (N = 2, 4 here): register 2 i of lane l goes to row l / 4, column 4 i + l % 4, register 2 i + 1
// to row l / 4 + 8.  This is how turned 8 x 8 matrices of BF16 pairs come from shared memory.
__device__ __forceinline__ void tmem_st_turned(uint32_t addr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st_turned(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// Tokens t0 .. t0 + 15 of elements d0 .. d0 + 15 of a chunk in shared memory, turned: register 2 i + j of lane l has
// tokens t0 + 8 i + 2 (l % 4) and the next one of element d0 + 8 j + l / 4.
__device__ __forceinline__ void load_turned(uint32_t chunk, int t0, int d0, uint32_t &r0, uint32_t &r1, uint32_t &r2, uint32_t &r3) {
    const int lane = threadIdx.x & 31, m = lane >> 3;
    const int row = t0 + 8 * (m >> 1) + (lane & 7), u = (d0 >> 3) + (m & 1);
    const uint32_t at = chunk + (u >> 3) * kPart + row * 128 + (((u & 7) ^ (row & 7)) << 4);
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(at)
                 : "memory");
}

__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ void unpack2(unsigned long long v, uint32_t &a, uint32_t &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(v));
}
__device__ __forceinline__ unsigned long long pack2(uint32_t a, uint32_t b) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
    return r;
}
// Two BF16 numbers, each times its factor, as three pairs of BF16 numbers whose sums the FP32 products
// are: 8 bits each, cut off.
__device__ __forceinline__ void split(uint32_t v, unsigned long long f, uint32_t (&o)[3]) {
    const unsigned long long minus = pack2(0xbf800000u, 0xbf800000u);  // -1, -1
    unsigned long long x = mul2(pack2(v << 16, v & 0xffff0000u), f);
#pragma unroll
    for (int m = 0; m < 3; ++m) {
        uint32_t a, b;
        unpack2(x, a, b);
        o[m] = __byte_perm(a, b, 0x7632);
        if (m < 2) x = ffma2(pack2(a & 0xffff0000u, b & 0xffff0000u), minus, x);
    }
}

// 32 columns of the warp's lanes.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, "
        "%20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
          "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
          "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, "
        "%21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
        "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
        "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

// A chunk's keys times their factors w, as three BF16 numbers each (arrays DK / 64 parts apart), by eight warps,
// 32 units of 16 bytes at a time.  Rows from `valid` on are 0, whatever lies there.
template <int DK>
__device__ __forceinline__ void scale_keys(const uint8_t *k, uint8_t *out, const float *w, int warp, int valid) {
    constexpr int kUnits = DK / 8, kRows = 32 / kUnits, kEach = kC / 8;  // units a row, rows at a time, rows a warp
    constexpr int kKeys = DK / 64 * kPart;
    const int lane = threadIdx.x & 31, u = lane % kUnits;
    const int row0 = warp * kEach + lane / kUnits;
    auto place = [&](int row) { return (u >> 3) * kPart + row * 128 + (((u & 7) ^ (row & 7)) << 4); };
    uint4 next = *reinterpret_cast<const uint4 *>(k + place(row0));
#pragma unroll 1
    for (int row = row0; row < (warp + 1) * kEach; row += kRows) {
        const uint4 x = next;
        const float f = w[row];
        if (row + kRows < (warp + 1) * kEach) next = *reinterpret_cast<const uint4 *>(k + place(row + kRows));
        const bool in = row < valid;
        const uint32_t v[4] = {x.x, x.y, x.z, x.w};
        const unsigned long long ff = pack_f32x2(f, f);
        uint32_t o[4][3];
#pragma unroll
        for (int e = 0; e < 4; ++e) split(in ? v[e] : 0u, ff, o[e]);
        uint8_t *to = out + place(row);
#pragma unroll
        for (int s = 0; s < 3; ++s) *reinterpret_cast<uint4 *>(to + s * kKeys) = make_uint4(o[0][s], o[1][s], o[2][s], o[3][s]);
    }
}

__host__ __device__ constexpr int chunk_bytes(int dk, int dv, bool with_q) { return ((with_q ? 2 : 1) * dk + dv) / 64 * kPart; }
// barriers, and arrays of each chunk's tokens or values
constexpr int kMiscOut = 1024 + 3 * kSums * kC * 4 + 4 * 128 * 4 + kMostSorted;
constexpr int kOutStage = kC * 256;  // a chunk's outputs on their way
__host__ __device__ constexpr int out_fixed(int dk) { return 2 * 3 * dk / 64 * kPart + kPart + kOutStage + kMiscOut; }
constexpr int kAhead = 8;  // chunks whose g the state kernel has on their way
constexpr int kStateFixed = 512 + 4 * kC * 4 + kAhead * kC * 4 + 64;
// Columns of tensor memory: the state kernel's (U, two buffers of keys in three numbers), the output kernel's
// (two buffers of O1 and of values: O1 is what the next state waits for, not the outputs' warps).
constexpr int kU = 0, kKeyT = 128;
constexpr int kState = 0, kSb = 128, kA = 192, kO1 = 256, kO2 = 384, kValueT = 448;

// ------------------------------------------------------------------------ 1. states of cut pieces
template <int DK, bool COUNTS>
__global__ void __launch_bounds__(kStateThreads, 1) linear_states_kernel(const __grid_constant__ LinearParams p) {
    constexpr int kKParts = DK / 64, kKeys = kKParts * kPart, kWarps = 4;
    extern __shared__ uint8_t raw[];
    uint8_t *base = raw + ((1024u - (saddr(raw) & 1023u)) & 1023u);
    const int stage = chunk_bytes(DK, p.Dv, false), S = p.stages;
    uint8_t *misc = base + S * stage;
    uint64_t *bars = reinterpret_cast<uint64_t *>(misc);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(misc + 256);
    int &stop = *reinterpret_cast<int *>(misc + 260);
    float *wk = reinterpret_cast<float *>(misc + 512);  // [4][64] exp of the sum of g behind a key in its chunk
    float *gs = wk + 4 * kC;                            // [kAhead][64] g
    float2 *sums = reinterpret_cast<float2 *>(gs + kAhead * kC);  // [4] a chunk's sum of g
    const uint32_t full = saddr(bars), empty = full + 8 * kStages, kready = empty + 8 * kStages, kfree = kready + 16, fin = kfree + 32,
                   gready = fin + 8;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = static_cast<int>(blockIdx.x);
    if (threadIdx.x == 0) {
        prefetch_tmap(&p.tk);
        prefetch_tmap(&p.tv);
        stop = 0;
        for (int i = 0; i < S; ++i) {
            bar_init(full + 8 * i, 1);
            bar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) bar_init(kready + 8 * i, kWarps);
        for (int i = 0; i < 4; ++i) {
            bar_init(kfree + 8 * i, 1);
            bar_init(gready + 8 * i, 1);
        }
        bar_init(fin, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    pdl_wait();
    const Share sh = share_of<COUNTS>(p, g, false, reinterpret_cast<int *>(base), base + 4 * (2 * kMostSorted + 1));
    Place last;
    last.k = 0;
    last.s.chunks = 0;
    if (sh.u1 > sh.u0 && !sh.whole) last = place_of(p, sh.u1 - 1);
    const bool cut = last.k + 1 < last.s.chunks;  // a sequence goes on behind this share
    if (threadIdx.x == 0) {
        // Where it begins here: the shares behind which it goes on (up to, not with, the one that has its
        // last chunk), its sequence and head.
        int4 join = make_int4(0, 0, 0, 0);
        if (cut && last.k < sh.u1 - sh.u0) {
            const long long u = sh.u1 - 1LL + (last.s.chunks - last.k - 1);  // its last chunk
            join = make_int4(g, static_cast<int>(((u + 1) * sh.groups - 1) / sh.units), last.b, last.h);
        }
        joins_of(p)[g] = join;
    }
    if (!cut) return;
    const int chunks = min(last.k + 1, sh.u1 - sh.u0);  // all of them whole
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(tmem_slot)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // The next kernels are this call's; they may come once nothing runs that was before it: this, and the return above,
    // stand behind the wait, and have to.  For the third kernel reads the call's offsets and slots before it waits (4
    // ragged prompts of up to 3000, 16 heads: 62.7 -> 61.2 us; the second lets it come at once, but comes itself
    // when all of this kernel's CTAs have got here).  Nor before this
    // CTA has its tensor memory: a kernel behind them that takes some before it waits would hold what this one wants.
    pdl_launch_dependents();
    const uint32_t tmem = *tmem_slot;
    const bool stall = (p.flags & kFlagTestStall) != 0;
    int issued = 0;
    if (warp == 0) {
        const uint64_t policy = policy_of(false);
        int slot = 0;
        unsigned ph = 1;
        for (int n = 0; n < chunks; ++n) {
            if (n >= S && !phase(empty + 8 * slot, ph, &stop)) break;
            if (!stall) issued = n + 1;
            const uint32_t dst = saddr(base) + slot * stage, bar = full + 8 * slot;
            if (elect()) {
                bar_expect_tx(bar, static_cast<unsigned>(stage));
                if (!stall) {
                    const int t = last.s.t0 + (last.k - n) * kC;
                    tma_4d(dst, &p.tk, 0, t, 0, last.h / p.share, bar, policy);
                    tma_4d(dst + kKeys, &p.tv, 0, t, 0, last.h, bar, policy);
                }
            }
            __syncwarp();
            if (++slot == S) {
                slot = 0;
                ph ^= 1;
            }
        }
    } else if (warp == 1) {
        int slot = 0;
        unsigned ph = 0;
        const uint32_t d = alike(static_cast<int>(tmem)), idesc = alike(static_cast<int>(idesc_of(128, p.Dv, false, true)));
        for (int n = 0; n < chunks; ++n) {
            if (!phase(full + 8 * slot, ph, &stop) || !phase(kready + 8 * (n & 1), (n >> 1) & 1, &stop)) break;
            tc_fence_after();
            if (elect()) {
                const uint64_t b = mn_desc(saddr(base) + slot * stage + kKeys);
                const uint32_t a = d + kKeyT + 96 * (n & 1);
#pragma unroll
                for (int part = 0; part < 3; ++part)
#pragma unroll
                    for (int kk = 0; kk < kC / 16; ++kk)
                        mma_ts(d + kU, a + 32 * part + 8 * kk, b + kk * (2048 >> 4), idesc, n != 0 || part != 0 || kk != 0);
                mma_commit(empty + 8 * slot);
                mma_commit(kfree + 8 * (n & 3));
            }
            __syncwarp();
            if (++slot == S) {
                slot = 0;
                ph ^= 1;
            }
        }
        finish(fin, &stop);
    } else if (warp >= 10) {
        // The sums of g, every other chunk a warp (its scan takes 1300 cycles, with one warp what a chunk
        // took), up to four chunks ahead of the keys; the copies of g are further ahead.
        auto fetch = [&](int n) {
            if (n < chunks) {
                const float *from = p.g + (last.s.t0 + static_cast<long long>(last.k - n) * kC + 2 * lane) * p.g_token + last.h * p.g_head;
                const uint32_t to = saddr(gs + (n & (kAhead - 1)) * kC + 2 * lane);
                copy4(to, from);
                copy4(to + 4, from + p.g_token);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        for (int n = warp - 10; n < kAhead - 2; n += 2) fetch(n);
        for (int n = warp - 10; n < chunks; n += 2) {
            fetch(n + kAhead - 2);
            asm volatile("cp.async.wait_group %0;" ::"n"(kAhead / 2 - 1) : "memory");  // (a lane reads what it copied)
            const float2 v = *reinterpret_cast<const float2 *>(gs + (n & (kAhead - 1)) * kC + 2 * lane);
            Pair a, b, all;
            sums_of(Decays{v.x, v.y}, a, b, all);
            if (n >= 3 && !phase(kfree + 8 * ((n - 3) & 3), (n - 3) >> 2, &stop)) break;  // (the factors of n - 4 are read)
            *reinterpret_cast<float2 *>(&wk[(n & 3) * kC + 2 * lane]) = make_float2(exp2f(less(all, a)), exp2f(less(all, b)));
            if (lane == 0) sums[n & 3] = make_float2(all.hi, all.lo);
            __syncwarp();
            if (lane == 0) bar_arrive(gready + 8 * (n & 3));
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        // keys: a warp's 32 elements (a quarter of the lanes); four warps take every other chunk
        const int q = warp & 3, half = (warp - 2) >> 2, d0 = 32 * q;
        const uint32_t quarter = static_cast<uint32_t>(32 * q) << 16;
        bool ok = true;
        Pair after{0.0f, 0.0f};  // the sum of g behind the chunk, to the piece's end
        auto more = [&](int n) {  // chunk n's is known, and counts from here on
            const float2 sum = sums[n & 3];
            after = add(Pair{sum.x, sum.y}, after);
        };
        int slot = half % S;
        unsigned ph = static_cast<unsigned>(half / S) & 1u;
        for (int n = half; n < chunks; n += 2) {
            if (n > 0) {
                if (!(ok = phase(gready + 8 * ((n - 1) & 3), (n - 1) >> 2, &stop))) break;
                more(n - 1);
            }
            ok = phase(gready + 8 * (n & 3), n >> 2, &stop) && phase(full + 8 * slot, ph, &stop) &&
                 (n < 2 || phase(kfree + 8 * ((n - 2) & 3), (n - 2) >> 2, &stop));
            if (!ok) break;
            tc_fence_after();
            if (d0 < DK) {
                const float behind = exp2f(after.hi + after.lo);
#pragma unroll 1
                for (int part = 0; part < 4; ++part) {  // 16 elements x 32 tokens
                    const int h = part & 1, t0 = 32 * (part >> 1);
                    uint32_t r[8], o[3][8];
                    load_turned(saddr(base) + slot * stage, t0, d0 + 16 * h, r[0], r[1], r[2], r[3]);
                    load_turned(saddr(base) + slot * stage, t0 + 16, d0 + 16 * h, r[4], r[5], r[6], r[7]);
                    // the factors of tokens t0 + 8 i + 2 (lane % 4) and the next
                    const unsigned long long *w = reinterpret_cast<const unsigned long long *>(wk + (n & 3) * kC + t0) + (lane & 3);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const unsigned long long f = mul2(w[4 * i], pack_f32x2(behind, behind));
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            uint32_t s[3];
                            split(r[2 * i + j], f, s);
#pragma unroll
                            for (int m = 0; m < 3; ++m) o[m][2 * i + j] = s[m];
                        }
                    }
#pragma unroll
                    for (int m = 0; m < 3; ++m)
                        tmem_st_turned(tmem + quarter + (static_cast<uint32_t>(16 * h) << 16) + kKeyT + 96 * (n & 1) + 32 * m + t0 / 2, o[m]);
                }
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            }
            more(n);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(kready + 8 * (n & 1));
            slot += 2;
            if (slot >= S) {
                slot -= S;
                ph ^= 1;
            }
        }
        if (ok && chunks > 0 && ((chunks - 1) & 1) != half) {
            // the last chunk was the others'
            if ((ok = phase(gready + 8 * ((chunks - 1) & 3), (chunks - 1) >> 2, &stop))) more(chunks - 1);
        }
        // the piece's state, [Dk][Dv]: a row a lane, half of the columns a warp
        ok = ok && phase(fin, 0, &stop) && *reinterpret_cast<volatile int *>(&stop) == 0;
        ok = __all_sync(0xffffffffu, ok);
        const float nan = __int_as_float(0x7fc00000);
        tc_fence_after();
        if (d0 < DK) {
            float4 *to = reinterpret_cast<float4 *>(state_of(p, g) + (d0 + lane) * p.Dv);
            for (int col = half * (p.Dv / 2); col < (half + 1) * (p.Dv / 2); col += 16) {
                uint32_t v[16];
                if (ok) tc05::tmem_ld16(tmem + quarter + kU + col, v);
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                    to[(col + i) / 4] = ok ? make_float4(__uint_as_float(v[i]), __uint_as_float(v[i + 1]), __uint_as_float(v[i + 2]),
                                                         __uint_as_float(v[i + 3]))
                                           : make_float4(nan, nan, nan, nan);
            }
        }
        if (warp == 2 && lane == 0) p.ws[g] = ok ? exp2f(after.hi + after.lo) : nan;
    }
    __syncwarp();
    if (lane == 0 && *reinterpret_cast<volatile int *>(&stop) && warp == 0)
        for (int i = max(0, issued - S); i < issued; ++i) landed(full + 8 * (i % S), (i / S) & 1);
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 32 && stop) atomicOr(p.err, 1);
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

// ------------------------------------------------------------------------------------ 2. joining
// Along a cut sequence, from the share it begins in: S' = exp(G) S + U, in place of U; and a copy of what it
// begins with, for the third kernel, whose other CTAs may have written its last state by the time it is
// read.  A thread has kJoinEach groups of four elements.
constexpr int kJoinThreads = 256, kJoinEach = 4, kJoinBatch = 2;
__global__ void __launch_bounds__(kJoinThreads) linear_join_kernel(const __grid_constant__ LinearParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const int4 join = joins_of(p)[blockIdx.x];
    if (join.x >= join.y) return;
    const int all = p.Dk * p.Dv / 4, step = static_cast<int>(gridDim.y) * kJoinThreads;
    const int at = static_cast<int>(blockIdx.y) * kJoinThreads + static_cast<int>(threadIdx.x);
    const long long slot = p.slots[join.z];
    const float4 *from = nullptr;
    if (slot >= 0 && slot < p.pool && !(p.fresh && p.fresh[join.z]))
        from = reinterpret_cast<const float4 *>(p.state + slot * p.s_slot + join.w * p.s_head);
    float4 s[kJoinEach];
    float4 *begin = reinterpret_cast<float4 *>(begin_state(p, join.x));
#pragma unroll
    for (int j = 0; j < kJoinEach; ++j) {
        const int e = at + j * step;
        s[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (from && e < all) s[j] = from[e];
    }
#pragma unroll
    for (int j = 0; j < kJoinEach; ++j)
        if (at + j * step < all) begin[at + j * step] = s[j];
    for (int i = join.x; i < join.y; i += kJoinBatch) {
        float4 u[kJoinBatch][kJoinEach];
        float f[kJoinBatch];
#pragma unroll
        for (int m = 0; m < kJoinBatch; ++m)
            if (i + m < join.y) {
                f[m] = p.ws[i + m];
                const float4 *w = reinterpret_cast<const float4 *>(state_of(p, i + m));
#pragma unroll
                for (int j = 0; j < kJoinEach; ++j)
                    if (at + j * step < all) u[m][j] = w[at + j * step];
            }
#pragma unroll
        for (int m = 0; m < kJoinBatch; ++m)
            if (i + m < join.y) {
                float4 *w = reinterpret_cast<float4 *>(state_of(p, i + m));
#pragma unroll
                for (int j = 0; j < kJoinEach; ++j)
                    if (at + j * step < all) {
                        s[j].x = fmaf(f[m], s[j].x, u[m][j].x);
                        s[j].y = fmaf(f[m], s[j].y, u[m][j].y);
                        s[j].z = fmaf(f[m], s[j].z, u[m][j].z);
                        s[j].w = fmaf(f[m], s[j].w, u[m][j].w);
                        w[at + j * step] = s[j];
                    }
            }
    }
}

// ------------------------------------------------------------------------------------ 3. outputs
template <int DK, bool COUNTS>
__global__ void __launch_bounds__(kOutThreads, 1) linear_outputs_kernel(const __grid_constant__ LinearParams p) {
    constexpr int kKParts = DK / 64, kKeys = kKParts * kPart;
    extern __shared__ uint8_t raw[];
    uint8_t *base = raw + ((1024u - (saddr(raw) & 1023u)) & 1023u);
    const int vparts = p.Dv / 64, stage = chunk_bytes(DK, p.Dv, true), S = p.stages;
    uint8_t *keys = base + S * stage;   // two buffers of three numbers
    uint8_t *ps = keys + 6 * kKeys;     // P
    uint8_t *os = ps + kPart;           // outputs on their way
    uint8_t *misc = os + kOutStage;
    uint64_t *bars = reinterpret_cast<uint64_t *>(misc);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(misc + 512);
    int &stop = *reinterpret_cast<int *>(misc + 516);
    float *all_e = reinterpret_cast<float *>(misc + 528);  // [kSums] exp(G) of a chunk
    int *vbad = reinterpret_cast<int *>(misc + 768);       // [4][4][2] whether a warp's values are not all finite
    // [kSums][64] of each token: G_i, scale exp(G_i), exp(G - G_i)
    float *gs = reinterpret_cast<float *>(misc + 1024), *eg = gs + kSums * kC, *wk = eg + kSums * kC;
    int *first_bad = reinterpret_cast<int *>(wk + kSums * kC);  // [4][128] the first token with such a value
    uint8_t *order = reinterpret_cast<uint8_t *>(first_bad + 4 * 128);  // [kMostSorted] sequences, the longest first
    // [8] what chunk n is, by the warp of the sums: {b, h, first token, tokens and flags}
    int4 *told = reinterpret_cast<int4 *>(misc + 640);
    uint32_t at = saddr(bars);
    auto take = [&](int n) {
        const uint32_t b = at;
        at += 8 * n;
        return b;
    };
    // values, keys and queries of a slot by themselves: each is free when it was read
    const uint32_t vfull = take(kStages), kfull = take(kStages), qfull = take(kStages), vempty = take(kStages),
                   kempty = take(kStages), qempty = take(kStages), gready = take(kSums), kready = take(2), vready = take(2),
                   sdone = take(2), afull = take(1), afree = take(1), pready = take(1), odone = take(2), ofree = take(2),
                   sready = take(1), o1done = take(2), fin = take(2);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = static_cast<int>(blockIdx.x);
    if (threadIdx.x == 0) {
        prefetch_tmap(&p.tq);
        prefetch_tmap(&p.tk);
        prefetch_tmap(&p.tv);
        stop = 0;
        auto init = [&](uint32_t b, int n, int count) {
            for (int i = 0; i < n; ++i) bar_init(b + 8 * i, static_cast<unsigned>(count));
        };
        init(vfull, kStages, 1);
        init(kfull, kStages, 1);
        init(qfull, kStages, 1);
        init(vempty, kStages, 8);
        init(kempty, kStages, 9);
        init(qempty, kStages, 2);
        init(gready, kSums, 1);
        init(kready, 2, 8);
        init(vready, 2, 8);
        init(sdone, 2, 1);
        init(afull, 1, 1);
        init(afree, 1, 4);
        init(pready, 1, 4);
        init(odone, 2, 1);
        init(ofree, 2, 4);
        init(sready, 1, 4);
        init(o1done, 2, 1);
        init(fin, 2, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    const bool alone = p.whole || p.groups == 1;  // no kernel of this call before
    if (alone) pdl_wait();
    const Share sh = share_of<COUNTS>(p, g, g == 0 && warp == 0, reinterpret_cast<int *>(os), order);
    if (!alone) pdl_wait();
    if (sh.u1 <= sh.u0) return;
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(tmem_slot)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    Cursor cursor(sh.whole ? Place{sh.b, sh.h, 0, seq_of(p, sh.b)} : place_of(p, sh.u0), sh.u1 - sh.u0, sh.whole ? order : nullptr);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (p.flags & kFlagPdl) pdl_launch_dependents();  // (as above: not before the tensor memory is taken)
    const uint32_t tmem = *tmem_slot;
    const bool stall = (p.flags & kFlagTestStall) != 0;
    const float nan = __int_as_float(0x7fc00000);
    const int total = sh.u1 - sh.u0;
    const int q = warp & 3;
    const uint32_t quarter = static_cast<uint32_t>(32 * q) << 16;
    int issued = 0, vissued = 0, qissued = 0;
    Chunk c;
    // (the sums of chunk n + 8 come after the state's product of n + 6, so after O1 of n + 5, so after the outputs
    // of n + 3: what is told and summed of n is not read any more)
    auto hear = [&](int n) {
        const int4 v = told[n & 7];
        c.b = v.x;
        c.h = v.y;
        c.t0 = v.z;
        c.valid = v.w & 255;
        c.head = (v.w & kHead) != 0;
        c.tail = (v.w & kTail) != 0;
        c.first = (v.w & kFirst) != 0;
    };

    // Barriers with two phases in flight are pairs, taken in turn: none is passed twice before everyone who
    // waits on it has seen it once.
    if (warp == 0) {
        // -------------------------------------------------------------------- the copies
        const uint64_t policy = policy_of(false);
        int slot = 0;
        unsigned ph = 1;
        for (int n = 0; cursor.next(p, c); ++n) {
            const bool any = c.valid > 0;  // (of a sequence without tokens nothing is read)
            const int hk = c.h / p.share;
            // part of the slot: `parts` boxes of one operand
            auto copy = [&](uint32_t full, uint32_t empty, const CUtensorMap &map, int at, int parts, int head, int &count) {
                if (n >= S && !phase(empty + 8 * slot, ph, &stop)) return false;
                if (!stall && any) count = n + 1;
                if (elect()) {
                    const uint32_t dst = saddr(base) + slot * stage + at, bar = full + 8 * slot;
                    if (any)
                        bar_expect_tx(bar, static_cast<unsigned>(parts * kPart));
                    else
                        bar_arrive(bar);
                    if (!stall && any) tma_4d(dst, &map, 0, c.t0, 0, head, bar, policy);
                }
                __syncwarp();
                return true;
            };
            if (!copy(vfull, vempty, p.tv, 2 * kKeys, vparts, c.h, vissued) || !copy(kfull, kempty, p.tk, kKeys, kKParts, hk, issued) ||
                !copy(qfull, qempty, p.tq, 0, kKParts, hk, qissued))
                break;
            if (++slot == S) {
                slot = 0;
                ph ^= 1;
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------- the state's products, and O1 of it
        constexpr uint32_t kIdO = idesc_of(128, 64, false, false), kIdS = idesc_of(128, DK, false, true);
        const uint32_t d = alike(static_cast<int>(tmem));
        int slot = 0;
        unsigned ph = 0;
        for (int n = 0; n < total; ++n) {
            if (!phase(vready + 8 * (n & 1), n >> 1, &stop) || !phase(kready + 8 * (n & 1), n >> 1, &stop) || !phase(sready, n, &stop)) break;
            tc_fence_after();
            if (elect()) {
                const uint64_t b = mn_desc(saddr(keys) + (n & 1) * 3 * kKeys);
#pragma unroll 1
                for (int part = 0; part < 3; ++part)
#pragma unroll
                    for (int kk = 0; kk < kC / 16; ++kk)
                        mma_ts(d + kState, d + kValueT + 32 * (n & 1) + 8 * kk, b + ((part * kKeys) >> 4) + kk * (2048 >> 4), kIdS, true);
                mma_commit(sdone + 8 * (n & 1));
            }
            __syncwarp();
            if (!phase(qfull + 8 * slot, ph, &stop) || (n >= 2 && !phase(ofree + 8 * (n & 1), (n >> 1) - 1, &stop))) break;
            tc_fence_after();
            if (elect()) {
                const uint32_t st = saddr(base) + slot * stage;
#pragma unroll 1
                for (int i = 0; i < kKParts; ++i)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_ts(d + kO1 + 64 * (n & 1), d + kSb + 32 * i + 8 * kk, tc05::sw128_desc(st + i * kPart) + ((32 * kk) >> 4), kIdO,
                               i != 0 || kk != 0);
                mma_commit(o1done + 8 * (n & 1));
                mma_commit(qempty + 8 * slot);
            }
            __syncwarp();
            if (++slot == S) {
                slot = 0;
                ph ^= 1;
            }
        }
        finish(fin, &stop);
    } else if (warp == 3) {
        // ------------------------------------------- A, and O2 of it: a warp of their own, for neither
        // is to wait for what the others' operands wait for
        constexpr uint32_t kIdA = idesc_of(64, 64, false, false), kIdO = idesc_of(128, 64, false, false);
        const uint32_t d = alike(static_cast<int>(tmem));
        int slot = 0;
        unsigned ph = 0;
        for (int n = 0; n < total; ++n) {
            if (!phase(qfull + 8 * slot, ph, &stop) || !phase(kfull + 8 * slot, ph, &stop) || (n > 0 && !phase(afree, n - 1, &stop))) break;
            tc_fence_after();
            if (elect()) {
                const uint32_t st = saddr(base) + slot * stage;
#pragma unroll 1
                for (int i = 0; i < kKParts; ++i)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma(d + kA, tc05::sw128_desc(st + i * kPart) + ((32 * kk) >> 4),
                            tc05::sw128_desc(st + kKeys + i * kPart) + ((32 * kk) >> 4), kIdA, i != 0 || kk != 0);
                mma_commit(afull);
                mma_commit(kempty + 8 * slot);
                mma_commit(qempty + 8 * slot);
            }
            __syncwarp();
            if (++slot == S) {
                slot = 0;
                ph ^= 1;
            }
            if (!phase(vready + 8 * (n & 1), n >> 1, &stop) || !phase(pready, n, &stop) ||
                (n > 0 && !phase(ofree + 8 * ((n - 1) & 1), (n - 1) >> 1, &stop)))
                break;
            tc_fence_after();
            if (elect()) {
                const uint64_t b = tc05::sw128_desc(saddr(ps));
#pragma unroll
                for (int kk = 0; kk < kC / 16; ++kk) mma_ts(d + kO2, d + kValueT + 32 * (n & 1) + 8 * kk, b + ((32 * kk) >> 4), kIdO, kk != 0);
                mma_commit(odone + 8 * (n & 1));
            }
            __syncwarp();
        }
        finish(fin + 8, &stop);
    } else if (warp == 2) {
        // ---------------------------------------------------------------- the sums of decays
        Cursor ahead = cursor;
        Chunk nc;
        Decays next{0.0f, 0.0f};
        if (ahead.next(p, nc)) next = load_g(p, nc);
        for (int n = 0; n < total; ++n) {
            const Decays now = next;
            const int4 what = make_int4(nc.b, nc.h, nc.t0, nc.valid | (nc.head ? kHead : 0) | (nc.tail ? kTail : 0) | (nc.first ? kFirst : 0));
            if (ahead.next(p, nc)) {
                next = load_g(p, nc);
                // the state that a sequence begins with, on its way while the one before ends (200 prompts of up to
                // 200, 16 heads: 297 -> 261 us)
                if (nc.first && nc.slot >= 0 && !(p.fresh && p.fresh[nc.b]) && elect())
                    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p.state + nc.slot * p.s_slot + nc.h * p.s_head),
                                 "r"(p.Dk * p.Dv * 4)
                                 : "memory");
                __syncwarp();
            }
            Pair a, b, all;
            sums_of(now, a, b, all);
            if (n >= 2 && !phase(sdone + 8 * (n & 1), ((n >> 1) - 1) & 1, &stop)) break;
            const int buf = n & (kSums - 1), to = buf * kC + 2 * lane;
            *reinterpret_cast<float2 *>(&gs[to]) = make_float2(a.hi, b.hi);
            *reinterpret_cast<float2 *>(&eg[to]) = make_float2(p.scale * exp2f(a.hi + a.lo), p.scale * exp2f(b.hi + b.lo));
            *reinterpret_cast<float2 *>(&wk[to]) = make_float2(exp2f(less(all, a)), exp2f(less(all, b)));
            if (lane == 0) {
                all_e[buf] = exp2f(all.hi + all.lo);
                told[n & 7] = what;
            }
            __syncwarp();
            if (lane == 0) bar_arrive(gready + 8 * buf);
        }
    } else if (warp >= 16) {
        // ------------------------------------------- the values turned, and the scaled keys
        int slot = 0;
        unsigned ph = 0;
        for (int n = 0; n < total; ++n) {
            const int buf = n & (kSums - 1), b4 = n & 3;
            // (the sums come after the state's product that read this buffer of keys)
            if (!phase(gready + 8 * buf, n / kSums, &stop) || !phase(kfull + 8 * slot, ph, &stop)) break;
            hear(n);
            scale_keys<DK>(base + slot * stage + kKeys, keys + (n & 1) * 3 * kKeys, wk + buf * kC, warp - 16, c.valid);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
                bar_arrive(kready + 8 * (n & 1));
                bar_arrive(kempty + 8 * slot);
            }
            if (!phase(vfull + 8 * slot, ph, &stop) || (n >= 2 && !phase(odone + 8 * (n & 1), (n >> 1) - 1, &stop))) break;
            tc_fence_after();
            {
                // 16 elements x 64 tokens a warp
                const int h = (warp - 16) >> 2;
                bool any = false;
                // which of the rows have one that is not finite is told for all 16 of them
                int *fb = first_bad + 128 * b4 + 32 * q + 16 * h;
                if (32 * q < p.Dv) {
                    uint32_t r[16], x = 0u;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        load_turned(saddr(base) + slot * stage + 2 * kKeys, 16 * i, 32 * q + 16 * h, r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
                    // tokens behind the chunk's are 0, whatever lies there
                    if (c.valid < kC)
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int tok = 8 * (i >> 1) + 2 * (lane & 3);
                            r[i] = tok + 1 < c.valid ? r[i] : tok < c.valid ? r[i] & 0xffffu : 0u;
                        }
                    // infinities and NaN: 0 x v is not 0
#pragma unroll
                    for (int i = 0; i < 16; ++i) asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(x) : "r"(r[i]), "r"(0u));
                    any = __any_sync(0xffffffffu, x != 0u);
                    if (lane < 16) fb[lane] = kC;
                    if (any) {
                        // They become 0 in the products, which sum over later tokens too, and the row's outputs and
                        // states NaN from the first such token on.
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int tok = 8 * (i >> 1) + 2 * (lane & 3);
                            const bool lo = (r[i] & 0x7f80u) == 0x7f80u, hi = (r[i] & 0x7f800000u) == 0x7f800000u;
                            if (lo || hi) atomicMin(&fb[8 * (i & 1) + (lane >> 2)], lo ? tok : tok + 1);
                            r[i] = finite_or_zero(r[i]);
                        }
                    }
                    tmem_st_turned(tmem + quarter + (static_cast<uint32_t>(16 * h) << 16) + kValueT + 32 * (n & 1), r);
                    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                }
                if (lane == 0) vbad[8 * b4 + 2 * q + h] = any;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                bar_arrive(vready + 8 * (n & 1));
                bar_arrive(vempty + 8 * slot);
            }
            if (++slot == S) {
                slot = 0;
                ph ^= 1;
            }
        }
    } else if (warp >= 4 && warp < 8) {
        // -------------------------------------------------------------------- the state
        const int dv = 32 * q + lane;
        const bool mine = dv < p.Dv;
        float poison = 0.0f;  // NaN once the sequence had a value of this row that is not finite
        int n = 0;
        auto spoilt = [&](int m) {  // by chunk m
            if ((vbad[8 * (m & 3) + 2 * q] | vbad[8 * (m & 3) + 2 * q + 1]) && first_bad[128 * (m & 3) + dv] < kC) poison = nan;
        };
        for (; n < total; ++n) {
            const int buf = n & (kSums - 1);
            if (!phase(gready + 8 * buf, n / kSums, &stop)) break;
            hear(n);
            if (c.head) {
                poison = 0.0f;
                const float *from = nullptr;
                const long long s = p.slots[c.b];
                if (!c.first)
                    from = state_of(p, g - 1);
                else if (s >= 0 && s < p.pool && !(p.fresh && p.fresh[c.b])) {
                    // a sequence cut by the share's end begins with the second kernel's copy
                    from = p.state + s * p.s_slot + c.h * p.s_head;
                    const int a = p.cu[c.b], chunks = (p.cu[c.b + 1] - a + kC - 1) / kC;
                    if (chunks > total - n) from = begin_state(p, g);
                }
#pragma unroll 1
                for (int col = 0; col < DK; col += 32) {
                    uint32_t v[2][16];
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i >> 4][i & 15] = from && mine ? __float_as_uint(from[(col + i) * p.Dv + dv]) : 0u;
                    tmem_st16(tmem + quarter + kState + col, v[0]);
                    tmem_st16(tmem + quarter + kState + col + 16, v[1]);
                }
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            } else {
                if (!phase(sdone + 8 * ((n - 1) & 1), (n - 1) >> 1, &stop)) break;
                spoilt(n - 1);
            }
            // O1 of the chunk before has read Sb
            if (n > 0 && !phase(o1done + 8 * ((n - 1) & 1), (n - 1) >> 1, &stop)) break;
            tc_fence_after();
            const unsigned long long e = pack_f32x2(all_e[buf], all_e[buf]);
            const bool poisoned = __any_sync(0xffffffffu, poison != 0.0f);
#pragma unroll 1
            for (int col = 0; col < DK; col += 32) {
                uint32_t v[32], sb[16];
                tmem_ld32(tmem + quarter + kState + col, v);
                if (poisoned)
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + poison);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    sb[i] = bf16x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
                    unpack2(mul2(pack2(v[2 * i], v[2 * i + 1]), e), v[2 * i], v[2 * i + 1]);
                }
                tmem_st16(tmem + quarter + kSb + col / 2, sb);
                tmem_st32(tmem + quarter + kState + col, v);
            }
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            tc_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(sready);
            if (c.tail) {
                // the sequence's last state
                if (!phase(sdone + 8 * (n & 1), n >> 1, &stop)) break;
                spoilt(n);
                const Seq s = seq_of(p, c.b);
                if (s.slot >= 0 && (s.len > 0 || (p.fresh && p.fresh[c.b]))) {
                    float *to = p.state + s.slot * p.s_slot + c.h * p.s_head + dv;
                    tc_fence_after();
#pragma unroll 1
                    for (int col = 0; col < DK; col += 16) {
                        uint32_t v[16];
                        tc05::tmem_ld16(tmem + quarter + kState + col, v);
                        if (mine)
#pragma unroll
                            for (int i = 0; i < 16; ++i) to[(col + i) * p.Dv] = __uint_as_float(v[i]) + poison;
                    }
                    tc_fence_before();
                }
            }
        }
        // after a stop: NaN for the sequences that were not finished
        if (n < total)
            for (int i = 0; cursor.next(p, c); ++i) {
                const Seq s = seq_of(p, c.b);
                if (i < n || !c.tail || s.slot < 0 || !mine) continue;
                for (int col = 0; col < DK; ++col) p.state[s.slot * p.s_slot + c.h * p.s_head + col * p.Dv + dv] = nan;
            }
    } else if (warp >= 8 && warp < 12) {
        // ------------------------------------------------------------- the decays of a chunk
        for (int n = 0; n < total; ++n) {
            const int buf = n & (kSums - 1);
            if (!phase(gready + 8 * buf, n / kSums, &stop) || !phase(afull, n, &stop)) break;
            tc_fence_after();
            hear(n);
            const int i0 = 16 * q + (lane >> 2), j0 = 2 * (lane & 3);
            const float *gj = gs + buf * kC;
            const float g0 = gj[i0], g1 = gj[i0 + 8];
            // a row's tokens up to its own; none of a row behind the chunk's
            const int last0 = i0 < c.valid ? i0 : -1, last1 = i0 + 8 < c.valid ? i0 + 8 : -1;
            uint8_t *row = ps + i0 * 128;  // (O2 of the chunk before was issued before A)
#pragma unroll 1
            for (int t = 0; t < 2; ++t) {
                uint32_t r[16];
                tmem_ld_s(tmem + quarter + kA + 32 * t, r);
                asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const int j = 32 * t + 8 * m + j0;
                    const float2 g = *reinterpret_cast<const float2 *>(&gj[j]);
                    // (later tokens' exponents may overflow: they are not used)
                    const float a = j <= last0 ? ex2(g0 - g.x) * __uint_as_float(r[4 * m]) : 0.0f;
                    const float b = j + 1 <= last0 ? ex2(g0 - g.y) * __uint_as_float(r[4 * m + 1]) : 0.0f;
                    const float e = j <= last1 ? ex2(g1 - g.x) * __uint_as_float(r[4 * m + 2]) : 0.0f;
                    const float f = j + 1 <= last1 ? ex2(g1 - g.y) * __uint_as_float(r[4 * m + 3]) : 0.0f;
                    const int to = (((4 * t + m) ^ (lane >> 2)) << 4) + 2 * j0;  // i0 % 8 = lane / 4
                    *reinterpret_cast<uint32_t *>(row + to) = bf16x2(a, b);
                    *reinterpret_cast<uint32_t *>(row + 8 * 128 + to) = bf16x2(e, f);
                }
            }
            tc_fence_before();
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
                bar_arrive(afree);
                bar_arrive(pready);
            }
        }
    } else if (warp >= 12) {
        // ------------------------------------------------------------------- the outputs
        // 32 tokens at a time, read in the 16 x 256-bit form, whose fragments stmatrix stores turned:
        // rows of a token's values, 16 bytes a thread from there on.
        const int tid = threadIdx.x - 12 * 32, c0 = 2 * (lane & 3);
        const uint32_t to_s = saddr(os);
        const unsigned long long scale = pack_f32x2(p.scale, p.scale);
        int n = 0;
        for (; n < total; ++n) {
            // the four warps go on together, or none (they meet at barriers); what was staged is stored
            if (tid == 0) copies_read();
            if (!all_of(phase(odone + 8 * (n & 1), n >> 1, &stop) && phase(o1done + 8 * (n & 1), n >> 1, &stop))) break;
            tc_fence_after();
            hear(n);
            const float *e = eg + (n & (kSums - 1)) * kC;
            const bool bad = (vbad[8 * (n & 3) + 2 * q] | vbad[8 * (n & 3) + 2 * q + 1]) != 0;
            uint16_t *out = p.out + static_cast<long long>(c.t0) * p.o_token + c.h * p.o_head;
            if (32 * q < p.Dv)
#pragma unroll 1
                for (int part = 0; part < 4; ++part) {  // 16 rows x 32 tokens
                    const int h = part & 1, t1 = 32 * (part >> 1);
                    const uint32_t from = tmem + quarter + (static_cast<uint32_t>(16 * h) << 16) + t1;
                    uint32_t a[16], b[16];
                    tmem_ld_s(from + kO1 + 64 * (n & 1), a);
                    tmem_ld_s(from + kO2, b);
                    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
                    if (bad)
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int first = first_bad[128 * (n & 3) + 32 * q + 16 * h + 8 * ((i >> 1) & 1) + (lane >> 2)];
                            if (t1 + 8 * (i >> 2) + c0 + (i & 1) >= first) b[i] = __float_as_uint(nan);
                        }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t o[4];
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            const int r = 8 * i + 2 * m;
                            const unsigned long long ee = *reinterpret_cast<const unsigned long long *>(&e[t1 + 16 * i + 8 * (m >> 1) + c0]);
                            uint32_t x, y;
                            unpack2(ffma2(ee, pack2(a[r], a[r + 1]), mul2(scale, pack2(b[r], b[r + 1]))), x, y);
                            o[m] = bf16x2(__uint_as_float(x), __uint_as_float(y));
                        }
                        stmatrix_turned(to_s + (q >> 1) * kPart + (t1 + 16 * i + 8 * (lane >> 4) + (lane & 7)) * 128 +
                                            (((4 * (q & 1) + 2 * h + ((lane >> 3) & 1)) ^ (lane & 7)) << 4), o);
                    }
                }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(ofree + 8 * (n & 1));
            const bool copied = p.out16 && c.valid == kC;
            if (copied) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            asm volatile("bar.sync 1, 128;" ::: "memory");
            if (copied) {
                if (tid == 0) tma_store_4d(to_s, &p.to, 0, c.t0, 0, c.h);
                continue;
            }
            const int shift = p.Dv == 128 ? 4 : 3, end = c.valid << shift;
#pragma unroll 1
            for (int i = tid; i < end; i += 128) {
                const int tok = i >> shift, u = i & ((1 << shift) - 1);
                const uint4 v = *reinterpret_cast<const uint4 *>(os + (u >> 3) * kPart + tok * 128 + (((u & 7) ^ (tok & 7)) << 4));
                uint16_t *to = out + tok * p.o_token + 8 * u;
                if (p.out16) {
                    *reinterpret_cast<uint4 *>(to) = v;
                } else {
                    uint32_t *w = reinterpret_cast<uint32_t *>(to);
                    w[0] = v.x;
                    w[1] = v.y;
                    w[2] = v.z;
                    w[3] = v.w;
                }
            }
        }
        if (tid == 0) copies_done();
        // after a stop: NaN for the chunks that were not finished
        if (n < total)
            for (int i = 0; cursor.next(p, c); ++i)
                if (i >= n && tid < p.Dv)
                    for (int m = 0; m < c.valid; ++m)
                        p.out[(static_cast<long long>(c.t0) + m) * p.o_token + c.h * p.o_head + tid] = 0x7fc0;
    }
    __syncwarp();
    // after a stop: the copies issued have landed before the shared memory goes
    if (lane == 0 && *reinterpret_cast<volatile int *>(&stop) && warp == 0) {
        for (int i = max(0, issued - S); i < issued; ++i) landed(kfull + 8 * (i % S), (i / S) & 1);
        for (int i = max(0, vissued - S); i < vissued; ++i) landed(vfull + 8 * (i % S), (i / S) & 1);
        for (int i = max(0, qissued - S); i < qissued; ++i) landed(qfull + 8 * (i % S), (i / S) & 1);
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 32 && stop) atomicOr(p.err, 1);
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

template <bool COUNTS>
const void *states_kernel(bool wide) {
    return wide ? reinterpret_cast<const void *>(&linear_states_kernel<128, COUNTS>) : reinterpret_cast<const void *>(&linear_states_kernel<64, COUNTS>);
}
template <bool COUNTS>
const void *outputs_kernel(bool wide) {
    return wide ? reinterpret_cast<const void *>(&linear_outputs_kernel<128, COUNTS>) : reinterpret_cast<const void *>(&linear_outputs_kernel<64, COUNTS>);
}

int stages_of(int dk, int dv, bool with_q) {
    const int room = static_cast<int>(kMaxSmemOptin) - 1024 - (with_q ? out_fixed(dk) : kStateFixed);
    return std::min(kStages, room / chunk_bytes(dk, dv, with_q));
}

// Shares of a line, at most: one an SM, of kLeastCut chunks, or one for each sequence and head.
int groups_of(const sgemm_linear_attention_t &a, int sms) {
    const long long units = (a.N / kC + 2 * a.B) * a.Hv;
    return static_cast<int>(std::max(1LL, std::min<long long>(sms, std::max((units + kLeastCut - 1) / kLeastCut, std::min(units, a.B * a.Hv)))));
}

sgemm_status_t check_sizes(const sgemm_linear_attention_t &a) {
    if (a.flags & ~(kDecodeFlags | SGEMM_FLAG_TEST_STALL)) return SGEMM_ERR_INVALID_ARG;
    if (a.N < 0 || a.B < 0 || a.Hk < 1 || a.Hv < a.Hk || a.Hv % a.Hk || a.Hv > 1024) return SGEMM_ERR_INVALID_ARG;
    if ((a.Dk != 64 && a.Dk != 128) || (a.Dv != 64 && a.Dv != 128)) return SGEMM_ERR_UNSUPPORTED_SHAPE;
    if (a.N >= (1LL << 31) / a.Hv || a.B >= (1LL << 28) / a.Hv) return SGEMM_ERR_UNSUPPORTED_SHAPE;
    return SGEMM_OK;
}

long long scratch(const sgemm_linear_attention_t &a, int groups) {
    return groups > 1 ? (groups + 3) / 4 * 16 + 16LL * groups + 2LL * groups * a.Dk * a.Dv * 4 : 0;
}

}  // namespace linear
}  // namespace sk

extern "C" sgemm_status_t sgemm_linear_attention_workspace(const sgemm_linear_attention_t *a, long long *bytes) {
    using namespace sk;
    using namespace sk::linear;
    if (!a || !bytes) return SGEMM_ERR_INVALID_ARG;
    *bytes = 0;
    sgemm_status_t st = check_sizes(*a);
    if (st != SGEMM_OK || a->B == 0) return st;
    int sms = 0, *err = nullptr;
    st = device_ready(&sms, &err);
    if (st != SGEMM_OK) return st;
    *bytes = scratch(*a, groups_of(*a, sms));
    return SGEMM_OK;
}

extern "C" sgemm_status_t sgemm_bf16_linear_attention(const sgemm_linear_attention_t *a, sgemm_stream_t stream) {
    using namespace sk;
    using namespace sk::linear;
    if (!a) return SGEMM_ERR_INVALID_ARG;
    sgemm_status_t st = check_sizes(*a);
    if (st != SGEMM_OK) return st;
    if (!std::isfinite(a->scale)) return SGEMM_ERR_INVALID_ARG;
    if (a->B == 0) return SGEMM_OK;
    if (!a->slots || !a->cu || (a->pool > 0 && !a->state) || (a->N > 0 && (!a->q || !a->k || !a->v || !a->g || !a->out)) || a->pool < 0 ||
        a->pool >= (1LL << 31) || a->workspace_bytes < 0)
        return SGEMM_ERR_INVALID_ARG;
    const LinearView io{a->q, a->k, a->v, a->g, a->state, a->out, a->q_token, a->q_head, a->k_token, a->k_head, a->v_token,
                        a->v_head, a->g_token, a->g_head, a->s_slot, a->s_head, a->o_token, a->o_head, a->N, a->pool, a->Hk,
                        a->Hv, a->Dk, a->Dv};
    st = check_linear(io);
    if (st != SGEMM_OK) return st;
    // the copies' strides
    if (a->N > 1 && (a->q_token < 8 || a->k_token < 8 || a->v_token < 8)) return SGEMM_ERR_INVALID_ARG;
    if ((a->Hk > 1 && (a->q_head < 8 || a->k_head < 8)) || (a->Hv > 1 && a->v_head < 8)) return SGEMM_ERR_INVALID_ARG;
    if (!aligned(a->slots, 8) || !aligned(a->cu, 4) || !aligned(a->fresh, 4) || !aligned(a->workspace, 16)) return SGEMM_ERR_MISALIGNED;
    if (linear_touches(io, a->slots, 8 * a->B) || linear_touches(io, a->cu, 4 * a->B + 4) || linear_touches(io, a->fresh, 4 * a->B))
        return SGEMM_ERR_INVALID_ARG;
    LinearParams p;
    std::memset(&p, 0, sizeof(p));
    int sms = 0;
    st = device_ready(&sms, &p.err);
    if (st != SGEMM_OK) return st;
    p.groups = groups_of(*a, sms);
    const long long need = scratch(*a, p.groups);
    if (need > 0 && (!a->workspace || a->workspace_bytes < need)) return SGEMM_ERR_NO_WORKSPACE;
    if (need > 0) {
        auto meets = [&](const void *b, long long bytes) { return b && rows_overlap(a->workspace, need, 0, b, bytes, 0, 1); };
        auto span = [&](long long tok, int heads, long long head, long long w) { return (a->N - 1) * tok + (heads - 1) * head + w; };
        if (linear_touches(io, a->workspace, need) || meets(a->q, 2 * span(a->q_token, a->Hk, a->q_head, a->Dk)) ||
            meets(a->k, 2 * span(a->k_token, a->Hk, a->k_head, a->Dk)) || meets(a->v, 2 * span(a->v_token, a->Hv, a->v_head, a->Dv)) ||
            meets(a->g, 4 * span(a->g_token, a->Hv, a->g_head, 1)) || meets(a->slots, 8 * a->B) || meets(a->cu, 4 * a->B + 4) ||
            meets(a->fresh, 4 * a->B))
            return SGEMM_ERR_INVALID_ARG;
    }
    // without tokens nothing is copied, and any address will do for the maps
    const long long rows = std::max(1LL, a->N);
    const void *none = reinterpret_cast<const void *>(4096);
    const CUtensorMapL2promotion promote = CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
    if (!map_4d(&p.tq, a->N ? a->q : none, a->Dk, rows, a->Hk, a->q_token, a->q_head, kC, a->Dk / 64, true, promote) ||
        !map_4d(&p.tk, a->N ? a->k : none, a->Dk, rows, a->Hk, a->k_token, a->k_head, kC, a->Dk / 64, true, promote) ||
        !map_4d(&p.tv, a->N ? a->v : none, a->Dv, rows, a->Hv, a->v_token, a->v_head, kC, a->Dv / 64, true, promote))
        return SGEMM_ERR_CUDA;
    p.g = a->g;
    p.state = a->state;
    p.slots = a->slots;
    p.cu = a->cu;
    p.fresh = a->fresh;
    p.out = a->out;
    p.ws = static_cast<float *>(a->workspace);
    p.g_token = a->g_token;
    p.g_head = a->g_head;
    p.s_slot = a->s_slot;
    p.s_head = a->s_head;
    p.o_token = a->o_token;
    p.o_head = a->o_head;
    p.pool = a->pool;
    p.N = a->N;
    p.B = static_cast<int>(a->B);
    p.Hv = a->Hv;
    p.share = a->Hv / a->Hk;
    p.Dk = a->Dk;
    p.Dv = a->Dv;
    p.scale = a->scale;
    p.out16 = aligned(a->out, 16) && a->o_token % 8 == 0 && a->o_head % 8 == 0 ? 1 : 0;
    if (p.out16 && !map_4d(&p.to, a->N ? a->out : none, a->Dv, rows, a->Hv, a->o_token, a->o_head, kC, a->Dv / 64, true, promote))
        return SGEMM_ERR_CUDA;
    p.flags = static_cast<int>(a->flags);
    // So few tokens that no sequence would be cut, if it had them all: neither a line nor two parts would pay against
    // the first two kernels' time (500 tokens, 16 heads: 20.4 us, 23.8 with them; 704, 16: 25.8, 29.8).
    const long long pairs = a->B * a->Hv, longest = (a->N + kC - 1) / kC;
    if (pairs <= p.groups && kChunkCost * longest <= kLineCost + kStarts) {
        p.whole = 1;
        p.groups = static_cast<int>(pairs);
    }
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    const bool wide = a->Dk == 128;
    const bool counts = pairs * longest >= kMostUnits;  // (chunks, if every sequence had all tokens)
    static std::atomic<unsigned long long> done[8];
    if (p.groups > 1 && !p.whole) {
        const void *fn = counts ? states_kernel<true>(wide) : states_kernel<false>(wide);
        if (!allow(fn, done[2 * counts + wide])) return SGEMM_ERR_CUDA;
        p.stages = stages_of(a->Dk, a->Dv, false);
        const size_t smem = std::max(kAloneSmem, 1024 + static_cast<size_t>(p.stages) * chunk_bytes(a->Dk, a->Dv, false) + kStateFixed);
        if (launch(fn, dim3(static_cast<unsigned>(p.groups)), dim3(kStateThreads), smem, cs, &p) != cudaSuccess) return SGEMM_ERR_CUDA;
        const unsigned slices = static_cast<unsigned>(a->Dk * a->Dv / 4 / kJoinThreads / kJoinEach);  // 1 .. 4
        if (launch(reinterpret_cast<const void *>(&linear_join_kernel), dim3(static_cast<unsigned>(p.groups), slices), dim3(kJoinThreads),
                   0, cs, &p) != cudaSuccess)
            return SGEMM_ERR_CUDA;
    }
    const void *fn = counts ? outputs_kernel<true>(wide) : outputs_kernel<false>(wide);
    if (!allow(fn, done[4 + 2 * counts + wide])) return SGEMM_ERR_CUDA;
    p.stages = stages_of(a->Dk, a->Dv, true);
    const size_t smem = 1024 + static_cast<size_t>(p.stages) * chunk_bytes(a->Dk, a->Dv, true) + out_fixed(a->Dk);
    if (launch(fn, dim3(static_cast<unsigned>(p.groups)), dim3(kOutThreads), smem, cs, &p) != cudaSuccess) return SGEMM_ERR_CUDA;
    return SGEMM_OK;
}
