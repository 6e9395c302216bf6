// Host helpers shared by the operators of sgemm_decode.h.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstring>

#include "internal.h"
#include "sgemm_decode.h"

namespace sk {

constexpr unsigned kDecodeFlags = SGEMM_FLAG_PDL | SGEMM_FLAG_WEIGHTS_READONLY;
constexpr int kErrBadIndex = 2;  // device error word: an index out of range was met and skipped

inline bool aligned(const void *p, unsigned bytes) {
    return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

// Whether two arrays of `rows` rows (`wa` and `wb` bytes wide, strides `sa` and
// `sb` bytes) share a byte.  Arrays of one stride are compared column by
// column, so that two column ranges of one buffer count as apart; arrays of
// different strides count as overlapping when their extents do.
inline bool rows_overlap(const void *a, long long wa, long long sa, const void *b, long long wb,
                         long long sb, long long rows) {
    if (!a || !b || rows < 1) return false;
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
    const uintptr_t ea = pa + static_cast<uintptr_t>((rows - 1) * sa + wa);
    const uintptr_t eb = pb + static_cast<uintptr_t>((rows - 1) * sb + wb);
    if (pa >= eb || pb >= ea) return false;
    if (sa != sb || sa < 1) return true;
    const uintptr_t s = static_cast<uintptr_t>(sa);
    if (pa <= pb) {
        const uintptr_t d = (pb - pa) % s;
        return d < static_cast<uintptr_t>(wa) || d + static_cast<uintptr_t>(wb) > s;
    }
    const uintptr_t d = (pa - pb) % s;
    return d < static_cast<uintptr_t>(wb) || d + static_cast<uintptr_t>(wa) > s;
}

// Whether a block of `n` bytes touches one of `rows` rows of `w` bytes, `s` bytes apart.
inline bool block_touches(const void *b, long long n, const void *a, long long w, long long s, long long rows) {
    if (!a || !b || n < 1 || w < 1 || rows < 1) return false;
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
    if (pb + static_cast<uintptr_t>(n) <= pa || pa + static_cast<uintptr_t>((rows - 1) * s + w) <= pb) return false;
    if (pb <= pa || s < w) return true;
    const uintptr_t d = (pb - pa) % static_cast<uintptr_t>(s);
    return d < static_cast<uintptr_t>(w) || d + static_cast<uintptr_t>(n) > static_cast<uintptr_t>(s);
}

// An array of T x H rows of `w` bytes, `tok` and `head` bytes apart.
struct Heads {
    const void *p;
    long long w, tok, head;
    long long extent(long long T, long long H) const { return (T - 1) * tok + (H - 1) * head + w; }
};

// Whether two such arrays (of the same T and H) share a byte: they are apart where their extents
// are, or, with one stride of both, where the ranges that a token, a head or a row takes of that
// stride are.
inline bool heads_overlap(const Heads &a, const Heads &b, long long T, long long H) {
    if (!rows_overlap(a.p, a.extent(T, H), 0, b.p, b.extent(T, H), 0, 1)) return false;
    if (T > 1 && !rows_overlap(a.p, a.extent(1, H), a.tok, b.p, b.extent(1, H), b.tok, T)) return false;
    if (H > 1 && !rows_overlap(a.p, a.extent(T, 1), a.head, b.p, b.extent(T, 1), b.head, H)) return false;
    if (T > 1 && H > 1 && a.tok == b.tok && a.head == b.head && a.tok > 0 && a.head > 0) {
        const bool inner = a.head <= a.tok;  // heads inside a token
        const long long step = inner ? a.head : a.tok, far = inner ? a.tok : a.head;
        if (far % step == 0)
            return rows_overlap(a.p, a.w, step, b.p, b.w, step, ((inner ? T : H) - 1) * (far / step) + (inner ? H : T));
    }
    return true;
}

inline bool valid_flags(unsigned flags) { return (flags & ~kDecodeFlags) == 0; }

// Allow a kernel all the shared memory that there is, once per device.
inline bool allow(const void *fn, std::atomic<unsigned long long> &done) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const unsigned long long bit = dev < 64 ? 1ULL << dev : 0ULL;
    if (!(done.load(std::memory_order_acquire) & bit)) {
        if (allow_max_dynamic_smem(fn) != cudaSuccess) return false;
        done.fetch_or(bit, std::memory_order_release);
    }
    return true;
}

// Launch `fn` with one parameter structure, as a programmatic dependent of the
// previous kernel on the stream.  A call's first kernel waits for that one
// (pdl_wait) before it reads or writes any memory, so the order is the stream's.
// A later kernel of the call may read the call's inputs before it waits, and only
// those, where the kernels before it in the call let it come (pdl_launch_dependents)
// after their own wait, or are let come so themselves: nothing from before the call runs then.
// What overlaps is the launch itself, which costs as much as a small call does
// (norm of 1 x 4096: 2.5 us a call, 4.1 without; attention of one token over
// 131072 rows: 36.7, 39.0; both as calls one after the other).
// `cluster`: CTAs of a thread-block cluster.
inline cudaError_t launch(const void *fn, dim3 grid, dim3 block, size_t smem, cudaStream_t stream, void *params,
                          int cluster = 1) {
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    void *args[] = {params};
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace sk
