// What the warps of the TMA + tcgen05 kernels share: bounded waits that end together, elected
// lanes, copies, products and tensor-memory accesses as inline PTX.
#pragma once

#include "skinny_tc05.cuh"

namespace sk {
namespace roles {

using tc05::bar_arrive;
using tc05::bar_try;
using tc05::mma_commit;
using tc05::prefetch_tmap;
using tc05::tc_fence_after;
using tc05::tc_fence_before;
using tc05::tmem_ld16;

// Shared memory that a CTA asks for at least where it takes half of the tensor memory or all of it.  It waits until it has
// it.  Beside it on the SM there might be two CTAs of another stream's GEMMs (a ring of two stages of 16 KiB each at least),
// of which one holds some until the other one is done, which waits behind this CTA for its own: there is no room for two.
// (All the shared memory would leave the next kernel's small CTAs none: 3 prompts of 3000, 16 heads of 128 x 64: 55.3 ->
// 56.8 us.)
constexpr size_t kAloneSmem = kMaxSmemOptin - 48 * 1024;

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

// 16 bytes global -> shared, asynchronously; zeros where `bytes` is 0.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// 4 bytes.
__device__ __forceinline__ void copy4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
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

// Columns in the 16 x 256-bit form: lane l of the warp gets rows l / 4 and l / 4 + 8 of the 16 lanes
// of tensor memory, and of each 8 columns the pair 2 (l % 4): r[4i], r[4i+1] of the first row, r[4i+2], r[4i+3] of
// the second.  (They are there after tcgen05.wait::ld.)
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

// 8 columns of this thread's lane (there after tcgen05.wait::ld).
__device__ __forceinline__ void tmem_ld8(uint32_t addr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
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

}  // namespace roles
}  // namespace sk
