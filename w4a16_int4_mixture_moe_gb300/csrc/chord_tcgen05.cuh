// Inline PTX of the block-scaled tensor-core kernels: tensor-memory
// allocation, the MXFP4 matrix instruction, scale copies, accumulator loads.
#pragma once

#include <stdint.h>

#include "chord_common.cuh"

namespace chord {
namespace tc5 {

// PAIR: the instructions of a cluster of two CTAs (cta_group::2).  Tensor memory is allocated
// and freed by a warp of each; one thread of the first CTA issues the copies and matrix
// instructions for both.
template <bool PAIR>
__device__ __forceinline__ void alloc(uint32_t* slot, uint32_t ncols) {
    if constexpr (PAIR) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(ncols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(ncols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
}
template <bool PAIR>
__device__ __forceinline__ void dealloc(uint32_t taddr, uint32_t ncols) {
    if constexpr (PAIR)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Arrive on `bar` (ALL: of both CTAs of a pair) once every tcgen05 operation this thread
// issued has completed.
template <bool PAIR, bool ALL>
__device__ __forceinline__ void commit(uint32_t bar) {
    if constexpr (!PAIR)
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
    else if constexpr (!ALL)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
            "h"((uint16_t)3)
            : "memory");
}

// One lane of the (converged) warp.  The issuing warp runs its loop with all
// lanes, so that addresses and descriptors stay warp-uniform, and this lane
// alone issues the tensor-core instructions.
__device__ __forceinline__ bool elect() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// cp.async.bulk into this CTA, and the arrivals that go with it, on shared-memory addresses.
__device__ __forceinline__ void bulk_g2s(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void arrive_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The address in CTA `cta` of the cluster of what is at `addr` in this one.
__device__ __forceinline__ uint32_t at_cta(uint32_t addr, uint32_t cta) {
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(cta));
    return remote;
}
// On the barrier at the same address of CTA `cta`: the tensor-memory loads that this thread has
// waited for, and fenced with fence_before(), are done.  Relaxed: it hands over nothing in memory.
__device__ __forceinline__ void arrive_relaxed_at(uint32_t bar, uint32_t cta) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(at_cta(bar, cta)) : "memory");
}
// A box of a 2-D tensor map from row `row` into this CTA, its bytes counted on the barrier at the
// cluster address `bar`: this CTA's or, as these copies may in a pair, the other one's.
__device__ __forceinline__ void box_g2s_pair(uint32_t dst, const void* map, int row, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(dst),
        "l"(map), "r"(0), "r"(row), "r"(bar)
        : "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// Every thread of every CTA of the cluster.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// D[128 x N] (+)= (A x scales)[128 x 64] * (B x scales)[N x 64]^T, E2M1 codes in
// shared memory, one E8M0 scale per 32 columns in tensor memory.  PAIR: D, A and A's scales
// are 256 rows, the first CTA's 128 and the second's; B's first half of rows is in the
// first CTA's shared memory, the other in the second's, and all its scales in both's
// tensor memory.
template <bool PAIR>
__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t sfa,
                                         uint32_t sfb, uint32_t accumulate) {
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
}

// 512 bytes of shared memory (32 rows of 16 bytes) to four tensor-memory
// columns, the 32 lanes repeated in all four lane quarters.  PAIR: each CTA's to its own.
template <bool PAIR>
__device__ __forceinline__ void cp_scales(uint32_t taddr, uint64_t desc) {
    if constexpr (PAIR)
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

__device__ __forceinline__ void ld16(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr)
        : "memory");
}

// K-major operand tile with the 128-byte swizzle: rows of 128 bytes, 8-row
// atoms of 1024 bytes.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)1u << 16 | (uint64_t)(1024u >> 4) << 32 |
           (uint64_t)1u << 46 | (uint64_t)2u << 61;
}
// Scale block: 32 rows of 16 bytes, unswizzled (8-row cores of 128 bytes).
__device__ __forceinline__ uint64_t desc_scales(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(128u >> 4) << 16 | (uint64_t)(128u >> 4) << 32 |
           (uint64_t)1u << 46;
}

// Instruction descriptor: E2M1 x E2M1, E8M0 scales, FP32 accumulator, M = 128 (a pair: 256);
// sf: which two of the four scales of a tensor-memory word the instruction
// takes (0 or 2), for both operands.
template <bool PAIR>
__device__ __forceinline__ uint32_t idesc_mxf4(int n, uint32_t sf) {
    return (sf << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) | (PAIR ? 2u << 27 : 1u << 27) |
           (sf << 29);
}

// CLUSTER: acquire at cluster scope, for phases that the other CTA of a pair, its copies or its
// commits take part in.
template <bool CLUSTER = false>
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    if constexpr (CLUSTER)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
    return ok != 0;
}

// Wait for a phase of the barrier at shared-memory address `bar`, bounded in
// time; gives up at once when another role has set the abort flag.  RELAX: poll
// every couple of hundred nanoseconds only (long waits off the critical path, whose
// polling would take issue slots from the other roles).
template <bool RELAX = false, bool CLUSTER = false>
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* err) {
    if (try_wait<CLUSTER>(bar, parity)) return true;
    const long long t0 = clock64();
    for (uint32_t it = 1;; ++it) {
        if constexpr (RELAX) __nanosleep(200);
        if (try_wait<CLUSTER>(bar, parity)) return true;
        if ((it & 63u) == 0) {
            if (*abort_flag) return false;
            if (clock64() - t0 > kWaitLimitCycles) {
                set_error(err, CHORD_DEV_TIMEOUT);
                *abort_flag = 1;
                return false;
            }
        }
    }
}
template <bool RELAX = false, bool CLUSTER = false>
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* err) {
    return wait<RELAX, CLUSTER>(smem_u32(bar), parity, abort_flag, err);
}

// Slot and parity of a ring of n stages.
struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int n) {
        if (++slot == n) {
            slot = 0;
            phase ^= 1u;
        }
    }
};

}  // namespace tc5
}  // namespace chord
