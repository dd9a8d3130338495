// pair_ptx.cuh - what two CTAs on neighbouring SMs (a cluster of two) need to work as one: barriers of either CTA,
// TMA that signals them, tcgen05 with cta_group::2.  The first CTA issues the products; every operand's half in the
// other CTA lies at the same shared address.
#pragma once

#include "paged_common.cuh"

namespace fa {
namespace paged {

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// The shared address `a` in the first CTA of the cluster.
__device__ __forceinline__ uint32_t in_first_cta(uint32_t a) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(a));
    return r;
}
// An arrival in either CTA.  What it orders is tensor memory (behind the tcgen05 fences) and the execution of what waits for
// it; a release to the cluster would first wait for all of the SM's memory traffic, the next tile's loads too (1.3 us).
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The same behind writes to shared memory that the tensor cores of the pair are to read, or reads of what is written there
// next at the other CTA's request.
__device__ __forceinline__ void arrive_remote_release(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void arrive_remote_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// Whether the phase is complete, with what both CTAs did before it visible (does not wait).
__device__ __forceinline__ bool test_cluster(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// A TMA load into this CTA that signals a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t c0, int32_t c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}
// D (tmem of both) (+)= A (smem, 64 rows of each) B (smem, half of the columns of each)^T over four steps of 16 along
// K, 32 bytes of swizzled rows each.  One elected lane of the (converged) warp issues.
__device__ __forceinline__ void mma_pair_k64(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred e, p0, p1;\n\t.reg .b64 x, y;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p0, %4, 0;\n\t"
        "setp.eq.b32 p1, %4, %4;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p0;\n\t"
        "add.s64 x, %1, 2;\n\tadd.s64 y, %2, 2;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], x, y, %3, p1;\n\t"
        "add.s64 x, %1, 4;\n\tadd.s64 y, %2, 4;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], x, y, %3, p1;\n\t"
        "add.s64 x, %1, 6;\n\tadd.s64 y, %2, 6;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], x, y, %3, p1;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// The same over twelve steps: three pieces of 64 channels, A's 16 KB apart, B's 8 KB.
__device__ __forceinline__ void mma_pair_k192(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred e, p0, p1;\n\t.reg .b64 x, y;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p0, %3, %3;\n\t"
        "setp.eq.b32 p1, %3, %3;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p0;\n\t"
#define FA_STEP(A, B) "add.s64 x, %1, " #A ";\n\tadd.s64 y, %2, " #B ";\n\t@e tcgen05.mma.cta_group::2.kind::f16 [%0], x, y, %3, p1;\n\t"
        FA_STEP(2, 2) FA_STEP(4, 4) FA_STEP(6, 6)
        FA_STEP(1024, 512) FA_STEP(1026, 514) FA_STEP(1028, 516) FA_STEP(1030, 518)
        FA_STEP(2048, 1024) FA_STEP(2050, 1026) FA_STEP(2052, 1028) FA_STEP(2054, 1030)
#undef FA_STEP
        "}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc)
        : "memory");
}
// The same with A in tensor memory (16 elements in 8 columns), B's steps 16 rows of 128 bytes.
__device__ __forceinline__ void mma_pair_ts_k64(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred e, p0, p1;\n\t.reg .b32 x;\n\t.reg .b64 y;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p0, %4, 0;\n\t"
        "setp.eq.b32 p1, %4, %4;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p0;\n\t"
        "add.u32 x, %1, 8;\n\tadd.s64 y, %2, 128;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [x], y, %3, p1;\n\t"
        "add.u32 x, %1, 16;\n\tadd.s64 y, %2, 256;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [x], y, %3, p1;\n\t"
        "add.u32 x, %1, 24;\n\tadd.s64 y, %2, 384;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [x], y, %3, p1;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrives on `bar` in both CTAs when what the elected lane issued before is done.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(bar),
        "h"(static_cast<unsigned short>(3))
        : "memory");
}

__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t c0, int32_t c1, int32_t c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
__device__ __forceinline__ void tma_load_4d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t c0, int32_t c1, int32_t c2, int32_t c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

// Bounded wait of a warp on a barrier that both CTAs signal (false after two seconds, with the device status set).
__device__ __forceinline__ bool wait_pair(uint32_t bar, uint32_t parity) {
    bool ok = test_cluster(bar, parity);
    if (!__all_sync(0xffffffffu, ok)) {
        const uint64_t t0 = ptx::globaltimer();
        while (!(ok = test_cluster(bar, parity))) {
            if (ptx::globaltimer() - t0 > kTimeoutNs) {
                report(kTimeout);
                break;
            }
        }
    }
    return __all_sync(0xffffffffu, ok);
}

// The same for the issuer of products, whose every instruction between a barrier and the product behind it is time that the
// tensor cores may stand still: the time is looked at once in 4096 tries.
__device__ __forceinline__ bool wait_pair_lean(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    uint64_t t0 = 0;
    for (;;) {
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t.reg .b32 n;\n\tmov.u32 n, 0;\n\t"
            "AGAIN:\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "@p bra DONE;\n\t"
            "add.u32 n, n, 1;\n\tsetp.lt.u32 q, n, 4096;\n\t"
            "@q bra AGAIN;\n\t"
            "DONE:\n\tselp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (__all_sync(0xffffffffu, ok)) return true;
        const uint64_t now = ptx::globaltimer();
        if (t0 == 0) t0 = now;
        if (__any_sync(0xffffffffu, now - t0 > kTimeoutNs)) {
            report(kTimeout);
            return false;
        }
    }
}

__device__ __forceinline__ void tmem_alloc_pair(uint32_t holder) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(holder), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t tmem) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}
// Arrives on `bar` of this CTA when what the elected lane issued before is done.
__device__ __forceinline__ void commit_pair_here(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
}

}  // namespace paged
}  // namespace fa
