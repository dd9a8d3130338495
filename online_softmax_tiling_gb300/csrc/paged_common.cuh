// paged_common.cuh - what the kernels around the paged 8-bit key/value cache
// share: the device status word, bounded waits, power-of-two scales and e4m3
// conversions.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "sm103_ptx.cuh"

namespace fa {
namespace paged {

// Status of the paged kernels on this device (FA_OK, FA_ERR_INVALID_ARG for
// bad device data, FA_ERR_TIMEOUT); read and cleared by fa_check_device_status.
__device__ unsigned int g_paged_status;

constexpr unsigned int kBadData = 1;  // FA_ERR_INVALID_ARG
constexpr unsigned int kTimeout = 5;  // FA_ERR_TIMEOUT
constexpr unsigned long long kTimeoutNs = 2000000000ull;

__device__ __forceinline__ void report(unsigned int code) { atomicCAS(&g_paged_status, 0u, code); }

// Bounded wait of one thread on an mbarrier phase (it sleeps in the barrier
// unit).  False after two seconds, with the device status set.
__device__ __forceinline__ bool wait_long(uint32_t bar, uint32_t parity) {
    const uint64_t t0 = ptx::globaltimer();
    for (;;) {
        if (ptx::mbar_try_wait_sleep(bar, parity, 200000)) return true;
        if (ptx::globaltimer() - t0 > kTimeoutNs) {
            report(kTimeout);
            return false;
        }
    }
}
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    return wait_long(bar, parity);
}
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait(bar, parity));
}

// Every kernel here is a programmatic dependent launch: it may be set up while
// the kernel before it in the stream still runs, and reads or writes
// global memory only behind wait_for_previous (that kernel's end, its writes visible).
// So nothing is read on the read-only path, whose data must stand still from the
// launch on (and whose loads may be moved ahead of the wait): ld() is a plain load.
// Lengths, tables and slots go past L1 altogether (ld_meta): the kernel that reads them is
// often the next behind the one that wrote them, from several SMs, line by line.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void dependents_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
template <typename T>
__device__ __forceinline__ T ld(const T* p) { return *p; }
__device__ __forceinline__ int ld_meta(const int* p) { return __ldcg(p); }

// Largest b in [0, n) with prefix[b] <= i (prefix ascending, prefix[0] = 0 <= i).
__device__ __forceinline__ int owner_of(const int* prefix, int n, int i) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] <= i) lo = mid; else hi = mid;
    }
    return lo;
}

// Barrier of a cluster's CTAs; shared memory writes before it are seen behind it.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
}

// Exponent of the smallest power of two s in [2^-60, 2^60] with a <= top s,
// for top = (1 + top_mant / 2^23) 2^top_exp and a finite a >= 0: compares the
// mantissa and subtracts the exponents (a below 2^-126 gives -60).
__device__ __forceinline__ int pow2_exp(float a, uint32_t top_mant, int top_exp) {
    const uint32_t b = __float_as_uint(a);
    const int e = static_cast<int>(b >> 23) - 127 - top_exp + ((b & 0x7FFFFFu) > top_mant ? 1 : 0);
    return a > 0.f ? max(-60, min(60, e)) : -60;
}
// 2^e for -126 <= e <= 127
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// a <= 448 s: 448 = 1.75 * 2^8
__device__ __forceinline__ int cache_scale_exp(float amax) { return pow2_exp(amax, 0x600000u, 8); }
// |q| <= 127 u: 127 = 1.984375 * 2^6
__device__ __forceinline__ int query_unit_exp(float amax) { return pow2_exp(amax, 0x7E0000u, 6); }

// Two fp32 values to e4m3 (nearest even, saturating, NaN kept), `lo` in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
// Two e4m3 codes (low 16 bits) to packed fp16: exact.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t v) {
    uint32_t r;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ float2 half2_floats(uint32_t v) {
    __half2 h;
    *reinterpret_cast<uint32_t*>(&h) = v;
    return __half22float2(h);
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Exact fp32 values of a packed 16-bit pair.
__device__ __forceinline__ float2 unpack16(uint32_t v, bool bf16) {
    if (bf16) return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
    return half2_floats(v);
}
__device__ __forceinline__ uint32_t pack16(float lo, float hi, bool bf16) {
    uint32_t r;
    if (bf16)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Shared-memory matrix descriptor for tcgen05.mma: 128-byte swizzle, start
// address, leading and stride byte offsets in 16-byte units, version 1.
__device__ __forceinline__ uint64_t pr_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(lbo >> 4) << 16) |
           (static_cast<uint64_t>(sbo >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// Instruction descriptor, kind::f16: fp16 operands, fp32 sums.
__host__ __device__ constexpr uint32_t pr_instr(int m, int n, bool b_mn_major) {
    return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((static_cast<uint32_t>(n) >> 3) << 17) |
           ((static_cast<uint32_t>(m) >> 4) << 24);
}

template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int32_t c0, int32_t c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}

}  // namespace paged
}  // namespace fa
