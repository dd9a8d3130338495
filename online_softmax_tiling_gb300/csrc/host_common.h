// host_common.h - what the host sides of the paged, rotary and latent operators share:
// tensor-map encoding, kernel attributes, launches, checks of sizes and strides.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>
#include <set>
#include <utility>

namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

[[maybe_unused]] EncodeTiledFn encode_fn() {
    static std::once_flag once;
    static EncodeTiledFn fn = nullptr;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

[[maybe_unused]] bool misaligned(const void* ptr, uintptr_t al) { return (reinterpret_cast<uintptr_t>(ptr) & (al - 1)) != 0; }

// Opt a kernel into its dynamic shared memory (and clusters of 16) once per device.
[[maybe_unused]] bool ensure_smem(const void* fn, int smem, int device) {
    static std::mutex mu;
    static std::set<std::pair<const void*, int>> done;
    std::lock_guard<std::mutex> lock(mu);
    if (done.count({fn, device})) return true;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
        cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
        return false;
    done.insert({fn, device});
    return true;
}

// Launch as a programmatic dependent of the kernel before it in the stream,
// in clusters of `cluster` CTAs.
[[maybe_unused]] bool launch(const void* fn, int64_t ctas, int grid_y, int threads, int smem, int cluster, void* stream, void** args) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(grid_y));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelExC(&cfg, fn, args) == cudaSuccess;
}

[[maybe_unused]] int sm_count() {
    int device = 0, sms = 152;
    if (cudaGetDevice(&device) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess)
        sms = 152;
    return sms;
}

// Keys of a request (and tokens of an append) that the kernels' 32-bit positions hold with room to spare.
constexpr int kMostKeys = 1 << 30;

[[maybe_unused]] int shift_of(int page_size) {
    switch (page_size) {
        case 16: return 4;
        case 32: return 5;
        case 64: return 6;
        case 128: return 7;
        default: return -1;
    }
}

// {token, head} strides of a 16-bit tensor: positive multiples of 16 bytes.
[[maybe_unused]] bool bad_strides(const long long* s) {
    for (int i = 0; i < 2; ++i)
        if (s[i] <= 0 || s[i] % 8 != 0 || s[i] >= (1ll << 39)) return true;
    return false;
}

}  // namespace
