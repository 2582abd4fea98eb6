// Dynamic LDS above the default limit is asked for once per kernel and device.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

namespace muir {

template <auto Kernel> hipError_t allow_lds(int bytes) {
    static std::atomic<uint64_t> done{0};  // one bit a device; setting it twice is harmless
    int device = 0;
    const hipError_t err = hipGetDevice(&device);
    if (err != hipSuccess) return err;
    const uint64_t bit = device < 64 ? uint64_t(1) << device : 0;
    if (done.load(std::memory_order_relaxed) & bit) return hipSuccess;
    const hipError_t set = hipFuncSetAttribute(reinterpret_cast<const void *>(Kernel),
                                               hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (set == hipSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return set;
}

}  // namespace muir
