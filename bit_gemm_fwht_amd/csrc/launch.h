// What launchers share: facts about a device that are looked up once.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

namespace bgf {

// Raises KERNEL's dynamic LDS limit to `lds` bytes once per device (the attribute belongs to the
// function on the current device), instead of on every launch.
template <auto KERNEL>
static hipError_t allow_lds(size_t lds) {
    static std::atomic<uint64_t> done{0};  // bit d: set on device d
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    if (dev < 64 && ((done.load(std::memory_order_acquire) >> dev) & 1u)) return hipSuccess;
    e = hipFuncSetAttribute((const void*)KERNEL, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e == hipSuccess && dev < 64) done.fetch_or(uint64_t(1) << dev, std::memory_order_acq_rel);
    return e;
}

// Compute units of the current device (looked up once per device).
inline hipError_t cu_count(int* n) {
    static std::atomic<int> cus[64];
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    if (dev < 64 && (*n = cus[dev].load(std::memory_order_acquire)) > 0) return hipSuccess;
    e = hipDeviceGetAttribute(n, hipDeviceAttributeMultiprocessorCount, dev);
    if (e == hipSuccess && dev < 64) cus[dev].store(*n, std::memory_order_release);
    return e;
}

}  // namespace bgf
