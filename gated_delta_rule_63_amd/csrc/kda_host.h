// kda_host.h -- host-side helpers of the C entry points beside the forward's.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/kda.h"

namespace kda {

template <typename... P>
inline bool aligned16(const P*... p) {
    return (... && ((reinterpret_cast<uintptr_t>(p) & 15u) == 0));
}

inline kda_status_t status(hipError_t e) { return e == hipSuccess ? KDA_OK : KDA_ERR_HIP; }

// Compute units of the current device, read once per device.
inline int compute_units() {
    static std::atomic<int> cache[64];
    int dev = 0, n = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) return 256;
    if (dev < 64 && (n = cache[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0) n = 256;
    if (dev < 64) cache[dev].store(n, std::memory_order_relaxed);
    return n;
}

}  // namespace kda
