// Host helpers shared by the files that implement entry points of include/w4a16.h.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>
#include <stdint.h>

#include "w4a16.h"

namespace w4a16 {

constexpr int64_t kMaxDim = (int64_t{1} << 31) - 1;
// Largest K: keeps every per-lane buffer offset of the kernels (at most 256 K bytes past a
// wave's base) inside 32 bits.
constexpr int64_t kMaxK = int64_t{1} << 20;

inline std::atomic<int> g_cu_cache[64];

inline int query_num_cus(int32_t* out) {
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return W4A16_ERR_DEVICE;
    if (dev >= 0 && dev < 64) {
        const int cached = g_cu_cache[dev].load(std::memory_order_relaxed);
        if (cached > 0) {
            *out = cached;
            return W4A16_OK;
        }
    }
    int cus = 0;
    if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0)
        return W4A16_ERR_DEVICE;
    if (dev >= 0 && dev < 64) g_cu_cache[dev].store(cus, std::memory_order_relaxed);
    *out = cus;
    return W4A16_OK;
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Byte ranges [p, p + n) of two buffers share at least one byte.
inline bool overlaps(const void* a, uint64_t na, const void* b, uint64_t nb) {
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
    return na > 0 && nb > 0 && pa < pb + nb && pb < pa + na;
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline int to_status(hipError_t e) { return e == hipSuccess ? W4A16_OK : W4A16_ERR_LAUNCH; }

}  // namespace w4a16
