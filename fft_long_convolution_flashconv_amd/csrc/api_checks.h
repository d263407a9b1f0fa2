// api_checks.h -- what the C-ABI shims check on the host before any HIP call,
// and the check of the current device.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>
#include <cstring>

#include "../../include/h3conv.h"

namespace h3c {

constexpr int kMaxDevices = 64;
inline std::atomic<int> g_dev_ok[kMaxDevices];  // 0 unknown, 1 usable gfx950, -1 not usable

inline bool valid_io(int io) { return io == H3CONV_F32 || io == H3CONV_F16 || io == H3CONV_BF16; }

// [p, p + n) and [q, q + m) overlap?
inline bool overlap(const void *p, size_t n, const void *q, size_t m) {
    if (!p || !q || n == 0 || m == 0) return false;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return a < b + m && b < a + n;
}

inline h3conv_status device_check() {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return H3CONV_ERR_NO_DEVICE;
    int st = g_dev_ok[dev].load(std::memory_order_acquire);
    if (st == 0) {
        hipDeviceProp_t p;
        if (hipGetDeviceProperties(&p, dev) != hipSuccess) return H3CONV_ERR_NO_DEVICE;
        st = (std::strncmp(p.gcnArchName, "gfx950", 6) == 0) ? 1 : -1;
        g_dev_ok[dev].store(st, std::memory_order_release);
    }
    return st == 1 ? H3CONV_OK : H3CONV_ERR_NO_DEVICE;
}

inline h3conv_status from_hip(hipError_t e) { return e == hipSuccess ? H3CONV_OK : H3CONV_ERR_HIP; }

}  // namespace h3c
