// Argument and device checks shared by the C entry points.
#pragma once

#include <atomic>
#include <cstring>
#include <initializer_list>

#include "qmm.h"
#include "qmm_device.h"

namespace qmm {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxBytes = int64_t(1) << 40;
constexpr int kMaxDevices = 64;

inline std::atomic<int> g_device_state[kMaxDevices];   // 0 unknown, 1 gfx950, 2 other

inline qmm_status check_device() {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return QMM_E_DEVICE;
    int s = g_device_state[dev].load(std::memory_order_acquire);
    if (s == 0) {
        hipDeviceProp_t p;
        if (hipGetDeviceProperties(&p, dev) != hipSuccess) return QMM_E_DEVICE;
        s = (std::strncmp(p.gcnArchName, "gfx950", 6) == 0) ? 1 : 2;
        g_device_state[dev].store(s, std::memory_order_release);
    }
    return s == 1 ? QMM_OK : QMM_E_DEVICE;
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline qmm_status check_ptrs(std::initializer_list<const void *> ps) {
    for (const void *p : ps)
        if (p == nullptr) return QMM_E_NULL;
    for (const void *p : ps)
        if (!aligned16(p)) return QMM_E_ALIGN;
    return QMM_OK;
}

inline qmm_status launched(hipError_t e) { return e == hipSuccess ? QMM_OK : QMM_E_LAUNCH; }

}  // namespace qmm
