// Argument and device checks shared by the C entry points.
#pragma once

#include <atomic>
#include <cstring>
#include <initializer_list>
#include <utility>

#include "kv_layout.h"
#include "qmm.h"

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

// Rows of f32, f16 or bf16 (qmm_dtype).
constexpr int64_t kMaxTokens = (int64_t(1) << 24) - 1;   // a workgroup of 256 each: a grid holds 2^32 threads

inline bool dtype_ok(int dt) { return dt == QMM_F32 || dt == QMM_F16 || dt == QMM_BF16; }

inline bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Rows of T tokens and H heads of D values: what the strides may be.
inline qmm_status check_rows(const void *p, int dt, int64_t T, int64_t H, int64_t D, int64_t token, int64_t head) {
    if (token < 0 || head < 0 || token > kMaxBytes || head > kMaxBytes) return QMM_E_SHAPE;
    const __int128 last = (__int128)(T - 1) * token + (__int128)(H - 1) * head + D;
    if (last > kMaxBytes / row_type_bytes(dt)) return QMM_E_SHAPE;
    if (p == nullptr) return QMM_E_NULL;
    if (token % 4 != 0 || head % 4 != 0 || !aligned(p, 4 * row_type_bytes(dt))) return QMM_E_ALIGN;
    return QMM_OK;
}

// Rows that are written, of which no two may share an element: their offsets
// t * token + h * head lie D and more apart.
inline bool rows_apart(int64_t T, int64_t H, int64_t D, int64_t token, int64_t head) {
    if ((T > 1 && token < D) || (H > 1 && head < D)) return false;
    if (T == 1 || H == 1 || (H - 1) * head + D <= token || (T - 1) * token + D <= head) return true;
    if (T < H) std::swap(T, H), std::swap(token, head);
    for (int64_t h = 1; h < H; ++h) {                 // neither is inside a step of the other: the row before h steps, and after
        const int64_t t = h * head / token, before = h * head - t * token;
        if ((t < T && before < D) || (t + 1 < T && token - before < D)) return false;
    }
    return true;
}

inline qmm_status check_out(const void *p, int dt, int64_t T, int64_t H, int64_t D, int64_t token, int64_t head) {
    const qmm_status s = check_rows(p, dt, T, H, D, token, head);
    return s != QMM_OK ? s : rows_apart(T, H, D, token, head) ? QMM_OK : QMM_E_SHAPE;
}

inline qmm_status check_index(const void *p, uintptr_t size) {
    if (p == nullptr) return QMM_E_NULL;
    return aligned(p, size) ? QMM_OK : QMM_E_ALIGN;
}

#define QMM_TRY(expr)                          \
    do {                                       \
        const qmm_status s_ = (expr);          \
        if (s_ != QMM_OK) return s_;           \
    } while (0)

}  // namespace qmm
