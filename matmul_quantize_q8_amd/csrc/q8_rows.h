// Rows quantized to Q8_0 or Q8_K by the kernel that computes them.
#pragma once

#include "kv_layout.h"

namespace qmm {

enum ActFmt { A_Q8_0 = 0, A_Q8_K = 1 };

constexpr int act_values(int fmt) { return fmt == A_Q8_0 ? 32 : 256; }
constexpr int act_bytes(int fmt) { return fmt == A_Q8_0 ? kQ80Bytes : kQ8KBytes; }

// Quantizes and stores values 4c .. 4c + 3 of a row whose blocks start at xq;
// lanes hold consecutive c, and the lanes of a block (8, or the whole wave) call
// it together.  The codes are those of the quantizer entry points; only, a block
// with a NaN gets a NaN as its scale (their maximum passes over it), so that
// it shows in every product.
template <int FMT>
__device__ __forceinline__ void store_quantized(uint8_t *xq, int c, float4 v) {
    const uint64_t nan = __ballot(__builtin_isunordered(v.x, v.y) || __builtin_isunordered(v.z, v.w));
    const int lane = threadIdx.x & 63;
    float d;
    if constexpr (FMT == A_Q8_0) {
        const uint32_t packed = q8_0_part(v, d);
        if ((nan >> (lane & 56)) & 0xff) d = __builtin_nanf("");
        store_q8_0_part(xq + (int64_t)(c >> 3) * kQ80Bytes, c & 7, packed, d);
    } else {
        int gsum;
        const uint32_t packed = q8_k_wave(v, gsum, d);
        if (nan) d = __builtin_nanf("");
        store_q8_k_lane(xq + (int64_t)(c >> 6) * kQ8KBytes, c & 63, packed, gsum, d);
    }
}

}  // namespace qmm
