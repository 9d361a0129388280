// Rows quantized to Q8_0 or Q8_K by the kernel that computes them.
#pragma once

#include "kv_layout.h"

namespace qmm {

enum ActFmt { A_Q8_0 = 0, A_Q8_K = 1 };

constexpr int act_values(int fmt) { return fmt == A_Q8_0 ? 32 : 256; }
constexpr int act_bytes(int fmt) { return fmt == A_Q8_0 ? kQ80Bytes : kQ8KBytes; }

// Quantizes and stores values V c .. V c + V - 1 of a row whose blocks start at xq;
// lanes hold consecutive c, and the lanes of a block (32 / V or 256 / V of them) call
// it together.  The codes are those of the quantizer entry points (the same f32
// steps, and a maximum is exact in any order); only, a block with a NaN gets a NaN
// as its scale (the maximum passes over it), so that it shows in every product.
template <int FMT, int V>
__device__ __forceinline__ void store_quantized(uint8_t *xq, int c, const float (&v)[V]) {
    static_assert(V == 4 || V == 8, "");
    const int lane = threadIdx.x & 63;
    bool unordered = false;
    float a = 0.0f;
#pragma unroll
    for (int k = 0; k < V; k += 2) {
        unordered |= __builtin_isunordered(v[k], v[k + 1]);
        a = fmaxf(a, fmaxf(fabsf(v[k]), fabsf(v[k + 1])));
    }
    uint64_t nan = __ballot(unordered);
    if constexpr (FMT == A_Q8_0) {
        constexpr int LANES = 32 / V;
        a = fmaxf(a, dpp_f32<kDppQuadXor1>(a));
        a = fmaxf(a, dpp_f32<kDppQuadXor2>(a));
        if constexpr (LANES == 8) a = fmaxf(a, dpp_f32<kDppHalfRowMirror>(a));
        nan = (nan >> (lane & ~(LANES - 1))) & ((1u << LANES) - 1);
    } else {
        a = max16_lanes(a);
        const int b = __builtin_bit_cast(int, a);
        const float r0 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 0));
        const float r1 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 16));
        const float r2 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 32));
        const float r3 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 48));
        if constexpr (V == 4) {
            a = fmaxf(fmaxf(r0, r1), fmaxf(r2, r3));
        } else {
            a = lane < 32 ? fmaxf(r0, r1) : fmaxf(r2, r3);
            nan = lane < 32 ? nan & 0xffffffffu : nan >> 32;
        }
    }
    const float d = nan ? __builtin_nanf("") : a / 127.0f;
    const float id = (a != 0.0f) ? 127.0f / a : 0.0f;
    uint32_t codes[V / 4] = {};
    int sum = 0;
#pragma unroll
    for (int k = 0; k < V; ++k) {
        float r = rintf(v[k] * id);
        if constexpr (FMT == A_Q8_K) r = fminf(fmaxf(r, -128.0f), 127.0f);
        const int q = (int)r;
        sum += q;
        codes[k / 4] |= (uint32_t)(q & 0xff) << (8 * (k & 3));
    }
    if constexpr (FMT == A_Q8_0) {
        // blocks lie at any even byte
        struct __attribute__((packed, aligned(2))) Codes { uint32_t w[V / 4]; } out;
#pragma unroll
        for (int k = 0; k < V / 4; ++k) out.w[k] = codes[k];
        uint8_t *blk = xq + (int64_t)(c / (32 / V)) * kQ80Bytes;
        const int part = c % (32 / V);
        *reinterpret_cast<Codes *>(blk + 2 + V * part) = out;
        if (part == 0) *reinterpret_cast<uint16_t *>(blk) = (uint16_t)f32_to_f16_bits(d);
    } else {
        struct __attribute__((packed, aligned(4))) Codes { uint32_t w[V / 4]; } out;
#pragma unroll
        for (int k = 0; k < V / 4; ++k) out.w[k] = codes[k];
        uint8_t *blk = xq + (int64_t)(c / (256 / V)) * kQ8KBytes;
        const int part = c % (256 / V), lanes = 16 / V;    // of a group of 16
        *reinterpret_cast<Codes *>(blk + 4 + V * part) = out;
        sum += __builtin_amdgcn_update_dpp(0, sum, kDppQuadXor1, 0xF, 0xF, false);
        if constexpr (V == 4) sum += __builtin_amdgcn_update_dpp(0, sum, kDppQuadXor2, 0xF, 0xF, false);
        if (part % lanes == 0) *reinterpret_cast<int16_t *>(blk + 260 + 2 * (part / lanes)) = (int16_t)sum;
        if (part == 0) *reinterpret_cast<float *>(blk) = d;
    }
}

}  // namespace qmm
