// The paged key-value cache: rows quantized as they are written (with the
// rotation of queries and keys in the same launch), and read back.
//
// Bit-exactness: as in quantize.hip, every step of a quantizer is one correctly
// rounded f32 operation, so a row's codes and scales are those of the weight
// quantizers of the same format.
#include "kv_layout.h"

namespace qmm {

int row_parts(int64_t T, int64_t rows, int rows_per_workgroup);

constexpr int kRowThreads = 256;

// Codes of a block's quad (four of 32 values, eight lanes a block), one a byte
// and offset to be unsigned; d is the block's scale.  All eight lanes call it.
template <int F>
__device__ __forceinline__ uint32_t quad_codes(float4 v, int part, float &d) {
    if constexpr (F == KV_Q8_0) {
        return q8_0_part(v, d) ^ 0x80808080u;
    } else {
        const float vv[4] = {v.x, v.y, v.z, v.w};
        float am = fabsf(vv[0]), mx = vv[0];              // largest magnitude, the first on ties
        int ix = 4 * part;
#pragma unroll
        for (int k = 1; k < 4; ++k) {
            const float a = fabsf(vv[k]);
            if (a > am) { am = a; mx = vv[k]; ix = 4 * part + k; }
        }
#pragma unroll
        for (int m = 1; m < 8; m <<= 1) {
            const float oam = xor_shfl(am, m), omx = xor_shfl(mx, m);
            const int oix = xor_shfl(ix, m);
            if (oam > am || (oam == am && oix < ix)) { am = oam; mx = omx; ix = oix; }
        }
        d = am != 0.0f ? mx / -8.0f : 0.0f;
        uint32_t codes = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            int c = d != 0.0f ? (int)rintf(vv[k] / d) + 8 : 8;
            codes |= (uint32_t)min(max(c, 0), 15) << (8 * k);
        }
        return codes;
    }
}

// Store a quad at `side` (one head's keys or values of one page).
template <int F, int NB>
__device__ __forceinline__ void store_quad(uint8_t *side, int page, int t, int quad, bool values, float4 v) {
    using K = Kv<F, NB>;
    uint8_t *grp = side + (t >> 4) * K::kGroupBytes;
    if constexpr (F == KV_F16) {
        const uint32_t lo = pack2<R_F16>(v.x, v.y), hi = pack2<R_F16>(v.z, v.w);
        if (values) {
            *reinterpret_cast<uint32_t *>(grp + K::value_byte(t, quad, 0)) = lo;
            *reinterpret_cast<uint32_t *>(grp + K::value_byte(t, quad, 1)) = hi;
        } else {
            *reinterpret_cast<uint2 *>(grp + K::key_byte(t, quad)) = make_uint2(lo, hi);
        }
    } else {
        float d;
        const uint32_t c = quad_codes<F>(v, quad & 7, d);
        if constexpr (F == KV_Q8_0) {
            if (values) {
                *reinterpret_cast<uint16_t *>(grp + K::value_byte(t, quad, 0)) = (uint16_t)c;
                *reinterpret_cast<uint16_t *>(grp + K::value_byte(t, quad, 1)) = (uint16_t)(c >> 16);
            } else {
                *reinterpret_cast<uint32_t *>(grp + K::key_byte(t, quad)) = c;
            }
        } else {
            const uint32_t two = c | (c >> 4);            // bytes 0 and 2: the pairs' nibbles
            if (values) {
                grp[K::value_byte(t, quad, 0)] = (uint8_t)two;
                grp[K::value_byte(t, quad, 1)] = (uint8_t)(two >> 16);
            } else {
                *reinterpret_cast<uint16_t *>(grp + K::key_byte(t, quad)) =
                    (uint16_t)((two & 0xffu) | ((two >> 8) & 0xff00u));
            }
        }
        if ((quad & 7) == 0) {
            uint16_t *sc = reinterpret_cast<uint16_t *>(side + (page >> 4) * K::kGroupBytes);
            sc[t * NB + (quad >> 3)] = (uint16_t)f32_to_f16_bits(d);
        }
    }
}

// The values of a quad.
template <int F, int NB>
__device__ __forceinline__ float4 load_quad(const uint8_t *side, int page, int t, int quad, bool values) {
    using K = Kv<F, NB>;
    const uint8_t *grp = side + (t >> 4) * K::kGroupBytes;
    const int k0 = K::key_byte(t, quad), v0 = K::value_byte(t, quad, 0), v1 = K::value_byte(t, quad, 1);
    if constexpr (F == KV_F16) {
        uint32_t lo, hi;
        if (values) {
            lo = *reinterpret_cast<const uint32_t *>(grp + v0);
            hi = *reinterpret_cast<const uint32_t *>(grp + v1);
        } else {
            const uint2 u = *reinterpret_cast<const uint2 *>(grp + k0);
            lo = u.x;
            hi = u.y;
        }
        return make_float4(f16_bits_to_f32(lo), f16_bits_to_f32(lo >> 16), f16_bits_to_f32(hi),
                           f16_bits_to_f32(hi >> 16));
    } else {
        const uint16_t *sc = reinterpret_cast<const uint16_t *>(side + (page >> 4) * K::kGroupBytes);
        const float d = f16_bits_to_f32(sc[t * NB + (quad >> 3)]);
        int c[4];
        if constexpr (F == KV_Q8_0) {
            const uint32_t u = values ? (uint32_t) * reinterpret_cast<const uint16_t *>(grp + v0) |
                                            (uint32_t) * reinterpret_cast<const uint16_t *>(grp + v1) << 16
                                      : *reinterpret_cast<const uint32_t *>(grp + k0);
#pragma unroll
            for (int k = 0; k < 4; ++k) c[k] = (int)((u >> (8 * k)) & 255u) - 128;
        } else {
            const uint32_t u = values ? (uint32_t)grp[v0] | (uint32_t)grp[v1] << 8
                                      : (uint32_t) * reinterpret_cast<const uint16_t *>(grp + k0);
#pragma unroll
            for (int k = 0; k < 4; ++k) c[k] = (int)((u >> (4 * k)) & 15u) - 8;
        }
        return make_float4(d * (float)c[0], d * (float)c[1], d * (float)c[2], d * (float)c[3]);
    }
}

// One workgroup a token (and part of its rows): query rows, then key rows, then
// value rows, each by D/4 lanes of one wave.
template <int F, int NB, int RT>
__global__ __launch_bounds__(kRowThreads) void k_kv_write(WriteArgs a) {
    constexpr int kQuads = 8 * NB, kPer = 64 / kQuads;
    __shared__ float2 cs[kMaxHeadDim / 2];
    const int64_t t = blockIdx.x;
    if (a.r.rot) {
        rope_table(a.r, a.positions[t], cs, threadIdx.x, kRowThreads);
        __syncthreads();
    }
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int sub = lane / kQuads, quad = lane - sub * kQuads;
    if (sub >= kPer) return;
    const int page = 1 << a.c.page_shift;
    const int64_t slot = a.slots[t], pg = slot >> a.c.page_shift;
    const bool keep = a.c.has_page(pg);
    const int at = (int)(slot & (page - 1));
    const int64_t side = Kv<F, NB>::side_bytes(page);
    uint8_t *base = a.c.page_at(keep ? pg : 0, side);
    const int H = a.c.heads, rows = a.Hq + 2 * H, step = gridDim.y * (kRowThreads / 64) * kPer;
    for (int row = (blockIdx.y * (kRowThreads / 64) + wave) * kPer + sub; row < rows; row += step) {
        if (row < a.Hq) {
            const float4 y = rotate4<RT>(a.q, t * a.qs.token + row * a.qs.head, 4 * quad, a.r, cs);
            store4<RT>(a.qo, t * a.qos.token + row * a.qos.head + 4 * quad, y);
        } else {
            const bool values = row >= a.Hq + H;
            const int h = row - a.Hq - (values ? H : 0);
            const float4 y = values ? load4<RT>(a.v, t * a.vs.token + h * a.vs.head + 4 * quad)
                                    : rotate4<RT>(a.k, t * a.ks.token + h * a.ks.head, 4 * quad, a.r, cs);
            if (keep) store_quad<F, NB>(base + (2 * h + values) * side, page, at, quad, values, y);
        }
    }
}

template <int F, int NB, int RT>
__global__ __launch_bounds__(kRowThreads) void k_kv_read(ReadArgs a) {
    constexpr int kQuads = 8 * NB, kPer = 64 / kQuads;
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int sub = lane / kQuads, quad = lane - sub * kQuads;
    if (sub >= kPer) return;
    const int page = 1 << a.c.page_shift;
    const int64_t slot = a.slots[t], pg = slot >> a.c.page_shift;
    const bool good = a.c.has_page(pg);
    const int at = (int)(slot & (page - 1));
    const int64_t side = Kv<F, NB>::side_bytes(page);
    const uint8_t *base = a.c.page_at(good ? pg : 0, side);
    const int H = a.c.heads, first = a.k ? 0 : H, rows = a.v ? 2 * H : H;
    const int step = gridDim.y * (kRowThreads / 64) * kPer;
    for (int row = first + (blockIdx.y * (kRowThreads / 64) + wave) * kPer + sub; row < rows; row += step) {
        const bool values = row >= H;
        const int h = row - (values ? H : 0);
        const float nan = __builtin_bit_cast(float, 0x7fc00000u);
        float4 y = make_float4(nan, nan, nan, nan);
        if (good) y = load_quad<F, NB>(base + (2 * h + values) * side, page, at, quad, values);
        const Strides s = values ? a.vs : a.ks;
        store4<RT>(values ? a.v : a.k, t * s.token + h * s.head + 4 * quad, y);
    }
}

template <int F, int NB>
static hipError_t launch_write_f(int rt, WriteArgs a, int64_t T, hipStream_t st) {
    const dim3 grid((unsigned)T, (unsigned)row_parts(T, a.Hq + 2 * a.c.heads, kRowThreads / 64 * (64 / (8 * NB))));
    void *args[] = {(void *)&a};
    const void *k = rt == R_F32   ? (const void *)k_kv_write<F, NB, R_F32>
                    : rt == R_F16 ? (const void *)k_kv_write<F, NB, R_F16>
                                  : (const void *)k_kv_write<F, NB, R_BF16>;
    return hipLaunchKernel(k, grid, dim3(kRowThreads), args, 0, st);
}

template <int F, int NB>
static hipError_t launch_read_f(int rt, ReadArgs a, int64_t T, hipStream_t st) {
    const int rows = a.c.heads * ((a.k != nullptr) + (a.v != nullptr));
    const dim3 grid((unsigned)T, (unsigned)row_parts(T, rows, kRowThreads / 64 * (64 / (8 * NB))));
    void *args[] = {(void *)&a};
    const void *k = rt == R_F32   ? (const void *)k_kv_read<F, NB, R_F32>
                    : rt == R_F16 ? (const void *)k_kv_read<F, NB, R_F16>
                                  : (const void *)k_kv_read<F, NB, R_BF16>;
    return hipLaunchKernel(k, grid, dim3(kRowThreads), args, 0, st);
}

hipError_t launch_kv_write(int fmt, int nb, int rt, WriteArgs a, int64_t T, hipStream_t st) {
    QMM_KV_DISPATCH(launch_write_f, rt, a, T, st);
}

hipError_t launch_kv_read(int fmt, int nb, int rt, ReadArgs a, int64_t T, hipStream_t st) {
    QMM_KV_DISPATCH(launch_read_f, rt, a, T, st);
}

}  // namespace qmm
