// The paged key-value cache: rows quantized as they are written (with the
// rotation of queries and keys in the same launch), and read back.
//
// Reading, a workgroup takes 16 tokens; a wave takes the rows of one head of all 16, in
// the lanes of the cache's byte order: for keys (and queries) lane (g, r) holds
// of token r the values 32b + 8g + i, for values lane (g, m) holds of tokens
// 4g + i the values 32b + 2m + e.  So 16 tokens of one aligned group, which is
// what a prompt writes and reads, move as whole lines of the cache and as 64-byte
// pieces of the rows; tokens with slots anywhere take the same path, each lane
// with its own address.
//
// Bit-exactness: as in quantize.hip, every step of a quantizer is one correctly
// rounded f32 operation, so a row's codes and scales are those of the weight
// quantizers of the same format.
#include "kv_layout.h"

namespace qmm {

int row_parts(int64_t T, int64_t rows, int rows_per_workgroup);

constexpr int kRowThreads = 256, kRowWaves = 4, kTokens = 16;

// BYTES bytes at p (aligned to them) into words, low bytes first.
template <int BYTES>
__device__ __forceinline__ void load_piece(const uint8_t *p, uint32_t *w) {
    if constexpr (BYTES == 1)
        *w = *p;
    else if constexpr (BYTES == 2)
        *w = *reinterpret_cast<const uint16_t *>(p);
    else {
        const Unit<BYTES> u = *reinterpret_cast<const Unit<BYTES> *>(p);
#pragma unroll
        for (int i = 0; i < BYTES / 4; ++i) w[i] = u.w[i];
    }
}

// A row's NB scales.
template <int NB>
__device__ __forceinline__ void load_row_scales(const uint8_t *p, float (&d)[NB]) {
#pragma unroll
    for (int b = 0; b < NB; ++b) d[b] = f16_bits_to_f32(reinterpret_cast<const uint16_t *>(p)[b]);
}

// ---------------------------------------------------------------------------
// Writing
// ---------------------------------------------------------------------------
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
    const int b = quad >> 3, part = quad & 7, e = K::byte_of(b * 8 + (part & 1) * 4), w = K::byte_of(2 * b);
    uint8_t *const kp = side + K::key_unit(t, part >> 1, e / K::U) + e % K::U;
    uint8_t *const v0 = side + K::value_byte(t, 2 * part, w), *const v1 = side + K::value_byte(t, 2 * part + 1, w);
    if constexpr (F == KV_F16) {
        const uint32_t lo = pack2<R_F16>(v.x, v.y), hi = pack2<R_F16>(v.z, v.w);
        if (values) {
            *reinterpret_cast<uint32_t *>(v0) = lo;
            *reinterpret_cast<uint32_t *>(v1) = hi;
        } else {
            *reinterpret_cast<uint2 *>(kp) = make_uint2(lo, hi);
        }
    } else {
        float d;
        const uint32_t c = quad_codes<F>(v, part, d);
        if constexpr (F == KV_Q8_0) {
            if (values) {
                *reinterpret_cast<uint16_t *>(v0) = (uint16_t)c;
                *reinterpret_cast<uint16_t *>(v1) = (uint16_t)(c >> 16);
            } else {
                *reinterpret_cast<uint32_t *>(kp) = c;
            }
        } else {
            const uint32_t two = c | (c >> 4);            // bytes 0 and 2: the pairs' nibbles
            if (values) {
                *v0 = (uint8_t)two;
                *v1 = (uint8_t)(two >> 16);
            } else {
                *reinterpret_cast<uint16_t *>(kp) =
                    (uint16_t)((two & 0xffu) | ((two >> 8) & 0xff00u));
            }
        }
        if (part == 0) {
            *reinterpret_cast<uint16_t *>(side + K::scale_byte(page, t) + 2 * b) = (uint16_t)f32_to_f16_bits(d);
        }
    }
}

// The token of workgroup i of T.  Workgroups go to the eight XCDs in turn, each
// with an L2 of its own; 16 consecutive tokens, which share lines of a group's
// codes when they are written in order, are given to one of them.
__device__ __forceinline__ int64_t token_of(int64_t i, int64_t T) {
    constexpr int64_t n = 8 * kTokens;
    if (i >= T / n * n) return i;
    const int64_t j = i % n;
    return i - j + (j % 8) * kTokens + j / 8;
}

// One workgroup a token (and part of its rows): query rows, then key rows, then
// value rows, each by D/4 lanes of one wave.
template <int F, int NB, int RT>
__global__ __launch_bounds__(kRowThreads) void k_kv_write(WriteArgs a) {
    constexpr int kQuads = 8 * NB, kPer = 64 / kQuads;
    __shared__ float2 cs[kMaxHeadDim / 2];
    const int64_t t = token_of(blockIdx.x, a.T);
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

// ---------------------------------------------------------------------------
// Reading
// ---------------------------------------------------------------------------
// Value number k of a lane's words, before its scale.
template <int F>
__device__ __forceinline__ float code_value(const uint32_t *w, int k) {
    if constexpr (F == KV_F16) return f16_bits_to_f32(w[k >> 1] >> (16 * (k & 1)));
    if constexpr (F == KV_Q8_0) return (float)((int)((w[k >> 2] >> (8 * (k & 3))) & 255u) - 128);
    return (float)((int)((w[k >> 3] >> (4 * (k & 7))) & 15u) - 8);
}

template <int F, int NB, int RT>
__global__ __launch_bounds__(kRowThreads) void k_kv_read(ReadArgs a) {
    using K = Kv<F, NB>;
    const int64_t t0 = (int64_t)blockIdx.x * kTokens;
    const int count = (int)min((int64_t)kTokens, a.T - t0);
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int g = lane >> 4, r = lane & 15, page = 1 << a.c.page_shift;
    const int64_t side = K::side_bytes(page);
    const int H = a.c.heads, first = a.k ? 0 : H, rows = a.v ? 2 * H : H;
    const float nan = __builtin_bit_cast(float, 0x7fc00000u);
    for (int row = first + blockIdx.y * kRowWaves + wave; row < rows; row += gridDim.y * kRowWaves) {
        if (row < H) {
            if (r >= count) continue;
            const int64_t slot = a.slots[t0 + r], pg = slot >> a.c.page_shift;
            const int at = (int)(slot & (page - 1));
            const bool good = a.c.has_page(pg);
            uint32_t w[K::L / 4];
            float d[NB];
            const uint8_t *base = a.c.page_at(good ? pg : 0, side) + 2 * row * side;
#pragma unroll
            for (int u = 0; u < K::NU; ++u) load_piece<K::U>(base + K::key_unit(at, g, u), w + u * (K::U / 4));
            if constexpr (K::kScaled) load_row_scales<NB>(base + K::scale_byte(page, at), d);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[i] = code_value<F>(w, 8 * b + i);
                    if constexpr (K::kScaled) x[i] *= d[b];
                    if (!good) x[i] = nan;
                }
                store8<RT>(a.k, (t0 + r) * a.ks.token + row * a.ks.head + 32 * b + 8 * g, x);
            }
        } else {
            const int h = row - H;
            uint32_t w[4][(K::W + 3) / 4] = {};
            float d[4][NB];
            bool good[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t slot = a.slots[t0 + min(4 * g + i, count - 1)], pg = slot >> a.c.page_shift;
                const int at = (int)(slot & (page - 1));
                good[i] = a.c.has_page(pg);
                const uint8_t *base = a.c.page_at(good[i] ? pg : 0, side) + (2 * h + 1) * side;
#pragma unroll
                for (int k = 0; k < K::W; k += K::P) {
                    uint32_t one[K::P < 4 ? 1 : K::P / 4];
                    load_piece<K::P>(base + K::value_byte(at, r, k), one);
                    if constexpr (K::P < 4)
                        w[i][k >> 2] |= one[0] << (8 * (k & 3));
                    else
#pragma unroll
                        for (int j = 0; j < K::P / 4; ++j) w[i][(k >> 2) + j] = one[j];
                }
                if constexpr (K::kScaled) load_row_scales<NB>(base + K::scale_byte(page, at), d[i]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (4 * g + i >= count) continue;
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    float x[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        x[e] = code_value<F>(w[i], 2 * b + e);
                        if constexpr (K::kScaled) x[e] *= d[i][b];
                        if (!good[i]) x[e] = nan;
                    }
                    store2<RT>(a.v, (t0 + 4 * g + i) * a.vs.token + h * a.vs.head + 32 * b + 2 * r, x);
                }
            }
        }
    }
}

template <int F, int NB>
static hipError_t launch_write_f(int rt, WriteArgs a, hipStream_t st) {
    const dim3 grid((unsigned)a.T, (unsigned)row_parts(a.T, a.Hq + 2 * a.c.heads, kRowWaves * (64 / (8 * NB))));
    void *args[] = {(void *)&a};
    const void *k = rt == R_F32   ? (const void *)k_kv_write<F, NB, R_F32>
                    : rt == R_F16 ? (const void *)k_kv_write<F, NB, R_F16>
                                  : (const void *)k_kv_write<F, NB, R_BF16>;
    return hipLaunchKernel(k, grid, dim3(kRowThreads), args, 0, st);
}

template <int F, int NB>
static hipError_t launch_read_f(int rt, ReadArgs a, hipStream_t st) {
    const int64_t groups = (a.T + kTokens - 1) / kTokens;
    const int rows = a.c.heads * ((a.k != nullptr) + (a.v != nullptr));
    const dim3 grid((unsigned)groups, (unsigned)row_parts(groups, rows, kRowWaves));
    void *args[] = {(void *)&a};
    const void *k = rt == R_F32   ? (const void *)k_kv_read<F, NB, R_F32>
                    : rt == R_F16 ? (const void *)k_kv_read<F, NB, R_F16>
                                  : (const void *)k_kv_read<F, NB, R_BF16>;
    return hipLaunchKernel(k, grid, dim3(kRowThreads), args, 0, st);
}

hipError_t launch_kv_write(int fmt, int nb, int rt, WriteArgs a, hipStream_t st) {
    QMM_KV_DISPATCH(launch_write_f, rt, a, st);
}

hipError_t launch_kv_read(int fmt, int nb, int rt, ReadArgs a, hipStream_t st) {
    QMM_KV_DISPATCH(launch_read_f, rt, a, st);
}

}  // namespace qmm
