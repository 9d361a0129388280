// Rows in f32 / f16 / bf16, the rotation of a row's values, and the byte
// layout of the paged key-value cache (include/qmm.h states the layout).
#pragma once

#include "qmm_device.h"

namespace qmm {

// Row types (qmm_dtype) and cache formats.
enum RowType { R_F32 = 0, R_F16 = 1, R_BF16 = 2 };
enum KvFmt { KV_F16 = 0, KV_Q8_0 = 1, KV_Q4_0 = 2 };

constexpr int kMaxHeadDim = 256;

constexpr int row_type_bytes(int rt) { return rt == R_F32 ? 4 : 2; }

// One rounding, to nearest even; NaN stays a NaN.
__device__ __forceinline__ uint32_t f32_to_bf16_bits(float f) {
    const uint32_t u = __builtin_bit_cast(uint32_t, f);
    if ((u & 0x7fffffffu) > 0x7f800000u) return (u >> 16) | 0x40u;
    return (u + 0x7fffu + ((u >> 16) & 1u)) >> 16;
}

template <int RT>
__device__ __forceinline__ float load1(const void *base, int64_t i) {
    if constexpr (RT == R_F32) return static_cast<const float *>(base)[i];
    const uint32_t h = static_cast<const uint16_t *>(base)[i];
    if constexpr (RT == R_F16) return f16_bits_to_f32(h);
    return __builtin_bit_cast(float, h << 16);
}

// Four consecutive values; i is a multiple of four and the base is aligned to four elements.
template <int RT>
__device__ __forceinline__ float4 load4(const void *base, int64_t i) {
    if constexpr (RT == R_F32) {
        return *reinterpret_cast<const float4 *>(static_cast<const float *>(base) + i);
    } else {
        const uint2 u = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(base) + i);
        if constexpr (RT == R_F16)
            return make_float4(f16_bits_to_f32(u.x), f16_bits_to_f32(u.x >> 16), f16_bits_to_f32(u.y),
                               f16_bits_to_f32(u.y >> 16));
        return make_float4(__builtin_bit_cast(float, u.x << 16), __builtin_bit_cast(float, u.x & 0xffff0000u),
                           __builtin_bit_cast(float, u.y << 16), __builtin_bit_cast(float, u.y & 0xffff0000u));
    }
}

template <int RT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (RT == R_F16) return f32_to_f16_bits(a) | (f32_to_f16_bits(b) << 16);
    return f32_to_bf16_bits(a) | (f32_to_bf16_bits(b) << 16);
}

template <int RT>
__device__ __forceinline__ void store4(void *base, int64_t i, float4 v) {
    if constexpr (RT == R_F32)
        *reinterpret_cast<float4 *>(static_cast<float *>(base) + i) = v;
    else
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(base) + i) =
            make_uint2(pack2<RT>(v.x, v.y), pack2<RT>(v.z, v.w));
}

// ---------------------------------------------------------------------------
// Rotation
// ---------------------------------------------------------------------------

// Cosine and sine of an f64 angle, to about 1e-15: the angle less the nearest
// multiple n of pi/2 (two-part constant, exact products through fma; |n| is
// below 2^33 for any int32 position and frequency of at most pi), then the
// Taylor polynomials on [-pi/4, pi/4], whose first dropped terms are
// (pi/4)^17/17! = 5e-17 and (pi/4)^16/16! = 1e-15.
__device__ __forceinline__ void cos_sin(double a, double &c, double &s) {
    const double n = rint(a * 0.63661977236758134308);
    double r = fma(-n, 1.57079632679489655800e+00, a);
    r = fma(-n, 6.12323399573676603587e-17, r);
    const double z = r * r;
    double p = -1.0 / 1307674368000.0;
    p = fma(p, z, 1.0 / 6227020800.0);
    p = fma(p, z, -1.0 / 39916800.0);
    p = fma(p, z, 1.0 / 362880.0);
    p = fma(p, z, -1.0 / 5040.0);
    p = fma(p, z, 1.0 / 120.0);
    p = fma(p, z, -1.0 / 6.0);
    const double sr = fma(p * z, r, r);
    double q = -1.0 / 87178291200.0;
    q = fma(q, z, 1.0 / 479001600.0);
    q = fma(q, z, -1.0 / 3628800.0);
    q = fma(q, z, 1.0 / 40320.0);
    q = fma(q, z, -1.0 / 720.0);
    q = fma(q, z, 1.0 / 24.0);
    q = fma(q, z, -0.5);
    const double cr = fma(q, z, 1.0);
    const int k = (int)((long long)n & 3);
    const double ss = (k & 1) ? cr : sr, cc = (k & 1) ? sr : cr;
    s = (k & 2) ? -ss : ss;
    c = (k == 1 || k == 2) ? -cc : cc;
}

struct Rope {
    const double *freqs;
    int rot, order, inverse;
    float mscale;
};

// The token's cosines and sines into LDS, one pair a thread; the caller has a
// barrier between this and rotate4.
__device__ __forceinline__ void rope_table(const Rope &r, int32_t pos, float2 *cs, int tid, int threads) {
    for (int i = tid; i < r.rot / 2; i += threads) {
        double c, s;
        cos_sin((double)pos * r.freqs[i], c, s);
        cs[i] = make_float2((float)(c * (double)r.mscale), (float)(s * (double)r.mscale));
        if (r.inverse) cs[i].y = -cs[i].y;
    }
}

// Values a lane takes of a row: 16 bytes.
constexpr int row_values(int rt) { return rt == R_F32 ? 4 : 8; }

// V consecutive values; base and i as for load4.
template <int RT, int V>
__device__ __forceinline__ void load_row(const void *base, int64_t i, float (&x)[V]) {
    static_assert(V == 4 || (V == 8 && RT != R_F32), "");
    if constexpr (V == 4) {
        const float4 v = load4<RT>(base, i);
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {                                              // one load, though only aligned to eight bytes
        struct __attribute__((packed, aligned(8))) Words { uint32_t w[4]; };
        const Words u = *reinterpret_cast<const Words *>(static_cast<const uint16_t *>(base) + i);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            x[2 * k] = RT == R_F16 ? f16_bits_to_f32(u.w[k]) : __builtin_bit_cast(float, u.w[k] << 16);
            x[2 * k + 1] = RT == R_F16 ? f16_bits_to_f32(u.w[k] >> 16)
                                       : __builtin_bit_cast(float, u.w[k] & 0xffff0000u);
        }
    }
}
template <int RT, int V>
__device__ __forceinline__ void store_row(void *base, int64_t i, const float (&x)[V]) {
    if constexpr (V == 4) {
        store4<RT>(base, i, make_float4(x[0], x[1], x[2], x[3]));
    } else {
        struct __attribute__((packed, aligned(8))) Words { uint32_t w[4]; } u;
#pragma unroll
        for (int k = 0; k < 4; ++k) u.w[k] = pack2<RT>(x[2 * k], x[2 * k + 1]);
        *reinterpret_cast<Words *>(static_cast<uint16_t *>(base) + i) = u;
    }
}

// Eight values for the cache's reader.
template <int RT>
__device__ __forceinline__ void store8(void *base, int64_t i, const float (&x)[8]) {
    if constexpr (RT == R_F32) {
        store4<RT>(base, i, make_float4(x[0], x[1], x[2], x[3]));
        store4<RT>(base, i + 4, make_float4(x[4], x[5], x[6], x[7]));
    } else {
        store_row<RT, 8>(base, i, x);
    }
}

// Two consecutive values; i is even.
template <int RT>
__device__ __forceinline__ void store2(void *base, int64_t i, const float (&x)[2]) {
    if constexpr (RT == R_F32)
        *reinterpret_cast<float2 *>(static_cast<float *>(base) + i) = make_float2(x[0], x[1]);
    else
        *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(base) + i) = pack2<RT>(x[0], x[1]);
}

// Values n .. n+V-1 of the rotated row that starts at element `row` of `base`.
// The pair's other value is read from memory again: the row is in the cache.
template <int RT, int V>
__device__ __forceinline__ void rotate(const void *base, int64_t row, int n, const Rope &r, const float2 *cs,
                                       float (&y)[V]) {
    load_row<RT, V>(base, row + n, y);
    if (n >= r.rot) return;
    const int half = r.rot >> 1;
    if (r.order) {                                        // interleaved: both values of a pair are here
#pragma unroll
        for (int k = 0; k < V; k += 2) {
            const bool in = n + k < r.rot;
            const float2 t = cs[in ? (n + k) >> 1 : 0];
            const float u = y[k], v = y[k + 1];
            y[k] = in ? u * t.x - v * t.y : u;
            y[k + 1] = in ? u * t.y + v * t.x : v;
        }
    } else if (half % V == 0) {                           // the V partners are aligned together
        const bool first = n < half;
        const int pair = first ? n : n - half;
        float p[V];
        load_row<RT, V>(base, row + (first ? n + half : pair), p);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const float2 t = cs[pair + k];
            y[k] = first ? y[k] * t.x - p[k] * t.y : p[k] * t.y + y[k] * t.x;
        }
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int i = n + k;
            if (i < r.rot) {
                const bool first = i < half;
                const int pair = first ? i : i - half;
                const float2 t = cs[pair];
                const float p = load1<RT>(base, row + (first ? i + half : pair));
                y[k] = first ? y[k] * t.x - p * t.y : p * t.y + y[k] * t.x;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Lanes of a wave as (g, r), lane = 16 g + r
// ---------------------------------------------------------------------------
// Maximum / sum over the four lanes n, n + 16, n + 32, n + 48, in all of them.
// A permlane swap exchanges the odd rows of 16 (or the upper 32 lanes) of one
// register with the even rows (the lower 32) of the other: of two copies of x,
// one comes back with the even row's value in both rows and the other with the
// odd row's.  (The results are taken into scalars before the casts: a bit cast
// of a vector's element yields element 0.)
template <bool W32>
__device__ __forceinline__ void swap_rows(float x, float &even, float &odd) {
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    uint32_t a, b;
    if constexpr (W32) {
        const auto s = __builtin_amdgcn_permlane32_swap(u, u, false, false);
        a = s[0], b = s[1];
    } else {
        const auto s = __builtin_amdgcn_permlane16_swap(u, u, false, false);
        a = s[0], b = s[1];
    }
    even = __builtin_bit_cast(float, a);
    odd = __builtin_bit_cast(float, b);
}
__device__ __forceinline__ float max_rows(float x) {
    float a, b;
    swap_rows<false>(x, a, b);
    swap_rows<true>(fmaxf(a, b), a, b);
    return fmaxf(a, b);
}
__device__ __forceinline__ float sum_rows(float x) {
    float a, b;
    swap_rows<false>(x, a, b);
    swap_rows<true>(a + b, a, b);
    return a + b;
}

// Maximum over each row of 16 lanes, in all of them.
__device__ __forceinline__ float max16_lanes(float a) {
    a = max8_lanes(a);
    return fmaxf(a, dpp_f32<kDppRowRor8>(a));
}

template <int BYTES>
struct __attribute__((packed, aligned(BYTES))) Unit {
    uint32_t w[BYTES / 4];
};

// ---------------------------------------------------------------------------
// The cache
// ---------------------------------------------------------------------------
constexpr int kGroup = 16;      // positions of a group of codes

constexpr int kv_bits(int fmt) { return fmt == KV_F16 ? 16 : fmt == KV_Q8_0 ? 8 : 4; }

// Sizes of a format at D = 32 * NB values a row.
template <int F, int NB>
struct Kv {
    static constexpr int D = 32 * NB;
    static constexpr bool kScaled = F != KV_F16;
    static constexpr int L = NB * kv_bits(F);                       // bytes of a lane in a group (8 * NB values)
    static constexpr int U = L % 16 == 0 ? 16 : L % 8 == 0 ? 8 : 4;  // bytes of a unit
    static constexpr int NU = L / U;
    static constexpr int kGroupBytes = 64 * L;
    static constexpr int W = L / 4;                                 // bytes of one position in a value lane

    __host__ __device__ static constexpr int64_t side_bytes(int64_t page) {
        return page / kGroup * kGroupBytes + (kScaled ? page * NB * 2 : 0);
    }
    // Byte of a group that holds byte j of lane (g, r).
    __host__ __device__ static constexpr int at(int g, int r, int j) {
        return ((j / U * 4 + g) * 16 + r) * U + j % U;
    }
    // Byte of a lane that holds its value number v.
    __host__ __device__ static constexpr int byte_of(int v) { return v * kv_bits(F) / 8; }

    // Where unit u of lane g of position t's key lies in a side, where byte w of
    // lane m of its value, and where its scales.
    __host__ __device__ static constexpr int key_unit(int t, int g, int u) {
        return (t >> 4) * kGroupBytes + at(g, t & 15, u * U);
    }
    __host__ __device__ static constexpr int value_byte(int t, int m, int w) {
        return (t >> 4) * kGroupBytes + at((t & 15) >> 2, m, (t & 3) * W + w);
    }
    __host__ __device__ static constexpr int scale_byte(int page, int t) {
        return (page >> 4) * kGroupBytes + t * NB * 2;
    }
    // Bytes of a value's W that lie together in a unit.
    static constexpr int P = W % 16 == 0 ? 16 : W % 8 == 0 ? 8 : W % 4 == 0 ? 4 : W % 2 == 0 ? 2 : 1;
};

constexpr int64_t kv_page_bytes(int fmt, int64_t page, int64_t heads, int64_t dim) {
    return heads * 2 * (page * dim * kv_bits(fmt) / 8 + (fmt == KV_F16 ? 0 : page * dim / 32 * 2));
}

struct KvCache {
    uint8_t *data;
    int64_t n_pages;
    int page_shift;             // log2 of the positions in a page
    int heads;

    __host__ __device__ bool has_page(int64_t p) const { return p >= 0 && p < n_pages; }
    // The sides of head h of a page it has: keys at 2h * side, values at (2h + 1) * side.
    __host__ __device__ uint8_t *page_at(int64_t p, int64_t side) const { return data + p * heads * 2 * side; }
};

// Strides of rows, in elements.
struct Strides {
    int64_t token, head;
};

struct WriteArgs {
    Rope r;                     // rot = 0: nothing is rotated
    KvCache c;
    const void *q, *k, *v;
    void *qo;
    const int32_t *positions;
    const int64_t *slots;
    int64_t T;
    int Hq;                     // 0: no queries
    Strides qs, qos, ks, vs;
};

struct ReadArgs {
    KvCache c;
    const int64_t *slots;
    void *k, *v;                // NULL: not wanted
    int64_t T;
    Strides ks, vs;
};

struct AttnArgs {
    KvCache c;
    const void *q;
    void *out;
    const int32_t *pages, *lens;
    int64_t pages_stride;
    const float *mask;          // NULL: none
    int64_t mask_stride;
    float *lse;                 // NULL: not wanted
    float *part;                // [B * Hq][splits][D] partial sums
    float2 *part_ml;            // [B * Hq][splits] their reference and sum of weights
    int Hq, max_len, window, splits, chunk;
    float scale, softcap;
    Strides qs, os;
};

// Calls fn<format, D / 32>(arguments) for a checked format and D.
#define QMM_KV_DISPATCH(fn, ...)                                     \
    switch (fmt * 16 + nb) {                                         \
        case KV_F16 * 16 + 2: return fn<KV_F16, 2>(__VA_ARGS__);     \
        case KV_F16 * 16 + 3: return fn<KV_F16, 3>(__VA_ARGS__);     \
        case KV_F16 * 16 + 4: return fn<KV_F16, 4>(__VA_ARGS__);     \
        case KV_F16 * 16 + 6: return fn<KV_F16, 6>(__VA_ARGS__);     \
        case KV_F16 * 16 + 8: return fn<KV_F16, 8>(__VA_ARGS__);     \
        case KV_Q8_0 * 16 + 2: return fn<KV_Q8_0, 2>(__VA_ARGS__);   \
        case KV_Q8_0 * 16 + 3: return fn<KV_Q8_0, 3>(__VA_ARGS__);   \
        case KV_Q8_0 * 16 + 4: return fn<KV_Q8_0, 4>(__VA_ARGS__);   \
        case KV_Q8_0 * 16 + 6: return fn<KV_Q8_0, 6>(__VA_ARGS__);   \
        case KV_Q8_0 * 16 + 8: return fn<KV_Q8_0, 8>(__VA_ARGS__);   \
        case KV_Q4_0 * 16 + 2: return fn<KV_Q4_0, 2>(__VA_ARGS__);   \
        case KV_Q4_0 * 16 + 3: return fn<KV_Q4_0, 3>(__VA_ARGS__);   \
        case KV_Q4_0 * 16 + 4: return fn<KV_Q4_0, 4>(__VA_ARGS__);   \
        case KV_Q4_0 * 16 + 6: return fn<KV_Q4_0, 6>(__VA_ARGS__);   \
        case KV_Q4_0 * 16 + 8: return fn<KV_Q4_0, 8>(__VA_ARGS__);   \
    }                                                                \
    return hipErrorInvalidValue

}  // namespace qmm
