// The paged key-value cache: rows quantized as they are written (with the
// rotation of queries and keys in the same launch), and read back.
//
// Writing, a workgroup takes one token and its waves whole rows, 16 bytes a lane:
// 4096 tokens of 32 + 8 + 8 heads of 128 in bf16 (93 MB) take 22 us, 4.2 TB/s of
// the 4.9 of a large copy.  Reading, a workgroup takes 16 tokens; a wave takes the
// rows of one head of all 16, in the lanes of the cache's byte order: for keys lane
// (g, r) holds of token r the values 32b + 8g + i, for values lane (g, m) holds of
// tokens 4g + i the values 32b + 2m + e.  So 16 tokens of one aligned group, which
// is what a prompt reads, move as whole lines of the cache and as 64-byte pieces of
// the rows; tokens with slots anywhere take the same path, each lane with its own
// address.  8192 tokens q8_0 to bf16 (51 MB): 22 us a token a workgroup, 12 us so.
// (Writing in that order took 41 us: a token's table of angles for each of 16
// tokens, and half the waves.)
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
// Codes of V consecutive values of a block, in 32 / V lanes, offset to be
// unsigned, and the block's scale.  All lanes of the block call it.
template <int F, int V>
__device__ __forceinline__ void block_codes(const float (&v)[V], int part, uint32_t (&c)[V], float &d) {
    float a = 0.0f;
#pragma unroll
    for (int k = 0; k < V; ++k) a = fmaxf(a, fabsf(v[k]));
    a = fmaxf(a, dpp_f32<kDppQuadXor1>(a));
    a = fmaxf(a, dpp_f32<kDppQuadXor2>(a));
    if constexpr (V == 4) a = fmaxf(a, dpp_f32<kDppHalfRowMirror>(a));
    if constexpr (F == KV_Q8_0) {
        d = a / 127.0f;
        const float id = a != 0.0f ? 127.0f / a : 0.0f;
#pragma unroll
        for (int k = 0; k < V; ++k) c[k] = (uint32_t)((int)rintf(v[k] * id) + 128) & 255u;
    } else {
        // the sign of the value of largest magnitude, the first on ties: the least
        // 2 * number + sign among the values of that magnitude
        float key = 1000.0f;
#pragma unroll
        for (int k = V - 1; k >= 0; --k)
            if (fabsf(v[k]) == a) key = (float)(2 * (V * part + k) + (v[k] < 0.0f));
        key = fminf(key, dpp_f32<kDppQuadXor1>(key));
        key = fminf(key, dpp_f32<kDppQuadXor2>(key));
        if constexpr (V == 4) key = fminf(key, dpp_f32<kDppHalfRowMirror>(key));
        const float mx = ((int)key & 1) ? -a : a;
        d = a != 0.0f ? mx / -8.0f : 0.0f;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int q = d != 0.0f ? (int)rintf(v[k] / d) + 8 : 8;
            c[k] = (uint32_t)min(max(q, 0), 15);
        }
    }
}

// The low BYTES bytes of w at p, aligned to them.
template <int BYTES>
__device__ __forceinline__ void store_piece(uint8_t *p, const uint32_t *w) {
    if constexpr (BYTES == 1)
        *p = (uint8_t)*w;
    else if constexpr (BYTES == 2)
        *reinterpret_cast<uint16_t *>(p) = (uint16_t)*w;
    else {
        Unit<BYTES> u;
#pragma unroll
        for (int i = 0; i < BYTES / 4; ++i) u.w[i] = w[i];
        *reinterpret_cast<Unit<BYTES> *>(p) = u;
    }
}

// Store values V part .. of a row of position t at `side` (one head's keys or
// values of one page).  A key's V are consecutive in their lane's bytes; a
// value's are two in each of V/2 lanes.
template <int F, int NB, int V>
__device__ __forceinline__ void store_values(uint8_t *side, int page, int t, int lane, bool values,
                                             const float (&v)[V]) {
    using K = Kv<F, NB>;
    constexpr int kBits = kv_bits(F), kBlockLanes = 32 / V;
    const int b = lane / kBlockLanes, part = lane % kBlockLanes, first = V * part;
    uint32_t c[V];
    if constexpr (F == KV_F16) {
#pragma unroll
        for (int k = 0; k < V; ++k) c[k] = f32_to_f16_bits(v[k]);
    } else {
        float d;
        block_codes<F, V>(v, part, c, d);
        if (part == 0)
            *reinterpret_cast<uint16_t *>(side + K::scale_byte(page, t) + 2 * b) = (uint16_t)f32_to_f16_bits(d);
    }
    uint32_t w[(V * kBits + 31) / 32] = {};
#pragma unroll
    for (int k = 0; k < V; ++k) w[k * kBits / 32] |= c[k] << (k * kBits % 32);
    if (values) {
        const int byte = K::byte_of(2 * b);
#pragma unroll
        for (int k = 0; k < V; k += 2) {
            const uint32_t two = w[k * kBits / 32] >> (k * kBits % 32);
            store_piece<kBits / 4>(side + K::value_byte(t, (first + k) / 2, byte), &two);
        }
    } else {
        const int byte = K::byte_of(b * 8 + first % 8);
        store_piece<V * kBits / 8>(side + K::key_unit(t, first / 8, byte / K::U) + byte % K::U, w);
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
// value rows, each by D/V lanes of one wave.
template <int F, int NB, int RT>
__global__ __launch_bounds__(kRowThreads) void k_kv_write(WriteArgs a) {
    constexpr int V = row_values(RT), kLanes = 32 * NB / V, kPer = 64 / kLanes;
    __shared__ float2 cs[kMaxHeadDim / 2];
    const int64_t t = token_of(blockIdx.x, a.T);
    if (a.r.rot) {
        rope_table(a.r, a.positions[t], cs, threadIdx.x, kRowThreads);
        __syncthreads();
    }
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int sub = lane / kLanes, at_lane = lane - sub * kLanes, n = V * at_lane;
    if (sub >= kPer) return;
    const int page = 1 << a.c.page_shift;
    const int64_t slot = a.slots[t], pg = slot >> a.c.page_shift;
    const bool keep = a.c.has_page(pg);
    const int at = (int)(slot & (page - 1));
    const int64_t side = Kv<F, NB>::side_bytes(page);
    uint8_t *base = a.c.page_at(keep ? pg : 0, side);
    const int H = a.c.heads, rows = a.Hq + 2 * H, step = gridDim.y * kRowWaves * kPer;
    for (int row = (blockIdx.y * kRowWaves + wave) * kPer + sub; row < rows; row += step) {
        float y[V];
        if (row < a.Hq) {
            rotate<RT, V>(a.q, t * a.qs.token + row * a.qs.head, n, a.r, cs, y);
            store_row<RT, V>(a.qo, t * a.qos.token + row * a.qos.head + n, y);
        } else {
            const bool values = row >= a.Hq + H;
            const int h = row - a.Hq - (values ? H : 0);
            if (values)
                load_row<RT, V>(a.v, t * a.vs.token + h * a.vs.head + n, y);
            else
                rotate<RT, V>(a.k, t * a.ks.token + h * a.ks.head, n, a.r, cs, y);
            if (keep) store_values<F, NB, V>(base + (2 * h + values) * side, page, at, at_lane, values, y);
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
    const int per_wave = 64 / (32 * NB / row_values(rt));
    const dim3 grid((unsigned)a.T, (unsigned)row_parts(a.T, a.Hq + 2 * a.c.heads, kRowWaves * per_wave));
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
