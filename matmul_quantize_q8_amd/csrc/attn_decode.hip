// Attention of one new token over the paged key-value cache (include/qmm.h
// states the formula).
//
// One pass over the cache with the running maximum m and sum l of the softmax.
// The sequence is cut into chunks of positions; a workgroup takes one chunk of
// one key head for up to 16 of its query heads, and its four waves take tiles
// of 32 positions in turn.  A wave works alone: no LDS and no barrier until its
// last tile.  Per tile, with matrix instructions of 16 x 16 x 32 (f16, f32 sums):
//
//   S[position][head] = K q   A = 16 key rows, B = the query heads; one per
//                             block of 32 values, its result times the block's
//                             scale, so that codes enter as small integers;
//   O[value][head] += V^T w   A = 16 values of 32 positions, B = the weights
//                             exp(S - m), times the positions' block scales.
//
// The cache's byte order makes both A operands a lane's own loaded bytes (the
// group's lane (g, r) is the wave's lane 16 g + r), and S comes out of the
// first in the lanes that the second needs it in, so nothing crosses lanes but
// the maximum.  Codes are exact in f16; queries and weights enter as two f16
// each (the value and what its rounding left: 22 bits), so a product keeps
// f32's accuracy to 2^-21.
//
// The partial results of several chunks are joined by a second launch:
//   M = max m,  l = sum l_i exp(m_i - M),  out = sum o_i exp(m_i - M) / l.
#include "kv_layout.h"

namespace qmm {

constexpr int kAttnThreads = 256, kAttnWaves = 4;
constexpr int kTile = 32;                       // positions of a wave's tile
constexpr int kHeadTile = 16;                   // query heads of a workgroup
constexpr float kLog2e = 1.44269504088896340736f;

typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

__device__ __forceinline__ v4f mfma(v4u a, v4u b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// Two f32 as two f16, to nearest even.
__device__ __forceinline__ v2h to_halves(float a, float b) {
    const v2f f = {a, b};
    return __builtin_convertvector(f, v2h);
}

// a and b as hi + lo of two f16 each.
__device__ __forceinline__ void split_halves(float a, float b, uint32_t &hi, uint32_t &lo) {
    const v2h h = to_halves(a, b);
    hi = __builtin_bit_cast(uint32_t, h);
    lo = __builtin_bit_cast(uint32_t, to_halves(a - (float)h.x, b - (float)h.y));
}

// Maximum / sum over the four lanes n, n + 16, n + 32, n + 48, in all of them.
// A permlane swap exchanges the odd rows of 16 (or the upper 32 lanes) of one
// register with the even rows (the lower 32) of the other: of two copies of x,
// one comes back with the even row's value in both rows and the other with the
// odd row's.  Written as instructions, with the wait that a register just
// written needs, because the compiler's builtin yields its first result twice.
template <bool W32>
__device__ __forceinline__ void swap_rows(float x, float &even, float &odd) {
    even = odd = x;
    if constexpr (W32)
        asm volatile("s_nop 1\n\tv_permlane32_swap_b32 %0, %1" : "+v"(even), "+v"(odd));
    else
        asm volatile("s_nop 1\n\tv_permlane16_swap_b32 %0, %1" : "+v"(even), "+v"(odd));
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

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// ---------------------------------------------------------------------------
// A lane's bytes of a group, and its scales
// ---------------------------------------------------------------------------
template <int BYTES>
struct __attribute__((packed, aligned(BYTES))) Unit {
    uint32_t w[BYTES / 4];
};

// A lane's L bytes of the codes at `codes`: unit u of lane i is at (64 u + i) U.
template <int F, int NB>
__device__ __forceinline__ void load_codes(const uint8_t *codes, int lane, uint32_t (&x)[Kv<F, NB>::L / 4]) {
    using K = Kv<F, NB>;
#pragma unroll
    for (int u = 0; u < K::NU; ++u) {
        const Unit<K::U> v = *reinterpret_cast<const Unit<K::U> *>(codes + (u * 64 + lane) * K::U);
#pragma unroll
        for (int i = 0; i < K::U / 4; ++i) x[u * (K::U / 4) + i] = v.w[i];
    }
}

// The f16 scales of positions 4g .. 4g+3 of a group: [4][NB], two to a word.
template <int NB>
__device__ __forceinline__ void load_scales(const uint8_t *scales, int g, uint32_t (&x)[2 * NB]) {
    constexpr int B = NB % 2 ? 8 : 16;
#pragma unroll
    for (int u = 0; u < 8 * NB / B; ++u) {
        const Unit<B> v = *reinterpret_cast<const Unit<B> *>(scales + g * 8 * NB + u * B);
#pragma unroll
        for (int i = 0; i < B / 4; ++i) x[u * (B / 4) + i] = v.w[i];
    }
}

// Scale of position i, block b of such words.
template <int NB>
__device__ __forceinline__ float scale_of(const uint32_t (&x)[2 * NB], int i, int b) {
    const int k = i * NB + b;
    const v2h h = __builtin_bit_cast(v2h, x[k >> 1]);
    return (float)((k & 1) ? h.y : h.x);
}

// ---------------------------------------------------------------------------
// Codes as operands
// ---------------------------------------------------------------------------
// Integers u < 256 in the low bytes of two halves are, as f16, u * 2^-24.  The
// key product takes them so (its accumulator starts at the offset's share, and
// its result is scaled by 2^24); the value product takes (u - offset) * 2^-9,
// one packed multiply-add away.
constexpr float kKeyUnit = 0x1p-24f, kValueUnit = 0x1p-9f;

template <int F, int NB>
__device__ __forceinline__ v4u key_operand(const uint32_t (&x)[Kv<F, NB>::L / 4], int b) {
    v4u a;
    if constexpr (F == KV_F16) {
#pragma unroll
        for (int j = 0; j < 4; ++j) a[j] = x[4 * b + j];
    } else if constexpr (F == KV_Q8_0) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            a[2 * j] = __builtin_amdgcn_perm(0u, x[2 * b + j], 0x0c010c00u);
            a[2 * j + 1] = __builtin_amdgcn_perm(0u, x[2 * b + j], 0x0c030c02u);
        }
    } else {                                    // pairs (j, j + 4): the queries are in that order too
#pragma unroll
        for (int j = 0; j < 4; ++j) a[j] = (x[b] >> (4 * j)) & 0x000f000fu;
    }
    return a;
}

// Query slots of lane g's eight values of a block, in the key operand's order.
template <int F>
__device__ __forceinline__ constexpr int query_slot(int s) {
    return F == KV_Q4_0 ? (s >> 1) + 4 * (s & 1) : s;
}

__device__ __forceinline__ uint32_t offset_codes(uint32_t u, float unit, float offset) {
    const v2h m = {(_Float16)unit, (_Float16)unit}, c = {(_Float16)offset, (_Float16)offset};
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(v2h, u), m, c));
}

// Values 32b + 2r + e of the lane's four positions of a group, as two words of
// two positions each.
template <int F, int NB>
__device__ __forceinline__ void value_words(const uint32_t (&x)[Kv<F, NB>::L / 4], int b, uint32_t (&lo)[2],
                                            uint32_t (&hi)[2]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {               // positions 2j, 2j + 1; lo: e = 0, hi: e = 1
        if constexpr (F == KV_F16) {
            const uint32_t p = x[2 * j * NB + b], q = x[(2 * j + 1) * NB + b];
            lo[j] = __builtin_amdgcn_perm(q, p, 0x05040100u);
            hi[j] = __builtin_amdgcn_perm(q, p, 0x07060302u);
        } else {
            constexpr int W = F == KV_Q8_0 ? 2 * NB : NB;
            const int kp = 2 * j * W + (F == KV_Q8_0 ? 2 * b : b), kq = kp + W;
            const uint32_t p = x[kp >> 2], q = x[kq >> 2];
            const uint32_t sel = 0x0c040c00u + (uint32_t)(kp & 3) + ((uint32_t)(kq & 3) << 16);
            const uint32_t u = __builtin_amdgcn_perm(q, p, sel);
            if constexpr (F == KV_Q8_0) {
                const uint32_t v = __builtin_amdgcn_perm(q, p, sel + 0x00010001u);
                lo[j] = offset_codes(u, 0x1p15f, -128.0f * kValueUnit);
                hi[j] = offset_codes(v, 0x1p15f, -128.0f * kValueUnit);
            } else {
                lo[j] = offset_codes(u & 0x000f000fu, 0x1p15f, -8.0f * kValueUnit);
                hi[j] = offset_codes(u & 0x00f000f0u, 0x1p11f, -8.0f * kValueUnit);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// One chunk
// ---------------------------------------------------------------------------
// Weights of up to e^4 are let stand before the maximum is moved (moving it
// multiplies every accumulator); they, the scales and the weights' factor stay
// inside f16: e^4 * 2 * 2^8 = 27 955.  A value scale of 2 and more (values
// beyond 254) drops the factor and the slack for the rest of the wave's tiles.
constexpr float kMaxSlack = 4.0f, kWeightScale = 256.0f;

template <int F, int NB, bool MASKED>
__global__ __launch_bounds__(kAttnThreads, NB == 8 ? 1 : 2) void k_attn_chunk(AttnArgs a, int rt) {
    using K = Kv<F, NB>;
    constexpr int D = 32 * NB, LW = K::L / 4;
    constexpr bool kScaled = K::kScaled;
    // scores are kept in log2 units, or with a mask in natural ones (the lowest f32 has to stay finite)
    constexpr float kUnit = MASKED ? 1.0f : kLog2e;
    __shared__ float join[2 * (8 * NB + 2) * 64];

    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;
    const int group = a.Hq / a.c.heads, tiles = (group + kHeadTile - 1) / kHeadTile;
    const int kv = blockIdx.y / tiles, h0 = (blockIdx.y - kv * tiles) * kHeadTile;
    const int b = blockIdx.z, split = blockIdx.x;
    const bool live = h0 + n < group;
    const int hq = kv * group + h0 + (live ? n : 0);

    const int len = a.lens[b], shift = a.c.page_shift, page = 1 << shift;
    const bool bad_len = len < 0 || len > a.max_len;
    const int lo = a.window && !bad_len ? max(0, len - a.window) : 0;
    const int from = (lo & ~(kGroup - 1)) + split * a.chunk;
    const int to = bad_len ? from : from + min(len - from, a.chunk);
    const int64_t side = K::side_bytes(page);

    // The queries: scaled by a power of two to below 2^8, split in two f16.
    v4u qh[NB], ql[NB];
    float qoff[NB], unit;
    {
        float x[NB][8], top = 0.0f;
        const int64_t row = b * a.qs.token + hq * a.qs.head;
#pragma unroll
        for (int blk = 0; blk < NB; ++blk)
#pragma unroll
            for (int s = 0; s < 8; s += 4) {
                const int64_t at = row + blk * 32 + g * 8 + s;
                float4 v = rt == R_F32 ? load4<R_F32>(a.q, at)
                                       : rt == R_F16 ? load4<R_F16>(a.q, at) : load4<R_BF16>(a.q, at);
                if (!live) v = make_float4(0.f, 0.f, 0.f, 0.f);
                x[blk][s] = v.x;
                x[blk][s + 1] = v.y;
                x[blk][s + 2] = v.z;
                x[blk][s + 3] = v.w;
                top = fmaxf(top, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
            }
        top = max_rows(top);
        const int e = top > 0.0f && top < INFINITY ? min(max(7 - ilogbf(top), -120), 120) : 0;
        const float up = ldexpf(1.0f, e);
        unit = ldexpf(a.scale, -e) * (kScaled ? 0x1p24f : 1.0f);
#pragma unroll
        for (int blk = 0; blk < NB; ++blk) {
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float u = x[blk][query_slot<F>(2 * j)] * up, v = x[blk][query_slot<F>(2 * j + 1)] * up;
                uint32_t hi, lw;
                split_halves(u, v, hi, lw);
                qh[blk][j] = hi;
                ql[blk][j] = lw;
                sum += u + v;
            }
            qoff[blk] = kScaled ? -(F == KV_Q8_0 ? 128.0f : 8.0f) * kKeyUnit * sum_rows(sum) : 0.0f;
        }
    }

    v4f o[NB][2];
#pragma unroll
    for (int blk = 0; blk < NB; ++blk) o[blk][0] = o[blk][1] = v4f{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.0f, factor = kWeightScale, slack = kMaxSlack * kUnit;

    int pages = 0;                              // lane i: the page of the i-th group of this wave's next 32 tiles
    const int ntiles = (to - from + kTile - 1) / kTile;
    int count = 0;
    for (int tile = wave; tile < ntiles; tile += kAttnWaves, ++count) {
        if ((count & 31) == 0) {
            const int t = from + (tile + (lane >> 1) * kAttnWaves) * kTile + (lane & 1) * kGroup;
            pages = t < to ? a.pages[b * a.pages_stride + (t >> shift)] : 0;
        }
        const int t0 = from + tile * kTile;
        uint32_t kx[2][LW], vx[2][LW], ks[2][2 * NB], vs[2][2 * NB];
        bool bad = false;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            // a second group past the end is not looked up: the first is read again and not used
            const int t = t0 + j * kGroup < to ? t0 + j * kGroup : t0;
            int p = __builtin_amdgcn_readlane(pages, 2 * (count & 31) + (t != t0));
            if (!a.c.has_page(p)) {
                bad = true;
                p = 0;
            }
            const uint8_t *kside = a.c.page_at(p, side) + 2 * kv * side, *vside = kside + side;
            const int at = t & (page - 1);
            load_codes<F, NB>(kside + (at >> 4) * K::kGroupBytes, lane, kx[j]);
            if constexpr (kScaled) load_scales<NB>(kside + (page >> 4) * K::kGroupBytes + at * NB * 2, g, ks[j]);
            load_codes<F, NB>(vside + (at >> 4) * K::kGroupBytes, lane, vx[j]);
            if constexpr (kScaled) load_scales<NB>(vside + (page >> 4) * K::kGroupBytes + at * NB * 2, g, vs[j]);
        }

        // scores of positions t0 + 16 j + 4 g + i
        float s[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            v4f z = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int blk = 0; blk < NB; ++blk) {
                const v4u key = key_operand<F, NB>(kx[j], blk);
                if constexpr (kScaled) {
                    v4f acc = {qoff[blk], qoff[blk], qoff[blk], qoff[blk]};
                    acc = mfma(key, qh[blk], acc);
                    acc = mfma(key, ql[blk], acc);
#pragma unroll
                    for (int i = 0; i < 4; ++i) z[i] = fmaf(scale_of<NB>(ks[j], i, blk), acc[i], z[i]);
                } else {
                    z = mfma(key, qh[blk], z);
                    z = mfma(key, ql[blk], z);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) s[j][i] = z[i] * unit;
        }
        if (a.softcap > 0.0f) {
#pragma unroll
            for (int k = 0; k < 8; ++k) s[k >> 2][k & 3] = a.softcap * tanhf(s[k >> 2][k & 3] / a.softcap);
        }
        if constexpr (!MASKED) {
#pragma unroll
            for (int k = 0; k < 8; ++k) s[k >> 2][k & 3] *= kLog2e;
        }
        if (bad) {
#pragma unroll
            for (int k = 0; k < 8; ++k) s[k >> 2][k & 3] = NAN;
        }
        if (MASKED || t0 < lo || t0 + kTile > to) {   // some positions may not be seen: whatever they hold is dropped
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int j = k >> 2, i = k & 3, t = t0 + j * kGroup + 4 * g + i;
                bool seen = t >= lo && t < to;
                if constexpr (MASKED) {
                    const float x = seen ? a.mask[b * a.mask_stride + t] : -INFINITY;
                    seen = x != -INFINITY;
                    s[j][i] += x;
                }
                if (!seen) {
                    s[j][i] = -INFINITY;
                    if constexpr (kScaled) {
#pragma unroll
                        for (int blk = 0; blk < NB; ++blk) {
                            const int w = i * NB + blk;
                            vs[j][w >> 1] &= (w & 1) ? 0x0000ffffu : 0xffff0000u;
                        }
                    } else {
#pragma unroll
                        for (int blk = 0; blk < NB; ++blk) vx[j][i * NB + blk] = 0u;
                    }
                }
            }
        }

        if constexpr (kScaled) {
            uint32_t any = 0;
#pragma unroll
            for (int i = 0; i < 2 * NB; ++i) any |= vs[0][i] | vs[1][i];
            if (factor != 1.0f && __any((any & 0x40004000u) != 0)) {
                factor = 1.0f;
                slack = 0.0f;
#pragma unroll
                for (int blk = 0; blk < NB; ++blk)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        o[blk][0][i] *= 1.0f / kWeightScale;
                        o[blk][1][i] *= 1.0f / kWeightScale;
                    }
            }
        }
        float top = fmaxf(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3])),
                          fmaxf(fmaxf(s[1][0], s[1][1]), fmaxf(s[1][2], s[1][3])));
        top = max_rows(top);
        if (__any(top > m + slack)) {
            const float next = fmaxf(m, top);
            const float alpha = m == next ? 1.0f : exp2_fast((m - next) * (kLog2e / kUnit));
            m = next;
            l *= alpha;
#pragma unroll
            for (int blk = 0; blk < NB; ++blk)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    o[blk][0][i] *= alpha;
                    o[blk][1][i] *= alpha;
                }
        }
        const float base = m == -INFINITY ? 0.0f : m;
        float p[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float d = s[k >> 2][k & 3] - base;
            p[k] = exp2_fast(MASKED ? d * kLog2e : d);
            l += p[k];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) p[k] *= factor;
        v4u wh, wl;
#pragma unroll
        for (int blk = 0; blk < NB; ++blk) {
            if (kScaled || blk == 0) {
#pragma unroll
                for (int k = 0; k < 8; k += 2) {
                    float u = p[k], v = p[k + 1];
                    if constexpr (kScaled) {
                        u *= scale_of<NB>(vs[k >> 2], k & 3, blk);
                        v *= scale_of<NB>(vs[k >> 2], (k & 3) + 1, blk);
                    }
                    uint32_t hi, lw;
                    split_halves(u, v, hi, lw);
                    wh[k >> 1] = hi;
                    wl[k >> 1] = lw;
                }
            }
            uint32_t x0[2][2], x1[2][2];
            value_words<F, NB>(vx[0], blk, x0[0], x1[0]);
            value_words<F, NB>(vx[1], blk, x0[1], x1[1]);
            const v4u va = {x0[0][0], x0[0][1], x0[1][0], x0[1][1]}, vb = {x1[0][0], x1[0][1], x1[1][0], x1[1][1]};
            o[blk][0] = mfma(va, wh, o[blk][0]);
            o[blk][1] = mfma(vb, wh, o[blk][1]);
            o[blk][0] = mfma(va, wl, o[blk][0]);
            o[blk][1] = mfma(vb, wl, o[blk][1]);
        }
    }

    // The wave's result, then the four waves' in a fixed order: 0 + 2, 1 + 3, both.
    l = sum_rows(l);
    const float back = (kScaled ? 1.0f / kValueUnit : 1.0f) / factor;
#pragma unroll
    for (int blk = 0; blk < NB; ++blk)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o[blk][0][i] *= back;
            o[blk][1][i] *= back;
        }
#pragma unroll
    for (int step = 2; step > 0; step >>= 1) {
        float *slot = join + (wave & (step - 1)) * (8 * NB + 2) * 64 + lane;
        if (step == 1) __syncthreads();
        if (wave >= step && wave < 2 * step) {
            slot[0] = m;
            slot[64] = l;
#pragma unroll
            for (int k = 0; k < 8 * NB; ++k) slot[(2 + k) * 64] = o[k >> 3][(k >> 2) & 1][k & 3];
        }
        __syncthreads();
        if (wave < step) {
            const float m2 = slot[0], l2 = slot[64], top = fmaxf(m, m2);
            const float base = top == -INFINITY ? 0.0f : top;
            const float w1 = exp2_fast((m - base) * (kLog2e / kUnit)), w2 = exp2_fast((m2 - base) * (kLog2e / kUnit));
            m = top;
            l = l * w1 + l2 * w2;
#pragma unroll
            for (int k = 0; k < 8 * NB; ++k)
                o[k >> 3][(k >> 2) & 1][k & 3] = o[k >> 3][(k >> 2) & 1][k & 3] * w1 + slot[(2 + k) * 64] * w2;
        }
    }
    if (wave != 0 || !live) return;
    if (bad_len) l = NAN;
    const int64_t head = (int64_t)b * a.Hq + hq;
    if (a.splits > 1) {
        float *part = a.part + (head * a.splits + split) * D;
#pragma unroll
        for (int blk = 0; blk < NB; ++blk)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<float2 *>(part + blk * 32 + 2 * (4 * g + i)) =
                    make_float2(o[blk][0][i], o[blk][1][i]);
        if (g == 0) a.part_ml[head * a.splits + split] = make_float2(m, l);
        return;
    }
    const float r = l == 0.0f ? 0.0f : 1.0f / l;
    const int64_t row = b * a.os.token + hq * a.os.head;
#pragma unroll
    for (int blk = 0; blk < NB; ++blk)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t at = row + blk * 32 + 2 * (4 * g + i);
            const float x = o[blk][0][i] * r, y = o[blk][1][i] * r;
            if (rt == R_F32)
                *reinterpret_cast<float2 *>(static_cast<float *>(a.out) + at) = make_float2(x, y);
            else
                *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.out) + at) =
                    rt == R_F16 ? pack2<R_F16>(x, y) : pack2<R_BF16>(x, y);
        }
    if (a.lse && g == 0) a.lse[head] = (m == -INFINITY ? 0.0f : m / kUnit) + logf(l);
}

// ---------------------------------------------------------------------------
// The chunks of a query head, one workgroup a head.  Their maxima are in the
// first launch's units.
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 256;

template <int RT>
__global__ __launch_bounds__(kJoinThreads) void k_attn_join(AttnArgs a, int D) {
    __shared__ float4 sums[kJoinThreads];
    __shared__ float red[4], ls[kJoinThreads];
    const int64_t head = blockIdx.x;
    const int tid = threadIdx.x, quads = D >> 2, rows = kJoinThreads / quads;
    const float2 *ml = a.part_ml + head * a.splits;
    float m = -INFINITY;
    for (int i = tid; i < a.splits; i += kJoinThreads) m = fmaxf(m, ml[i].x);
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) m = fmaxf(m, xor_shfl(m, k));
    if ((tid & 63) == 0) red[tid >> 6] = m;
    __syncthreads();
    m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const float base = m == -INFINITY ? 0.0f : m;
    const float to_log2 = a.mask ? kLog2e : 1.0f;

    const int row = tid / quads, quad = tid - row * quads;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.0f;
    if (row < rows) {
        for (int i = row; i < a.splits; i += rows) {
            const float2 x = ml[i];
            const float w = exp2_fast((x.x - base) * to_log2);
            const float4 v = reinterpret_cast<const float4 *>(a.part + (head * a.splits + i) * D)[quad];
            l = fmaf(w, x.y, l);
            o.x = fmaf(w, v.x, o.x);
            o.y = fmaf(w, v.y, o.y);
            o.z = fmaf(w, v.z, o.z);
            o.w = fmaf(w, v.w, o.w);
        }
    }
    sums[tid] = o;
    ls[tid] = l;
    __syncthreads();
    if (tid >= quads) return;
    for (int k = 1; k < rows; ++k) {
        const float4 v = sums[k * quads + tid];
        o.x += v.x;
        o.y += v.y;
        o.z += v.z;
        o.w += v.w;
        l += ls[k * quads + tid];
    }
    const float r = l == 0.0f ? 0.0f : 1.0f / l;
    const int64_t b = head / a.Hq, h = head - b * a.Hq;
    store4<RT>(a.out, b * a.os.token + h * a.os.head + 4 * quad, make_float4(o.x * r, o.y * r, o.z * r, o.w * r));
    if (a.lse && tid == 0) a.lse[head] = base * (to_log2 / kLog2e) + logf(l);
}

struct AttnSplit {
    int chunk, splits;
};

// Chunks of a multiple of 128 positions (a tile for each wave).
static AttnSplit attn_split(int64_t B, int64_t Hq, int64_t heads, int64_t max_len, int64_t window) {
    // a window starts anywhere in a group of 16
    const int64_t span = window > 0 && window < max_len ? window + kGroup - 1 : max_len;
    const int64_t group = Hq / heads, columns = B * heads * ((group + kHeadTile - 1) / kHeadTile);
    const int64_t want = (8 * kCUs + columns - 1) / columns;
    int64_t chunk = (span + want - 1) / want;
    chunk = (chunk + 127) / 128 * 128;
    if (chunk < 256) chunk = 256;
    return {(int)chunk, (int)((span + chunk - 1) / chunk)};
}

int64_t attn_workspace(int64_t B, int64_t Hq, int64_t heads, int64_t D, int64_t max_len, int64_t window) {
    const AttnSplit s = attn_split(B, Hq, heads, max_len, window);
    return B * Hq * s.splits * (D + 2) * 4;
}

template <int F, int NB>
static hipError_t launch_attn_f(int rt, AttnArgs a, int64_t B, void *workspace, hipStream_t st) {
    const AttnSplit s = attn_split(B, a.Hq, a.c.heads, a.max_len, a.window);
    int D = 32 * NB;
    a.splits = s.splits;
    a.chunk = s.chunk;
    a.part = static_cast<float *>(workspace);
    a.part_ml = reinterpret_cast<float2 *>(a.part + B * a.Hq * s.splits * D);
    const int group = a.Hq / a.c.heads, tiles = (group + kHeadTile - 1) / kHeadTile;
    void *args[] = {(void *)&a, (void *)&rt};
    const void *k = a.mask ? (const void *)k_attn_chunk<F, NB, true> : (const void *)k_attn_chunk<F, NB, false>;
    hipError_t e = hipLaunchKernel(k, dim3((unsigned)s.splits, (unsigned)(a.c.heads * tiles), (unsigned)B),
                                   dim3(kAttnThreads), args, 0, st);
    if (e != hipSuccess || s.splits == 1) return e;
    void *jargs[] = {(void *)&a, (void *)&D};
    const void *j = rt == R_F32 ? (const void *)k_attn_join<R_F32>
                    : rt == R_F16 ? (const void *)k_attn_join<R_F16> : (const void *)k_attn_join<R_BF16>;
    return hipLaunchKernel(j, dim3((unsigned)(B * a.Hq)), dim3(kJoinThreads), jargs, 0, st);
}

hipError_t launch_attn(int fmt, int nb, int rt, AttnArgs a, int64_t B, void *workspace, hipStream_t st) {
    QMM_KV_DISPATCH(launch_attn_f, rt, a, B, workspace, st);
}

}  // namespace qmm
