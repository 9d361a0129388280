// Attention of one new token over the paged key-value cache (include/qmm.h
// states the formula).
//
// One pass over the cache with the running maximum m and sum l of the softmax.
// The sequence is cut into chunks of positions; a workgroup takes one chunk of
// one key head for up to 16 of its query heads, and its four waves take tiles
// of 32 or 64 positions in turn.  A wave works alone, with no barrier until its
// last tile; only the queries and the tile's scales and mask pass through LDS.
// Per tile, with matrix instructions of 16 x 16 x 32 (f16, f32 sums):
//
//   S[position][head] = K q   A = 16 key rows, B = the query heads; one per
//                             block of 32 values, its result times the block's
//                             scale, so that codes enter as small integers;
//   O[value][head] += V^T w   A = 16 values of 32 positions, B = the weights
//                             2^(S - r), times the positions' block scales (r: below).
//
// The cache's byte order makes both A operands a lane's own loaded bytes (the
// group's lane (g, r) is the wave's lane 16 g + r), and S comes out of the
// first in the lanes that the second needs it in, so nothing crosses lanes but
// the maximum.  Codes are exact in f16; queries and weights enter as two f16
// each (the value and what its rounding left: 22 bits), so a product keeps
// f32's accuracy to 2^-21.
//
// What bounds it: memory in large unquantized caches (32 sequences of 32 heads of
// 128, f16, 1.46 GB: 248 us, 5.9 TB/s); in quantized ones a wave's own chain, whose every
// code takes about one vector instruction to become an operand.  There vector
// instructions run for 26 to 50 % of a wave's time, 18 to 45 % are waits for loads and LDS, and
// over the kernel about one wave a SIMD is left to fill them (131072 positions q4_0,
// 151 MB: 34 us, 4.5 TB/s; 16 heads a key head 2.8).
//
// The partial results of several chunks are joined by a second launch (attn_decode.hip).
#pragma once

#include <cfloat>
#include <type_traits>

#include "kv_layout.h"

namespace qmm {

constexpr int kAttnThreads = 256, kAttnWaves = 4;
constexpr int kHeadTile = 16;                   // query heads of a workgroup
constexpr float kLog2e = 1.44269504088896340736f, kLog2eRest = 1.92596299e-8f;     // log2 e in two parts
constexpr int kDppRowRor4 = 0x124;              // row_ror:4: lane i of 16 reads lane (i - 4) mod 16

typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

__device__ __forceinline__ v4f mfma(v4u a, v4u b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// a * x and b * y as hi + lo of two f16 each, x and y f16: hi is the product
// rounded to nearest even, lo what is left of it (one fused operation each, whose
// f16 factors and f16 result need no conversions of their own).
__device__ __forceinline__ void split_products(float a, _Float16 x, float b, _Float16 y, uint32_t &hi, uint32_t &lo) {
    const v2h h = {(_Float16)fmaf((float)x, a, 0.0f), (_Float16)fmaf((float)y, b, 0.0f)};
    const v2h l = {(_Float16)fmaf((float)x, a, -(float)h.x), (_Float16)fmaf((float)y, b, -(float)h.y)};
    hi = __builtin_bit_cast(uint32_t, h);
    lo = __builtin_bit_cast(uint32_t, l);
}
__device__ __forceinline__ void split_halves(float a, float b, uint32_t &hi, uint32_t &lo) {
    split_products(a, (_Float16)1.0f, b, (_Float16)1.0f, hi, lo);
}


__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// tanh to about 2^-22: Lambert's continued fraction, five levels deep, up to 0.6
// (its first dropped part is below 1e-9 there), beyond that (e^2x - 1) / (e^2x + 1).
__device__ __forceinline__ float tanh_f32(float x) {
    const float y = fminf(fabsf(x), 20.0f), z = y * y, e = exp2_fast(2.0f * kLog2e * y);
    const float num = y < 0.6f ? y * fmaf(z, fmaf(z, 21.0f, 1260.0f), 10395.0f) : e - 1.0f;
    const float den = y < 0.6f ? fmaf(z, fmaf(z, z + 210.0f, 4725.0f), 10395.0f) : e + 1.0f;
    return x != x ? x : copysignf(num / den, x);
}

// ---------------------------------------------------------------------------
// A lane's bytes of a group, and its scales
// ---------------------------------------------------------------------------
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

// A wave's scales of one side of a tile, [32][NB] halves in LDS: those of
// positions 16 j + 4 g .. + 3, two to a word.
template <int NB>
__device__ __forceinline__ void read_scales(const uint32_t *sc, int j, int g, uint32_t (&x)[2 * NB]) {
    constexpr int B = NB % 2 ? 8 : 16;
    const uint8_t *p = reinterpret_cast<const uint8_t *>(sc + j * 8 * NB + g * 2 * NB);
#pragma unroll
    for (int u = 0; u < 8 * NB / B; ++u) {
        const Unit<B> v = *reinterpret_cast<const Unit<B> *>(p + u * B);
#pragma unroll
        for (int i = 0; i < B / 4; ++i) x[u * (B / 4) + i] = v.w[i];
    }
}

// Scale of position i, block b of such words.
template <int NB>
__device__ __forceinline__ _Float16 scale_of(const uint32_t (&x)[2 * NB], int i, int b) {
    const int k = i * NB + b;
    const v2h h = __builtin_bit_cast(v2h, x[k >> 1]);
    return (k & 1) ? h.y : h.x;
}

// ---------------------------------------------------------------------------
// Codes as operands
// ---------------------------------------------------------------------------
// Codes u as halves without an integer conversion: u in the low bits of a half
// is, as f16, u * 2^-24, and one packed multiply-add makes it (u - offset) * 2^-9,
// exactly.  (The product could take u * 2^-24 and have its accumulator start at
// the offset's share.  That was tried, and cost accuracy: a matrix instruction
// aligns its products by their exponent fields, so a subnormal's leading zeros
// push out low bits.  Score errors were ten times as large with 4-bit codes.)
template <int F> constexpr float kCodeUnit = F == KV_F16 ? 1.0f : 0x1p-9f;

// Words of two codes each, at bit 0 (SHIFT = 0) or 4 of their halves.
template <int F, int SHIFT>
__device__ __forceinline__ uint32_t code_halves(uint32_t u) {
    constexpr float unit = SHIFT == 4 ? 0x1p11f : 0x1p15f, offset = -(F == KV_Q8_0 ? 128.0f : 8.0f) * 0x1p-9f;
    const v2h m = {(_Float16)unit, (_Float16)unit}, c = {(_Float16)offset, (_Float16)offset};
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(v2h, u), m, c));
}

template <int F, int NB>
__device__ __forceinline__ v4u key_operand(const uint32_t (&x)[Kv<F, NB>::L / 4], int b) {
    v4u a;
    if constexpr (F == KV_F16) {
#pragma unroll
        for (int j = 0; j < 4; ++j) a[j] = x[4 * b + j];
    } else if constexpr (F == KV_Q8_0) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            a[2 * j] = code_halves<F, 0>(__builtin_amdgcn_perm(0u, x[2 * b + j], 0x0c010c00u));
            a[2 * j + 1] = code_halves<F, 0>(__builtin_amdgcn_perm(0u, x[2 * b + j], 0x0c030c02u));
        }
    } else {                                    // pairs (j, j + 4): the queries are in that order too
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t y = x[b] >> (8 * j);
            a[2 * j] = code_halves<F, 0>(y & 0x000f000fu);
            a[2 * j + 1] = code_halves<F, 4>(y & 0x00f000f0u);
        }
    }
    return a;
}

// Query slots of lane g's eight values of a block, in the key operand's order.
template <int F>
__device__ __forceinline__ constexpr int query_slot(int s) {
    return F == KV_Q4_0 ? (s >> 1) + 4 * (s & 1) : s;
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
                lo[j] = code_halves<F, 0>(u);
                hi[j] = code_halves<F, 0>(v);
            } else {
                lo[j] = code_halves<F, 0>(u & 0x000f000fu);
                hi[j] = code_halves<F, 4>(u & 0x00f000f0u);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// One chunk
// ---------------------------------------------------------------------------
// Scores s are in log2 units.  A column's weights are p = 2^(s - r) for a reference r
// that lies kWeightBits under the largest score it was set by; r is moved (which
// multiplies every accumulator) when a score passes that one by kSlackBits.
//   What becomes two halves is p times its block's scale.  Two halves hold a product to
// 2^-22 of itself only above 2^-3: below, the low half is an f16 subnormal, and the
// error 2^-25 whatever the product.  So scales are staged times 2^lift (exact), and a
// tile of a quantized cache is common when they then all lie in [2^-7, 2), which two bits
// of a half tell: products stay below 2^(8 + 6 + 1), and a column's largest so far is
// above 1.
//   Other tiles (values of another magnitude, blocks of zeros) and those that follow get a
// reference rp of their own for the products, p 2^(r - rp), until r serves again: with e =
// log2 of a position's largest lifted scale, the largest s + e is kept between kLeastBits
// and kMostBits over rp, and moving rp multiplies the accumulators.  rp falls at most
// kReachBits under r, and a position without scales counts as kNoScale: sums stay in f32's
// range.  In f16 caches e is 0, and a tile is uncommon when some column's largest score is
// more than kSunkBits under r (it follows a position whose score exceeds all others by far).
//   (Without lift and rp results lost 2e-5 with q8_0 values of 1e-3, 4e-4 with values of
// 1e-4, and every digit beside a position of zero values whose score lay 16 above the rest.
// The price: 0 to 2 % of the time, 4 to 6 % with q4_0 rows of 192 and 256 values; where
// every tile is uncommon 5 to 12 %.)
constexpr float kWeightBits = 8.0f, kSlackBits = 6.0f, kSunkBits = 3.0f;
constexpr float kMostBits = 15.0f, kSetBits = 12.0f, kLeastBits = 8.0f, kReachBits = 56.0f, kNoScale = -40.0f;
constexpr uint32_t kScaleBits = 0x60006000u, kCommonScale = 0x20002000u;
// The lift a wave starts with: blocks whose largest value is in [0.06, 16) are common ones.
template <int F> constexpr int kFirstLift = F == KV_Q8_0 ? 4 : 0;
constexpr int kMostLift = 15;                   // 2^lift is an f16
constexpr __host__ __device__ uint32_t two_halves(int e) {      // of 2^e
    return (e >= -14 ? (uint32_t)(e + 15) << 10 : 1u << (e + 24)) * 0x10001u;
}

// A whole number at most `bits` under `top`, where the next reference is put: sums are
// then scaled exactly.  Where an f32 step is 16 (masks of -1e8) the difference is 16 or
// 0, and a weight of 2^16 is no f16: the reference is then `top` itself.
__device__ __forceinline__ float under(float top, float bits) {
    const float x = floorf(top - bits);
    return top - x > kMostBits ? top : x;
}

// ln(2^r l) for a whole r: l = m 2^k, m near 1, and r + k is exact, so the result carries
// one rounding of its own size.  (A mask's lowest value stands at r = -FLT_MAX, though its
// product with log2 e is below that.)
__device__ __forceinline__ float log_sum(float r, float l) {
    if (l == 0.0f) return -INFINITY;
    if (r == -FLT_MAX && l > 0.0f) return -FLT_MAX;
    int k;
    float m = frexpf(l, &k);
    if (m < 0.70710678f) {
        m *= 2.0f;
        --k;
    }
    const float n = r + (float)k;
    return fmaf(n, 0.693147182464599609375f, fmaf(n, -1.904654323148236e-9f, logf(m)));   // ln 2 in two parts
}

// e of position t of a tile whose scales are at sc; an infinite or NaN scale counts as the largest finite.
template <int NB>
__device__ __forceinline__ float scale_log2(const uint32_t *sc, int t) {
    uint32_t top = 0;
    if constexpr (NB % 2) {
#pragma unroll
        for (int k = t * NB; k < (t + 1) * NB; ++k) top = max(top, sc[k >> 1] >> (16 * (k & 1)) & 0x7fffu);
    } else {
        constexpr int B = NB == 6 ? 4 : 2 * NB;
        const uint8_t *d = reinterpret_cast<const uint8_t *>(sc + t * (NB / 2));
#pragma unroll
        for (int u = 0; u < 2 * NB / B; ++u) {
            const Unit<B> v = *reinterpret_cast<const Unit<B> *>(d + u * B);
#pragma unroll
            for (int i = 0; i < B / 4; ++i) top = max(top, max(v.w[i] & 0x7fffu, v.w[i] >> 16 & 0x7fffu));
        }
    }
    top = min(top, 0x7bffu);
    return top ? __builtin_amdgcn_logf(f16_bits_to_f32(top)) : kNoScale;
}

// Query heads of a key head fill the 16 columns of the score product only when
// there are more than eight.  With fewer, COLS = 2 or 4 groups of positions share
// the columns: head h of group c is column c * 16/COLS + h.  The products of all
// groups go into one accumulator, each with the queries in its own columns and
// zeros in the others, so scales, softmax and weights, the work per score, is
// done on full columns.  For the values' product the weights are masked to their
// group's columns again; the columns of a head are added up at the end.
constexpr int attn_cols(int group) { return group <= 4 ? 4 : group <= 8 ? 2 : 1; }

// A lane's bytes of four groups fit its registers beside the accumulators.
template <int F, int NB> constexpr bool kFourColumns = Kv<F, NB>::L <= 48;
// Groups of 16 positions in a wave's tile: four where a lane's bytes of them and the
// accumulators fit its registers (9 and more heads a key head, q8_0 of 96 values:
// 2980 GB/s with two, 3300 with four; q4_0 of 128 2625 and 2800, of 192, which
// spills, 2300 and 2130).
template <int F, int NB, int COLS>
constexpr int kTileGroups = COLS == 4 || Kv<F, NB>::L <= (COLS == 2 || NB <= 4 ? 24 : 0) ? 4 : 2;

// Waves a SIMD, which set the registers a wave has: three, but two for rows of 192 values
// and more and for tiles of four groups whose lanes hold 12 bytes and more of each, which
// spill at three or keep too few loads in flight (three and two, GB/s: q4_0 of 128 values
// with four heads a key head and f32 rows 3240, 3430; of 96 2510, 2630; q8_0 of 96 with one
// head and 16-bit rows 3840, 4050; rows of 64 values do not differ).  One wave for 256
// f16 values with f32 rows.
template <int F, int NB, int COLS>
constexpr bool kTwoWaves = NB >= 6 || (NB >= 3 && Kv<F, NB>::L >= 12 && kTileGroups<F, NB, COLS> == 4);
template <int F, int NB, int RT, int COLS>
constexpr int kAttnOccupancy = F == KV_F16 && NB == 8 && RT == R_F32 ? 1 : kTwoWaves<F, NB, COLS> ? 2 : 3;

template <int F, int NB, int RT, int COLS>
__global__ __launch_bounds__(kAttnThreads, (kAttnOccupancy<F, NB, RT, COLS>)) void k_attn_chunk(AttnArgs a) {
    using K = Kv<F, NB>;
    constexpr int D = 32 * NB, LW = K::L / 4;
    constexpr bool kScaled = K::kScaled;
    constexpr int GR = kTileGroups<F, NB, COLS>, kTile = GR * kGroup, HC = 16 / COLS, NS = GR / COLS;
    static_assert(COLS <= GR, "");
    static_assert(kScaled || COLS == 1, "an f16 cache's values are dropped by the lane that weighs them");
    // Rows of 16 bits are exact in one f16 once scaled (what an f16's subnormals
    // take from the smallest of them is 2^-32 of the largest), so only f32 queries
    // need their low parts.  (Weights keep theirs for results of every type: where
    // the values cancel, 2^-12 of a weight is more than a bf16 result's rounding.)
    constexpr int kQueryParts = RT == R_F32 ? 2 : 1;
    constexpr int SW = 8 * NB * GR, SR = (SW + 63) / 64;  // words of a side's scales of a tile, and of a lane
    constexpr int QE = COLS == 1 ? 64 : 4 * HC + 1;       // entries of a block's queries: (g, head), and one of zeros
    __shared__ float join[2 * (8 * NB + 2) * 64];
    __shared__ v4u queries[kQueryParts][NB][QE];
    __shared__ __attribute__((aligned(16))) uint32_t scales[kScaled ? kAttnWaves : 1][kScaled ? SW : 4];
    __shared__ float4 extras[kAttnWaves][kTile / 4];      // what is added to a tile's scores; -inf: not seen

    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4, c = n / HC;
    const int group = a.Hq / a.c.heads, tiles = COLS > 1 ? 1 : (group + kHeadTile - 1) / kHeadTile;
    const int kv = blockIdx.y / tiles, h0 = (blockIdx.y - kv * tiles) * kHeadTile, h = h0 + n % HC;
    const int b = blockIdx.z, split = blockIdx.x;
    const bool live = h < group;
    const int hq = kv * group + (live ? h : h0);

    float4 qx[NB][2];
#pragma unroll
    for (int k = 0; k < 2 * NB; ++k)
        qx[k >> 1][k & 1] = load4<RT>(a.q, b * a.qs.token + hq * a.qs.head + (k >> 1) * 32 + g * 8 + (k & 1) * 4);

    const int len = a.lens[b], shift = a.c.page_shift, page = 1 << shift;
    const bool bad_len = len < 0 || len > a.max_len;
    const int lo = a.window && !bad_len ? max(0, len - a.window) : 0;
    const int from = (lo & ~(kGroup - 1)) + split * a.chunk;
    const int to = bad_len ? from : from + min(len - from, a.chunk);
    const int64_t side = K::side_bytes(page);

    // Tiles wave, wave + 4, ... of the chunk.  A tile's keys are loaded as soon as
    // the last tile's are used up, and its values likewise, into the same
    // registers: the loads have the other half of a tile's work to arrive in.
    const int ntiles = (to - from + kTile - 1) / kTile;
    int pages = 0;                              // lane i: the page of the i-th group of this wave's next 64 / GR tiles
    const uint8_t *kside[GR];                   // the tile's groups: keys' side of the page and place in it
    int place[GR];
    bool bad = false, whole = false;
    uint32_t kx[GR][LW], vx[GR][LW], ks[SR], vs[SR];
    const auto look_up = [&](int tile) {
        const int t = from + (tile + lane / GR * kAttnWaves) * kTile + lane % GR * kGroup;
        pages = t < to ? a.pages[b * a.pages_stride + (t >> shift)] : 0;
    };
    const auto locate = [&](int tile, int count) {
        if (count > 0 && count % (64 / GR) == 0) {
            look_up(tile);
            asm volatile("" : "+v"(pages));     // waited for here, not at every tile's readlane
        }
        bad = false;
        const int t0 = from + tile * kTile;
        const auto group_at = [&](int j, int t) {
            int p = __builtin_amdgcn_readlane(pages, GR * (count % (64 / GR)) + (t != t0 ? j : 0));
            if (!a.c.has_page(p)) {
                bad = true;
                p = 0;
            }
            kside[j] = a.c.page_at(p, side) + 2 * kv * side;
            place[j] = t & (page - 1);
        };
        group_at(0, t0);
        whole = place[0] + kTile <= page;
        if (!whole) {
#pragma unroll
            for (int j = 1; j < GR; ++j)        // a group past the end is not looked up: the first is read again and not used
                group_at(j, t0 + j * kGroup < to ? t0 + j * kGroup : t0);
        }
    };
    const auto load = [&](bool values, uint32_t(&x)[GR][LW], uint32_t(&sc)[SR]) {
        const int64_t off = values ? side : 0;
        const uint8_t *const codes = kside[0] + off + (place[0] >> 4) * K::kGroupBytes;
        const uint8_t *const first = kside[0] + off + K::scale_byte(page, place[0]);
        if (whole) {                            // the tile lies in one page: its codes and its scales in one piece each
#pragma unroll
            for (int j = 0; j < GR; ++j) load_codes<F, NB>(codes + j * K::kGroupBytes, lane, x[j]);
            if constexpr (kScaled) {
#pragma unroll
                for (int k = 0; k < SR; ++k)
                    if (SW % 64 == 0 || lane + 64 * k < SW)
                        sc[k] = *reinterpret_cast<const uint32_t *>(first + 4 * (lane + 64 * k));
            }
            return;
        }
        load_codes<F, NB>(codes, lane, x[0]);
#pragma unroll
        for (int j = 1; j < GR; ++j)
            load_codes<F, NB>(kside[j] + off + (place[j] >> 4) * K::kGroupBytes, lane, x[j]);
        if constexpr (kScaled) {
#pragma unroll
            for (int k = 0; k < SR; ++k) {
                const int i = lane + 64 * k, j = i / (8 * NB);
                const uint8_t *p = first;
#pragma unroll
                for (int m = 64 * k / (8 * NB); m < GR && m <= (64 * k + 63) / (8 * NB); ++m)
                    if (m > 0 && j == m) p = kside[m] + off + K::scale_byte(page, place[m]);
                if (SW % 64 == 0 || i < SW) sc[k] = *reinterpret_cast<const uint32_t *>(p + 4 * (i - j * 8 * NB));
            }
        }
    };
    uint32_t *const sc = scales[kScaled ? wave : 0];
    const auto stage = [&](const uint32_t(&x)[SR]) {
#pragma unroll
        for (int k = 0; k < SR; ++k)
            if (SW % 64 == 0 || lane + 64 * k < SW) sc[lane + 64 * k] = x[k];
        __builtin_amdgcn_wave_barrier();
    };
    float mask = 0.0f;                          // lane i: the mask at the tile's position i
    const auto load_mask = [&](int tile) {      // before the keys, so that no wait is added
        const int t = from + tile * kTile + lane;
        if (a.mask && lane < kTile && t < to) mask = a.mask[b * a.mask_stride + t];
    };
    float4 *const extra = extras[wave];
    look_up(wave);
    asm volatile("" : "+v"(pages));             // and the queries with them: no wait for them reaches past the tile's loads
#pragma unroll
    for (int k = 0; k < 2 * NB; ++k) asm volatile("" : "+v"(qx[k >> 1][k & 1].x));
    if (wave < ntiles) {
        locate(wave, 0);
        load_mask(wave);
        load(false, kx, ks);
        load(true, vx, vs);
    }

    // The queries: scaled by a power of two to below 2^8, split in two f16, in LDS.
    float to_score, rest;                       // of the products: the score is their sum times it (or tanh's argument)
    {
        float x[NB][8], top = 0.0f;
#pragma unroll
        for (int k = 0; k < 2 * NB; ++k) {
            const float4 v = qx[k >> 1][k & 1];
            const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[k >> 1][(k & 1) * 4 + i] = live ? f[i] : 0.0f;
                top = fmaxf(top, live ? fabsf(f[i]) : 0.0f);
            }
        }
        top = max_rows(top);
        const int e = top > 0.0f && top < INFINITY ? min(max(7 - ilogbf(top), -120), 120) : 0;
        const float up = copysignf(ldexpf(1.0f, e), a.scale), unit = ldexpf(fabsf(a.scale), -e) / kCodeUnit<F>;
        if (a.softcap > 0.0f) {
            to_score = unit / a.softcap, rest = 0.0f;
        } else {                                // unit * log2 e in two parts, neither negative: -inf stays -inf
            to_score = unit * kLog2e;
            rest = fmaf(unit, kLog2e, -to_score) + unit * kLog2eRest;
            if (rest < 0.0f) {
                to_score = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, to_score) - 1u);
                rest = fmaf(unit, kLog2e, -to_score) + unit * kLog2eRest;
            }
        }
#pragma unroll
        for (int blk = 0; blk < NB; ++blk) {
            if ((blk & (kAttnWaves - 1)) != wave) continue;   // every wave has them all and writes its share
            v4u part[2];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t hi, lw;
                split_halves(x[blk][query_slot<F>(2 * j)] * up, x[blk][query_slot<F>(2 * j + 1)] * up, hi, lw);
                part[0][j] = hi;
                part[1][j] = lw;
            }
#pragma unroll
            for (int k = 0; k < kQueryParts; ++k) {
                if (c == 0) queries[k][blk][g * HC + n % HC] = part[k];
                if (COLS > 1 && lane == 0) queries[k][blk][QE - 1] = v4u{0, 0, 0, 0};
            }
        }
    }
    __syncthreads();
    int qat[COLS];                              // this lane's entry in the product of group j (mod COLS)
    uint32_t mine[COLS];                        // all ones where the lane's column is of that group
#pragma unroll
    for (int j = 0; j < COLS; ++j) {
        qat[j] = c == j ? g * HC + n % HC : QE - 1;
        mine[j] = c == j ? 0xffffffffu : 0u;
        if (COLS > 1) asm volatile("" : "+v"(mine[j]));     // stays a mask: as conditions they hold scalar registers, which spill
    }

    v4f o[NB][2];
#pragma unroll
    for (int blk = 0; blk < NB; ++blk) o[blk][0] = o[blk][1] = v4f{0.f, 0.f, 0.f, 0.f};
    float r = -INFINITY, rp = -INFINITY, l = 0.0f;

    int count = 0, lift = kFirstLift<F>;
    uint32_t factor = two_halves(kFirstLift<F>);
    uint64_t apart = 0;                         // the lanes whose column's rp is not its r
    const auto step = [&](int tile, auto last) {
        constexpr bool more = !decltype(last)::value;
        const int t0 = from + tile * kTile;
        const bool masked = a.mask || t0 < lo || t0 + kTile > to;
        const bool finished = masked || a.softcap > 0.0f;       // s holds scores, not the products' sums they come from
        ++count;
        if (bad) l = NAN;                       // and stays so: a bad page is told whatever the mask hides

        // scores of positions t0 + 16 (COLS j + c) + 4 g + i
        float s[NS][4];
        if constexpr (kScaled) stage(ks);
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            uint32_t kd[2 * NB];
            if constexpr (kScaled) read_scales<NB>(sc, COLS * j + c, g, kd);
            v4f z = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int blk = 0; blk < NB; ++blk) {
                v4f acc = kScaled ? v4f{0.f, 0.f, 0.f, 0.f} : z;
#pragma unroll
                for (int m = 0; m < COLS; ++m) {
                    const v4u key = key_operand<F, NB>(kx[COLS * j + m], blk);
#pragma unroll
                    for (int k = 0; k < kQueryParts; ++k) acc = mfma(key, queries[k][blk][qat[m]], acc);
                }
                if constexpr (kScaled) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) z[i] = fmaf((float)scale_of<NB>(kd, i, blk), acc[i], z[i]);
                } else {
                    z = acc;
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) s[j][i] = z[i];
        }
        if (masked && lane < kTile) {           // the lowest f32 stays finite in log2 units, NaN stays NaN
            const float y = mask * kLog2e;
            reinterpret_cast<float *>(extra)[lane] = t0 + lane < lo || t0 + lane >= to || mask == -INFINITY ? -INFINITY
                                                     : y < -FLT_MAX ? -FLT_MAX : y;
        }
        __builtin_amdgcn_wave_barrier();
        if constexpr (more) {
            locate(tile + kAttnWaves, count);
            load_mask(tile + kAttnWaves);
            load(false, kx, ks);
        }
        if (a.softcap > 0.0f) {
#pragma unroll
            for (int k = 0; k < 4 * NS; ++k)
                s[k >> 2][k & 3] = a.softcap * kLog2e * tanh_f32(s[k >> 2][k & 3] * to_score);
        } else if (masked) {
#pragma unroll
            for (int k = 0; k < 4 * NS; ++k) s[k >> 2][k & 3] = fmaf(s[k >> 2][k & 3], to_score, s[k >> 2][k & 3] * rest);
        }
        if (masked) {                           // some positions may not be seen: whatever they hold is dropped
#pragma unroll
            for (int j = 0; j < NS; ++j) {
                const float4 v = extra[(COLS * j + c) * (kGroup / 4) + g];
                const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[j][i] = x[i] == -INFINITY ? -INFINITY : s[j][i] + x[i];
                    if constexpr (!kScaled) {
#pragma unroll
                        for (int blk = 0; blk < NB; ++blk)
                            if (x[i] == -INFINITY) vx[j][i * NB + blk] = 0u;
                    }
                }
            }
            if constexpr (kScaled) {            // codes are finite, scales need not be: a common one instead
                const float *const x = reinterpret_cast<const float *>(extra);
                const uint32_t least_common = two_halves(-7 - lift);
#pragma unroll
                for (int k = 0; k < SR; ++k) {
                    const int e = 2 * (lane + 64 * k);
                    if (SW % 64 != 0 && e >= 2 * SW) continue;
                    if (x[e / NB] == -INFINITY) vs[k] = (vs[k] & 0xffff0000u) | (least_common & 0x0000ffffu);
                    if (x[(e + 1) / NB] == -INFINITY) vs[k] = (vs[k] & 0x0000ffffu) | (least_common & 0xffff0000u);
                }
            }
        }

        uint32_t odd = 0u;                      // kScaleBits of scales that are not in the common range
        const auto stage_lifted = [&] {
            uint32_t x[SR];
#pragma unroll
            for (int k = 0; k < SR; ++k)
                x[k] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(v2h, vs[k]) * __builtin_bit_cast(v2h, factor));
            stage(x);
            odd = 0u;
#pragma unroll
            for (int k = 0; k < SR; ++k)
                if (SW % 64 == 0 || lane + 64 * k < SW) odd |= x[k] ^ kCommonScale;
        };
        if constexpr (kScaled) stage_lifted();
        float f = finished ? 1.0f : to_score;   // what turns s into a score
        float top = s[0][0];
#pragma unroll
        for (int k = 1; k < 4 * NS; ++k) top = fmaxf(top, s[k >> 2][k & 3]);
        top = max_rows(top) * f;
        const float over = top - r;
        constexpr float kMid = 0.5f * (kWeightBits + kSlackBits - kSunkBits), kHalf = kMid + kSunkBits;
        uint64_t uncommon = apart;              // lanes that make the tile an uncommon one; moved: or move r
        if constexpr (kScaled) uncommon |= __builtin_amdgcn_ballot_w64((odd & kScaleBits) != 0);
        const uint64_t moved = uncommon | __builtin_amdgcn_ballot_w64(kScaled ? over > kWeightBits + kSlackBits
                                                                              : fabsf(over - kMid) > kHalf);
        float base = r, sum = 0.0f;             // the exponents' subtrahend; the weights' sum of an uncommon tile
        if (moved != 0) {
            const bool rise = over > kWeightBits + kSlackBits;
            const float next = rise ? under(top, kWeightBits) : r;
            float set = next, by = 1.0f;        // rp, and what the accumulators are multiplied by beside its move
            if constexpr (!kScaled) uncommon |= __builtin_amdgcn_ballot_w64(over < -kSunkBits && over > -kReachBits);
            if (uncommon != 0) {
                float most = top;
                if constexpr (kScaled) {
                    stage(vs);
                    const float e = lane < kTile ? scale_log2<NB>(sc, lane) : kNoScale, largest = max_rows(max16_lanes(e));
                    if (largest > kNoScale && fabsf(largest + (float)lift + 2.5f) > 3.5f) {      // to [2^-2, 2^-1)
                        const int was = lift;
                        lift = uniform(min(max(-2 - (int)floorf(largest), 0), kMostLift));
                        factor = two_halves(lift);
                        by = ldexpf(1.0f, lift - was);
                    }
                    if (lane < kTile) reinterpret_cast<float *>(extra)[lane] = e + (float)lift;
                    __builtin_amdgcn_wave_barrier();
                    most = -INFINITY;
#pragma unroll
                    for (int j = 0; j < NS; ++j) {
                        const float4 v = extra[(COLS * j + c) * (kGroup / 4) + g];
                        const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) most = fmaxf(most, fmaf(s[j][i], f, x[i]));
                    }
                    most = max_rows(most);
                    stage_lifted();
                }
                // r serves the products too where they lie high enough over it: a tile of common scales (lifted
                // anew, or after an uncommon one) need not reach what one with blocks far below the others has to
                const bool wide = kScaled && __builtin_amdgcn_ballot_w64((odd & kScaleBits) != 0) != 0;
                const float over_r = most - next, over_p = most - rp;
                if (!(over_r >= (wide ? kLeastBits : 0.0f) && over_r <= kMostBits)) {
                    const bool move = over_p > kMostBits || (over_p < kLeastBits && most > next - kReachBits);
                    set = move ? fmaxf(under(most, kSetBits), next - kReachBits) : rp;
                }
                apart = __builtin_amdgcn_ballot_w64(set != next);
            }
            l *= r == next ? 1.0f : exp2_fast(r - next);
            by *= rp == set ? 1.0f : exp2_fast(rp - set);
            r = base = next;
            rp = set;
#pragma unroll
            for (int blk = 0; blk < NB; ++blk)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    o[blk][0][i] *= by;
                    o[blk][1][i] *= by;
                }
            if (uncommon != 0) {                // r and rp may be far apart: an exponent for each, without a rounding of s
                const float base_r = r == -INFINITY ? 0.0f : r, base_p = rp == -INFINITY ? 0.0f : rp;
#pragma unroll
                for (int k = 0; k < 4 * NS; ++k) {
                    const float x = s[k >> 2][k & 3];
                    sum += exp2_fast(finished ? x - base_r : fmaf(x, rest, fmaf(x, f, -base_r)));
                    s[k >> 2][k & 3] = finished ? x - base_p : fmaf(x, rest, fmaf(x, f, -base_p));
                }
                f = 1.0f, base = 0.0f;
            }
        }
        base = base == -INFINITY ? 0.0f : base;
        float p[NS][4], total = 0.0f;
#pragma unroll
        for (int k = 0; k < 4 * NS; ++k) {
            p[k >> 2][k & 3] = exp2_fast(fmaf(s[k >> 2][k & 3], f, -base));
            total += p[k >> 2][k & 3];
        }
        l += uncommon != 0 ? sum : total;
        uint32_t vd[NS][2 * NB];
        if constexpr (kScaled) {
#pragma unroll
            for (int j = 0; j < NS; ++j) read_scales<NB>(sc, COLS * j + c, g, vd[j]);
        }
        uint32_t wh[NS][2], wl[NS][2];          // the weights, two positions a word
#pragma unroll
        for (int blk = 0; blk < NB; ++blk) {
            if (kScaled || blk == 0) {
#pragma unroll
                for (int k = 0; k < 2 * NS; ++k) {
                    const int j = k >> 1, i = 2 * (k & 1);
                    const _Float16 one = (_Float16)1.0f;
                    split_products(p[j][i], kScaled ? scale_of<NB>(vd[j], i, blk) : one, p[j][i + 1],
                                   kScaled ? scale_of<NB>(vd[j], i + 1, blk) : one, wh[j][k & 1], wl[j][k & 1]);
                }
            }
#pragma unroll
            for (int pair = 0; pair < GR / 2; ++pair) {   // two groups of positions to a product
                uint32_t e0[2][2], e1[2][2];
                value_words<F, NB>(vx[2 * pair], blk, e0[0], e1[0]);
                value_words<F, NB>(vx[2 * pair + 1], blk, e0[1], e1[1]);
                const v4u va = {e0[0][0], e0[0][1], e0[1][0], e0[1][1]};
                const v4u vb = {e1[0][0], e1[0][1], e1[1][0], e1[1][1]};
                const auto weights = [&](const uint32_t(&w)[NS][2]) {
                    const int j0 = 2 * pair / COLS, j1 = (2 * pair + 1) / COLS;
                    if constexpr (COLS == 1) return v4u{w[j0][0], w[j0][1], w[j1][0], w[j1][1]};
                    const uint32_t m0 = mine[(2 * pair) % COLS], m1 = mine[(2 * pair + 1) % COLS];
                    return v4u{w[j0][0] & m0, w[j0][1] & m0, w[j1][0] & m1, w[j1][1] & m1};
                };
                const v4u high = weights(wh), low = weights(wl);
                o[blk][0] = mfma(va, high, o[blk][0]);
                o[blk][1] = mfma(vb, high, o[blk][1]);
                o[blk][0] = mfma(va, low, o[blk][0]);
                o[blk][1] = mfma(vb, low, o[blk][1]);
            }
        }
        if constexpr (more) load(true, vx, vs);
    };
    // The last tile is a call of its own: with one loop and a condition on the
    // loads, every tile waits for all of them.
    int tile = wave;
    for (; tile + kAttnWaves < ntiles; tile += kAttnWaves) step(tile, std::false_type{});
    if (tile < ntiles) step(tile, std::true_type{});

    // The wave's result, then the four waves' in a fixed order: 0 + 2, 1 + 3, both.
    l = sum_rows(l);
    const float back = ldexpf(r == rp ? 1.0f : exp2_fast(rp - r), -lift) / kCodeUnit<F>;      // sums of p times the values
#pragma unroll
    for (int blk = 0; blk < NB; ++blk)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o[blk][0][i] *= back;
            o[blk][1][i] *= back;
        }
    if constexpr (COLS > 1) {                   // a head's columns: 8 lanes apart, and 4
        const auto fold = [&](auto dpp) {
            constexpr int kCtrl = decltype(dpp)::value;
            const float r2 = dpp_f32<kCtrl>(r), l2 = dpp_f32<kCtrl>(l), top = fmaxf(r, r2);
            const float base = top == -INFINITY ? 0.0f : top;
            const float w1 = exp2_fast(r - base), w2 = exp2_fast(r2 - base);
            r = top;
            l = l * w1 + l2 * w2;
#pragma unroll
            for (int k = 0; k < 8 * NB; ++k) {
                const float x = o[k >> 3][(k >> 2) & 1][k & 3];
                o[k >> 3][(k >> 2) & 1][k & 3] = x * w1 + dpp_f32<kCtrl>(x) * w2;
            }
        };
        fold(std::integral_constant<int, kDppRowRor8>{});
        if constexpr (COLS == 4) fold(std::integral_constant<int, kDppRowRor4>{});
    }
#pragma unroll
    for (int step = 2; step > 0; step >>= 1) {
        float *slot = join + (wave & (step - 1)) * (8 * NB + 2) * 64 + lane;
        if (step == 1) __syncthreads();
        if (wave >= step && wave < 2 * step) {
            slot[0] = r;
            slot[64] = l;
#pragma unroll
            for (int k = 0; k < 8 * NB; ++k) slot[(2 + k) * 64] = o[k >> 3][(k >> 2) & 1][k & 3];
        }
        __syncthreads();
        if (wave < step) {
            const float r2 = slot[0], l2 = slot[64], top = fmaxf(r, r2);
            const float base = top == -INFINITY ? 0.0f : top;
            const float w1 = exp2_fast(r - base), w2 = exp2_fast(r2 - base);
            r = top;
            l = l * w1 + l2 * w2;
#pragma unroll
            for (int k = 0; k < 8 * NB; ++k)
                o[k >> 3][(k >> 2) & 1][k & 3] = o[k >> 3][(k >> 2) & 1][k & 3] * w1 + slot[(2 + k) * 64] * w2;
        }
    }
    if (wave != 0 || !live || c != 0) return;
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
        if (g == 0) a.part_ml[head * a.splits + split] = make_float2(r, l);
        return;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int64_t row = b * a.os.token + hq * a.os.head;
#pragma unroll
    for (int blk = 0; blk < NB; ++blk)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x[2] = {o[blk][0][i] * inv, o[blk][1][i] * inv};
            store2<RT>(a.out, row + blk * 32 + 2 * (4 * g + i), x);
        }
    if (a.lse && g == 0) a.lse[head] = log_sum(r, l);
}

// The first launch of a format, for the query heads of a key head that decide the columns.
template <int F, int NB, int COLS>
hipError_t launch_chunks_c(int rt, AttnArgs a, int64_t B, hipStream_t st) {
    const int group = a.Hq / a.c.heads, tiles = COLS > 1 ? 1 : (group + kHeadTile - 1) / kHeadTile;
    void *args[] = {(void *)&a};
    const void *k = rt == R_F32   ? (const void *)k_attn_chunk<F, NB, R_F32, COLS>
                    : rt == R_F16 ? (const void *)k_attn_chunk<F, NB, R_F16, COLS>
                                  : (const void *)k_attn_chunk<F, NB, R_BF16, COLS>;
    return hipLaunchKernel(k, dim3((unsigned)a.splits, (unsigned)(a.c.heads * tiles), (unsigned)B),
                           dim3(kAttnThreads), args, 0, st);
}

template <int F, int NB>
hipError_t launch_chunks_f(int rt, AttnArgs a, int64_t B, hipStream_t st) {
    if constexpr (F != KV_F16) {
        const int cols = attn_cols(a.Hq / a.c.heads);
        if constexpr (kFourColumns<F, NB>)
            if (cols == 4) return launch_chunks_c<F, NB, 4>(rt, a, B, st);
        if (cols >= 2) return launch_chunks_c<F, NB, 2>(rt, a, B, st);
    }
    return launch_chunks_c<F, NB, 1>(rt, a, B, st);
}

template <int F>
hipError_t launch_chunks(int nb, int rt, const AttnArgs &a, int64_t B, hipStream_t st) {
    switch (nb) {
        case 2: return launch_chunks_f<F, 2>(rt, a, B, st);
        case 3: return launch_chunks_f<F, 3>(rt, a, B, st);
        case 4: return launch_chunks_f<F, 4>(rt, a, B, st);
        case 6: return launch_chunks_f<F, 6>(rt, a, B, st);
        case 8: return launch_chunks_f<F, 8>(rt, a, B, st);
    }
    return hipErrorInvalidValue;
}

}  // namespace qmm
