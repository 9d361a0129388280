// Experts' products of up to 32 rows a tile, 32-value weight formats:
//   y[m][n] = sum_b dx[m,b] dw[n,b] I_b[m,n]   (+ dx sx m_w for the _1 formats)
//
// A stage is eight blocks.  Lane half h feeds codes 16 h .. 16 h + 15 of a block: of
// 4- and 5-bit weights all low or all high nibbles.  Codes, bias and fold are those
// of the prefill matmul: 4-bit codes enter as 16 (q - 8), 5-bit ones as 8 (q - 16),
// the MFMA starts from 0x4B400000, so that its result read as f32 is
// 1.5 2^23 + S I, and each block costs two FMAs an output, for the 8 FR rows that
// the tile has.
#include "experts_stream.h"

namespace qmm {

struct __attribute__((packed, aligned(4))) Dwords4 { uint32_t w[4]; };

// Rows of whole stages, of any number of blocks above a stage's, of an odd number (of
// formats of 2 mod 4 bytes a block).
enum Rows { WHOLE, PART, ODD_ROWS };

template <int F, Rows R>
struct Blocks32 {
    static constexpr bool TAIL = R != WHOLE, ODD = R == ODD_ROWS, XLEAD = ODD, WLEAD = ODD;
    static constexpr int MORE = 1;                            // with a lead, the chunk after the part's last is moved on
    static constexpr bool HALF = false;                      // many rows take the prefill matmul's tiles
    static constexpr bool Q8 = F == F_Q8_0, Q5 = F == F_Q5_0 || F == F_Q5_1, MIN = F == F_Q4_1 || F == F_Q5_1;
    static constexpr int WB = F == F_Q4_0 ? kQ40Bytes : Q8 ? kQ80Bytes : F == F_Q4_1 ? kQ41Bytes
                              : F == F_Q5_0 ? kQ50Bytes : kQ51Bytes;
    static constexpr int BLOCKS = 8, XBYTES = 8 * kQ80Bytes, WBYTES = 8 * WB;
    static_assert(!ODD || (WB % 4 == 2 && !MIN), "weights and activations both lie off the dword grid");
    // chunks of an LDS row, those of the lead among them: an odd number, so that 16 rows lie in distinct banks
    static constexpr int XC = (XBYTES / 16 + ODD) | 1, WC = (WBYTES / 16 + ODD) | 1;
    static constexpr float OUT_SCALE = Q8 ? 1.0f : Q5 ? 0.125f : 0.0625f;
    // the chunk after a row's last ends with it; with a lead the copy moves it on to the dword that holds its last bytes,
    // which is then at byte END + 12 of the LDS row
    static constexpr int xchunk(int c) { return c < XBYTES / 16 ? 16 * c : XBYTES - 16; }
    static constexpr int wchunk(int c) { return c < WBYTES / 16 ? 16 * c : WBYTES - 16; }
    // a wave's f32 dx (and dx * code sum) of a stage: [block][row]
    template <int ROWS, int WPG> using Lds = es::Layout<ROWS, WPG, XC, WC, 8 * ROWS * 4 * (MIN ? 2 : 1)>;

    template <int ROWS, int FR>
    struct Step {
        const uint8_t *ws;                                 // the lane's weight row
        float *dxw;
        int lane, lh;
        uint32_t up;                                       // the nibbles that the lane half feeds, into the high halves
        uint32_t hi_nibbles = 0xF0F0F0F0u, sign = 0x80808080u;
        int wodd = 0, xodd = 0, xlead = 0;                 // ODD: rows' numbers odd (xodd: bit i of row 8i + lane / 8)
        v16i bias;
        static constexpr int NV = Q8 ? 36 : WBYTES / 4;
        uint32_t v[NV];
        static_assert(ROWS <= 32 && FR <= 4, "one MFMA tile of 32 rows");
        float acc[16];

        __device__ __forceinline__ Step(const uint8_t *w, uint8_t *own, int l)
            : ws(w), dxw(reinterpret_cast<float *>(own)), lane(l), lh(l >> 5), up(lh ? 0u : 4u) {
#pragma unroll
            for (int r = 0; r < 16; ++r) bias[r] = 0x4B400000;
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[r] = 0.0f;
            asm volatile("" : "+v"(bias));                 // in vector registers for the whole loop
            asm volatile("" : "+v"(hi_nibbles), "+v"(sign));
        }

        // ODD: the lane's weight row's number, and the activation rows that it reads
        __device__ __forceinline__ void parities(int n, const int *src, int M) {
            wodd = n & 1;
#pragma unroll
            for (int i = 0; i < FR; ++i) xodd |= (src[min(8 * i + (lane >> 3), M - 1)] & 1) << i;
            xlead = src[min(lane & (ROWS - 1), M - 1)] & 1;
        }
        // the 16 codes of block b of a Q8_0 row that the lane's half feeds: the dwords that hold them, and out of these;
        // lead: the bytes before the row's stage (0 or 2, ODD only)
        struct Raw { uint32_t w[5]; };
        __device__ __forceinline__ Raw raw16(const uint8_t *row, int b, int lead) const {
            if constexpr (ODD) {
                const int at = 34 * b + 2 + lead + 16 * lh;
                const uint8_t *p = row + (at & ~3);
                const Dwords4 d = *reinterpret_cast<const Dwords4 *>(p);
                // past byte XBYTES: the dword of the chunk that was moved
                return {{d.w[0], d.w[1], d.w[2], d.w[3],
                         *reinterpret_cast<const uint32_t *>(b == 7 && lh ? row + XBYTES + 12 : p + 16)}};
            } else {
                const uint8_t *p = row + kQ80Bytes * b + 16 * lh + 2 * (b & 1);
                const Dwords4 d = *reinterpret_cast<const Dwords4 *>(p);
                return {{d.w[0], d.w[1], d.w[2], d.w[3], b & 1 ? 0u : *reinterpret_cast<const uint32_t *>(p + 16)}};
            }
        }
        static __device__ __forceinline__ v4i codes16(const Raw &r, int b, int lead) {
            v4i c;
            const uint32_t shift = (uint32_t)(2 * b + 2 + lead) & 3u;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                c[k] = (int)(ODD ? align_bytes(r.w[k + 1], r.w[k], shift)
                                 : b & 1 ? r.w[k] : align_bytes(r.w[k + 1], r.w[k], 2));
            return c;
        }
        // Q8_0: the codes that the lane's half feeds and the scales; else the row's stage
        __device__ __forceinline__ void empty(int first) {
            const int lead = ODD ? 2 * ((wodd + first) & 1) : 0;
            if constexpr (Q8) {
#pragma unroll
                for (int b = 0; b < 8; ++b) {
                    const v4i c = codes16(raw16(ws, b, lead), b, lead);
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[4 * b + k] = (uint32_t)c[k];
                    const uint32_t d = *reinterpret_cast<const uint16_t *>(ws + kQ80Bytes * b + lead);
                    v[32 + b / 2] = b & 1 ? v[32 + b / 2] | d << 16 : d;
                }
            } else {
#pragma unroll
                for (int c = 0; c < WBYTES / 16; ++c) {
                    const uint4 q = *reinterpret_cast<const uint4 *>(ws + 16 * c);
                    v[4 * c] = q.x, v[4 * c + 1] = q.y, v[4 * c + 2] = q.z, v[4 * c + 3] = q.w;
                }
                if constexpr (ODD) {
                    const uint32_t last = *reinterpret_cast<const uint32_t *>(ws + WBYTES + 12);
#pragma unroll
                    for (int k = 0; k < NV; ++k) v[k] = align_bytes(k + 1 < NV ? v[k + 1] : last, v[k], (uint32_t)lead);
                }
            }
#pragma unroll
            for (int k = 0; k < NV; ++k) asm volatile("" : "+v"(v[k]));     // read now
        }
        // the dword at byte o of the weight row's stage
        __device__ __forceinline__ uint32_t at(int o) const {
            return o % 4 == 0 ? v[o / 4] : align_bytes(v[o / 4 + 1], v[o / 4], 2);
        }
        __device__ __forceinline__ v4i operand(int b) const {
            v4i c;
            if constexpr (Q8) {
#pragma unroll
                for (int k = 0; k < 4; ++k) c[k] = (int)v[4 * b + k];
            } else {
                const int o = WB * b, qs = o + (F == F_Q4_0 ? 2 : F == F_Q4_1 ? 4 : F == F_Q5_0 ? 6 : 8);
                uint32_t nq = 0;
                if constexpr (Q5) nq = ~(at(o + (F == F_Q5_0 ? 2 : 4)) >> (16 * lh));
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t q = at(qs + 4 * k) << up;
                    if constexpr (Q5)
                        c[k] = (int)(((q >> 1) & 0x78787878u) |
                                     ((bits_to_bytes((nq >> (4 * k)) & 15u) << 7) & 0x80808080u));
                    else
                        c[k] = (int)((q & hi_nibbles) ^ sign);
                }
            }
            return c;
        }
        __device__ __forceinline__ float scale(int b) const {
            float d = f16_bits_to_f32(Q8 ? v[32 + b / 2] >> (16 * (b & 1)) : v[WB * b / 4] >> (8 * (WB * b % 4)));
            asm volatile("" : "+v"(d));                    // an f16 operand would halve the fold's rate
            return d;
        }
        // first: the stage's first block; skip: blocks of it that were in the stage before
        __device__ __forceinline__ void work(const uint8_t *xs, int first, int skip) {
            const int xrow = lane & (ROWS - 1);                                  // rows past the tile's LDS rows repeat them
            const uint8_t *const xl = xs + 16 * XC * xrow;
            const int lead = ODD ? 2 * ((xlead + first) & 1) : 0;
            // the wave's dx as f32: lane l takes block l % 8 of rows l / 8, l / 8 + 8, ..
#pragma unroll
            for (int i = 0; i < FR; ++i) {
                const int row = 8 * i + (lane >> 3), b = lane & 7;
                const int off = ODD ? 2 * (((xodd >> i) + first) & 1) : 0;
                const uint8_t *p = xs + 16 * XC * row + kQ80Bytes * b + off;
                const float d = f16_bits_to_f32(*reinterpret_cast<const uint16_t *>(p));
                // blocks of the stage before count as zeros here (their NaN and infinities are in the sums already)
                dxw[ROWS * b + row] = TAIL && b < skip ? 0.0f : d;
                if constexpr (MIN) {
                    // the code sum, from the dwords that hold the block: its first or last two bytes are no codes
                    const uint32_t *q = reinterpret_cast<const uint32_t *>(p - 2 * (b & 1));
                    int sum = dot4((int)q[0], b & 1 ? 0 : 0x01010000, 0);
#pragma unroll
                    for (int k = 1; k < 8; ++k) sum = dot4((int)q[k], 0x01010101, sum);
                    sum = dot4((int)q[8], b & 1 ? 0x01010101 : 0x00000101, sum);
                    dxw[8 * ROWS + ROWS * b + row] = TAIL && b < skip ? 0.0f : d * (float)sum;
                }
            }
            // Rows' codes are read two blocks ahead of their fold and dx one block ahead, and the next block's product is
            // under way while one is folded: a wave that is alone on its SIMD waits for none of them.
            struct Dx { float4 x[4]; };
            auto dx = [&](int b) {
                Dx q;
#pragma unroll
                for (int i = 0; i < FR; ++i) q.x[i] = *reinterpret_cast<const float4 *>(dxw + ROWS * b + 8 * i + 4 * lh);
                return q;
            };
            Raw raw = raw16(xl, 0, lead);
            v4i x = codes16(raw, 0, lead), w = operand(0);
            v16i d = __builtin_amdgcn_mfma_i32_32x32x32_i8(x, w, bias, 0, 0, 0);
            raw = raw16(xl, 1, lead);
            Dx x0 = dx(0), x1 = x0;
#pragma unroll
            for (int b = 0; b < 8; ++b) {
                v16i next = bias;
                if (b + 1 < 8) {
                    x = codes16(raw, b + 1, lead);
                    if (b + 2 < 8) raw = raw16(xl, b + 2, lead);
                    x1 = dx(b + 1);
                    w = operand(b + 1);
                    next = __builtin_amdgcn_mfma_i32_32x32x32_i8(x, w, bias, 0, 0, 0);
                }
                __builtin_amdgcn_sched_barrier(0);
                const float dw = scale(b), nb = dw * -es::kBias;
                float v0[16];
#pragma unroll
                for (int r = 0; r < 4 * FR; ++r) {
                    const int e = d[r];
                    v0[r] = fmaf(__int_as_float(e), dw, nb);
                }
#pragma unroll
                for (int i = 0; i < FR; ++i) {
                    const float4 q = x0.x[i];
                    float *a = acc + 4 * i;
                    a[0] = fmaf(v0[4 * i], q.x, a[0]);
                    a[1] = fmaf(v0[4 * i + 1], q.y, a[1]);
                    a[2] = fmaf(v0[4 * i + 2], q.z, a[2]);
                    a[3] = fmaf(v0[4 * i + 3], q.w, a[3]);
                }
                __builtin_amdgcn_sched_barrier(0);
                d = next;
                x0 = x1;
                if constexpr (MIN) {
                    // the offset term of blocks b - 1 and b: (dx sx)(m) (2^7 d + m / S)(n), an outer product a block, K = block
                    if (b & 1) {
                        const uint32_t dm = lh ? v[WB * b / 4] : v[WB * (b - 1) / 4];
                        const float c = fmaf(f16_bits_to_f32(dm), 128.0f, f16_bits_to_f32(dm >> 16) * (1.0f / OUT_SCALE));
                        v16f s;
#pragma unroll
                        for (int r = 0; r < 16; ++r) s[r] = acc[r];
                        const float m = dxw[8 * ROWS + ROWS * (b - 1 + lh) + xrow];
                        s = __builtin_amdgcn_mfma_f32_32x32x2f32(m, c, s, 0, 0, 0);
#pragma unroll
                        for (int r = 0; r < 16; ++r) acc[r] = s[r];
                    }
                }
            }
        }
    };
};

// Which rows take which way, of those that are no whole number of stages:
//   * rows of an odd number of blocks, where every other weight row too then lies off
//     the dword grid, on which the two-block stages of the prefill tiles copy slowly
//     (us, those / ODD_ROWS: 128 experts of 1536 x 1056, 64 tokens Q4_0 51 / 33, Q8_0
//     69 / 54, Q5_0 51 / 39; 3 experts of 2728 x 4960, 8 tokens Q5_0 36 / 16), not
//     where tiles of 32 rows leave less workgroups than would hide the last stage's
//     blocks that count twice (3 experts of 2336 x 1696, 118 tokens Q4_0 16 / 19, Q8_0
//     18 / 30);
//   * the others where there are so few workgroups that K is cut (PART);
//   * else the prefill tiles: on the grid the part of a stage costs what the longer
//     stages give (81 experts of 592 x 704, 622 tokens: Q4_0 16.4 / 16.7, Q8_0 19.7 /
//     21.6).
static bool odd_rows(int fmt, const ExpertArgs &a) {
    return (fmt == F_Q4_0 || fmt == F_Q8_0 || fmt == F_Q5_0) && a.nb % 2 && a.nb > 8 &&
           (a.rows <= kFewRows || stream_blocks(a) >= kEnoughBlocks);
}

bool experts_stream_32_suits(int fmt, const ExpertArgs &a) {
    return a.nb % 8 == 0 || odd_rows(fmt, a) || (a.nb > 8 && stream_blocks(a) < kFewBlocks);
}

template <int F>
static hipError_t pick(const ExpertArgs &a, hipStream_t st) {
    if (a.nb < 8) return hipErrorInvalidValue;             // less than a stage
    if (a.nb % 8 == 0) return experts_stream<Blocks32<F, WHOLE>>(a, st);
    if constexpr (F == F_Q4_0 || F == F_Q8_0 || F == F_Q5_0)
        if (odd_rows(F, a))
            return a.rows <= kFewRows ? pick_stream<Blocks32<F, ODD_ROWS>, kFewRows>(a, st)
                                      : launch_stream<Blocks32<F, ODD_ROWS>, kNarrowRows, 1, 4>(a, st);
    return a.rows <= kFewRows ? launch_stream<Blocks32<F, PART>, kFewRows, 4, 2>(a, st)
                              : launch_stream<Blocks32<F, PART>, kNarrowRows, 4, 2>(a, st);
}

hipError_t launch_experts_stream_32(int fmt, const ExpertArgs &a, hipStream_t st) {
    switch (fmt) {
        case F_Q4_0: return pick<F_Q4_0>(a, st);
        case F_Q8_0: return pick<F_Q8_0>(a, st);
        case F_Q4_1: return pick<F_Q4_1>(a, st);
        case F_Q5_0: return pick<F_Q5_0>(a, st);
        case F_Q5_1: return pick<F_Q5_1>(a, st);
    }
    return hipErrorInvalidValue;
}

}  // namespace qmm
