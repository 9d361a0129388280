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

template <int F>
struct Blocks32 {
    static constexpr bool Q8 = F == F_Q8_0, Q5 = F == F_Q5_0 || F == F_Q5_1, MIN = F == F_Q4_1 || F == F_Q5_1;
    static constexpr int WB = F == F_Q4_0 ? kQ40Bytes : Q8 ? kQ80Bytes : F == F_Q4_1 ? kQ41Bytes
                              : F == F_Q5_0 ? kQ50Bytes : kQ51Bytes;
    static constexpr int BLOCKS = 8, XBYTES = 8 * kQ80Bytes, WBYTES = 8 * WB;
    static constexpr int XC = XBYTES / 16;                    // 17 chunks: 16 rows lie in distinct banks
    static constexpr int WC = WBYTES / 16 | 1;                // odd, for the same reason: a 10- or 12-chunk row has a spare
    static constexpr float OUT_SCALE = Q8 ? 1.0f : Q5 ? 0.125f : 0.0625f;
    static constexpr int xchunk(int c) { return 16 * c; }
    static constexpr int wchunk(int c) { return 16 * (c < WBYTES / 16 ? c : c - 1); }
    // a wave's f32 dx (and dx * code sum) of a stage: [block][row]
    template <int ROWS, int WPG> using Lds = es::Layout<ROWS, WPG, XC, WC, 8 * ROWS * 4 * (MIN ? 2 : 1)>;

    template <int ROWS, int FR>
    struct Step {
        const uint8_t *ws;                                 // the lane's weight row
        float *dxw;
        int lane, lh;
        uint32_t up;                                       // the nibbles that the lane half feeds, into the high halves
        uint32_t hi_nibbles = 0xF0F0F0F0u, sign = 0x80808080u;
        v16i bias;
        static constexpr int NV = Q8 ? 36 : WBYTES / 4;
        uint32_t v[NV];
        float acc[16];

        __device__ __forceinline__ Step(const uint8_t *w, uint8_t *own, int l)
            : ws(w), dxw(reinterpret_cast<float *>(own)), lane(l), lh(l >> 5), up(lh ? 0u : 4u) {
#pragma unroll
            for (int r = 0; r < 16; ++r) bias[r] = 0x4B400000, acc[r] = 0.0f;
            asm volatile("" : "+v"(bias));                 // in vector registers for the whole loop
            asm volatile("" : "+v"(hi_nibbles), "+v"(sign));
        }

        // the 16 codes of block b of a Q8_0 row that the lane's half feeds: the dwords that hold them, and out of these
        struct Raw { uint32_t w[5]; };
        __device__ __forceinline__ Raw raw16(const uint8_t *row, int b) const {
            const uint8_t *p = row + kQ80Bytes * b + 16 * lh + 2 * (b & 1);
            const Dwords4 d = *reinterpret_cast<const Dwords4 *>(p);
            return {{d.w[0], d.w[1], d.w[2], d.w[3], b & 1 ? 0u : *reinterpret_cast<const uint32_t *>(p + 16)}};
        }
        static __device__ __forceinline__ v4i codes16(const Raw &r, int b) {
            v4i c;
#pragma unroll
            for (int k = 0; k < 4; ++k) c[k] = (int)(b & 1 ? r.w[k] : align_bytes(r.w[k + 1], r.w[k], 2));
            return c;
        }
        // Q8_0: the codes that the lane's half feeds and the scales; else the row's stage
        __device__ __forceinline__ void empty() {
            if constexpr (Q8) {
#pragma unroll
                for (int b = 0; b < 8; ++b) {
                    const v4i c = codes16(raw16(ws, b), b);
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[4 * b + k] = (uint32_t)c[k];
                    const uint32_t d = *reinterpret_cast<const uint16_t *>(ws + kQ80Bytes * b);
                    v[32 + b / 2] = b & 1 ? v[32 + b / 2] | d << 16 : d;
                }
            } else {
#pragma unroll
                for (int c = 0; c < WBYTES / 16; ++c) {
                    const uint4 q = *reinterpret_cast<const uint4 *>(ws + 16 * c);
                    v[4 * c] = q.x, v[4 * c + 1] = q.y, v[4 * c + 2] = q.z, v[4 * c + 3] = q.w;
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
        __device__ __forceinline__ void work(const uint8_t *xs) {
            const int xi = lane & (ROWS - 1);              // rows past the tile's LDS rows repeat them
            const uint8_t *xl = xs + XBYTES * (ROWS < 32 ? xi : lane & 31);
            const int xrow = ROWS < 32 ? xi : lane & 31;
            // the wave's dx as f32: lane l takes block l % 8 of rows l / 8, l / 8 + 8, ..
#pragma unroll
            for (int i = 0; i < FR; ++i) {
                const int row = 8 * i + (lane >> 3), b = lane & 7;
                const uint8_t *p = xs + XBYTES * row + kQ80Bytes * b;
                const float d = f16_bits_to_f32(*reinterpret_cast<const uint16_t *>(p));
                dxw[ROWS * b + row] = d;
                if constexpr (MIN) {
                    // the code sum, from the dwords that hold the block: its first or last two bytes are no codes
                    const uint32_t *q = reinterpret_cast<const uint32_t *>(p - 2 * (b & 1));
                    int sum = dot4((int)q[0], b & 1 ? 0 : 0x01010000, 0);
#pragma unroll
                    for (int k = 1; k < 8; ++k) sum = dot4((int)q[k], 0x01010101, sum);
                    sum = dot4((int)q[8], b & 1 ? 0x01010101 : 0x00000101, sum);
                    dxw[8 * ROWS + ROWS * b + row] = d * (float)sum;
                }
            }
            // Rows' codes are read two blocks ahead of their fold and dx one block ahead, and the next block's product
            // is under way while a block is folded: a wave that is alone on its SIMD waits for none of them.
            struct Dx { float4 x[FR]; };
            auto dx = [&](int b) {
                Dx q;
#pragma unroll
                for (int i = 0; i < FR; ++i)
                    q.x[i] = *reinterpret_cast<const float4 *>(dxw + ROWS * b + 8 * i + 4 * lh);
                return q;
            };
            Raw raw = raw16(xl, 0);
            v4i x = codes16(raw, 0);
            v16i d = __builtin_amdgcn_mfma_i32_32x32x32_i8(x, operand(0), bias, 0, 0, 0);
            raw = raw16(xl, 1);
            Dx x0 = dx(0), x1 = x0;
#pragma unroll
            for (int b = 0; b < 8; ++b) {
                v16i next = bias;
                if (b < 7) {
                    x = codes16(raw, b + 1);
                    if (b < 6) raw = raw16(xl, b + 2);
                    x1 = dx(b + 1);
                    next = __builtin_amdgcn_mfma_i32_32x32x32_i8(x, operand(b + 1), bias, 0, 0, 0);
                }
                __builtin_amdgcn_sched_barrier(0);
                const float dw = scale(b), nb = dw * -es::kBias;
                float u[4 * FR];
#pragma unroll
                for (int r = 0; r < 4 * FR; ++r) {
                    const int e = d[r];
                    u[r] = fmaf(__int_as_float(e), dw, nb);
                }
#pragma unroll
                for (int i = 0; i < FR; ++i) {
                    const float4 q = x0.x[i];
                    acc[4 * i] = fmaf(u[4 * i], q.x, acc[4 * i]);
                    acc[4 * i + 1] = fmaf(u[4 * i + 1], q.y, acc[4 * i + 1]);
                    acc[4 * i + 2] = fmaf(u[4 * i + 2], q.z, acc[4 * i + 2]);
                    acc[4 * i + 3] = fmaf(u[4 * i + 3], q.w, acc[4 * i + 3]);
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
                        s = __builtin_amdgcn_mfma_f32_32x32x2f32(dxw[8 * ROWS + ROWS * (b - 1 + lh) + xrow], c, s, 0, 0, 0);
#pragma unroll
                        for (int r = 0; r < 16; ++r) acc[r] = s[r];
                    }
                }
            }
        }
    };
};

hipError_t launch_experts_stream_32(int fmt, const ExpertArgs &a, hipStream_t st) {
    switch (fmt) {
        case F_Q4_0: return experts_stream<Blocks32<F_Q4_0>>(a, st);
        case F_Q8_0: return experts_stream<Blocks32<F_Q8_0>>(a, st);
        case F_Q4_1: return experts_stream<Blocks32<F_Q4_1>>(a, st);
        case F_Q5_0: return experts_stream<Blocks32<F_Q5_0>>(a, st);
        case F_Q5_1: return experts_stream<Blocks32<F_Q5_1>>(a, st);
    }
    return hipErrorInvalidValue;
}

}  // namespace qmm
