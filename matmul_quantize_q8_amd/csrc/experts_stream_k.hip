// Experts' products of up to 64 rows a tile, K-quant weight formats.
//
// A stage is one super-block; the products are those of the K-quant prefill:
//   Q2_K  d8 (d V - dmin Mn), V = sum sc I on int8 MFMA with the group scales folded
//         into the codes (sc q <= 45);
//   Q4_K  the same with V = 8 A1 + A2, two contractions with the scale's two halves
//         (sc = 8 sh + sl, sh q and sl q <= 105);
//   Q6_K  d8 d (V - Mn), V = sum_g sc_g I_g in int32, I_g of a 16-deep MFMA a group on
//         the unsigned codes, Mn = sum 32 sc_g bsum_g;
// Mn on one f16 MFMA over the activation's block sums (|bsum| <= 2048 and the
// factors are exact in f16), one fold of the 8 FR rows that the tile has a super-block.
#include "experts_stream.h"

namespace qmm {

typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

template <int F>
struct SuperBlocks {
    static constexpr int WBYTES = F == F_Q2_K ? kQ2KBytes : F == F_Q4_K ? kQ4KBytes : kQ6KBytes;
    static constexpr int BLOCKS = 1, XBYTES = kQ8KBytes;
    static constexpr bool HALF = true;
    static constexpr bool TAIL = false, XLEAD = false, WLEAD = F == F_Q6_K;         // the others' bytes are whole dwords
    static constexpr int MORE = 2;                            // no chunk after a part's last
    // activation row: the codes in 16 chunks, the block sums in two, the chunk that starts with d
    static constexpr int XC = 19;
    static constexpr int xchunk(int c) { return c < 16 ? 4 + 16 * c : c == 16 ? 260 : c == 17 ? 276 : 0; }
    // weight row: chunks in order, the last one moved back to end with the super-block; an odd count, so that rows
    // start in many banks
    static constexpr int FULL = WBYTES / 16, WC = F == F_Q2_K ? 7 : F == F_Q4_K ? 9 : 15;
    // (Q6_K's with a lead: the dword that holds its last two bytes is then at byte 16 FULL + 12)
    static constexpr int wchunk(int c) { return c < FULL ? 16 * c : WLEAD ? (WBYTES + 3) / 4 * 4 - 16 : WBYTES - 16; }
    static constexpr float OUT_SCALE = 1.0f;
    // a wave's f32 d8 of a stage's rows
    template <int ROWS, int WPG> using Lds = es::Layout<ROWS, WPG, XC, WC, 4 * ROWS>;
    static constexpr int XROW = 16 * XC;

    template <int ROWS, int FR>
    struct Step {
        const uint8_t *ws;                                 // the lane's weight row
        float *d8w;
        int lane, lh, wodd = 0;                            // wodd: Q6_K, of the weight row's first super-block
        v16i bias;
        // scales (with d and dmin), then the code bytes that the lane's half feeds
        static constexpr int NV = F == F_Q2_K ? 13 : F == F_Q4_K ? 20 : 29;
        uint32_t v[NV];
        static constexpr int NT = FR > 4 ? 2 : 1;          // MFMA tiles of 32 rows
        float acc[16 * NT];

        __device__ __forceinline__ Step(const uint8_t *w, uint8_t *own, int l)
            : ws(w), d8w(reinterpret_cast<float *>(own)), lane(l), lh(l >> 5) {
#pragma unroll
            for (int r = 0; r < 16; ++r) bias[r] = 0x4B400000;
#pragma unroll
            for (int r = 0; r < 16 * NT; ++r) acc[r] = 0.0f;
        }
        static __device__ __forceinline__ uint4 rd16(const uint8_t *p) { return *reinterpret_cast<const uint4 *>(p); }
        static __device__ __forceinline__ float half_lo(uint32_t x) { return f16_bits_to_f32(x); }

        __device__ __forceinline__ void parities(int n, const int *, int) { wodd = n & 1; }
        // eight bytes at byte o of a super-block behind its lead
        __device__ __forceinline__ uint2 rd8(int o, uint32_t lead) const {
            const uint2 q = *reinterpret_cast<const uint2 *>(ws + o);
            const uint32_t e = *reinterpret_cast<const uint32_t *>(ws + o + 8);
            return make_uint2(align_bytes(q.y, q.x, lead), align_bytes(e, q.y, lead));
        }

        __device__ __forceinline__ void empty(int first) {
            if constexpr (F == F_Q6_K) {
                // codes of group 8hh + 2k + gg, values l = 16gg + 8lh .. + 7: eight bytes of ql at 64hh + 16gg + 8lh (k
                // even) and 32 on (odd), of qh at 128 + 32hh + 16gg + 8lh; pair p = 2hh + gg
                const uint32_t lead = 2u * (uint32_t)((wodd + first) & 1);
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const int hh = p >> 1, gg = p & 1;
                    const uint2 qa = rd8(64 * hh + 16 * gg + 8 * lh, lead);
                    const uint2 qb = rd8(64 * hh + 32 + 16 * gg + 8 * lh, lead);
                    const uint2 qh = rd8(128 + 32 * hh + 16 * gg + 8 * lh, lead);
                    v[6 * p] = qa.x, v[6 * p + 1] = qa.y, v[6 * p + 2] = qb.x, v[6 * p + 3] = qb.y;
                    v[6 * p + 4] = qh.x, v[6 * p + 5] = qh.y;
                }
                const uint4 s = rd16(ws + 192);
                const uint32_t end = *reinterpret_cast<const uint32_t *>(ws + 16 * FULL + 12);     // behind a lead two scales, d
                v[24] = align_bytes(s.y, s.x, lead), v[25] = align_bytes(s.z, s.y, lead);
                v[26] = align_bytes(s.w, s.z, lead), v[27] = align_bytes(end, s.w, lead);
                v[28] = end >> (8 * lead);
            } else {
#pragma unroll
                for (int c = 0; c < NV / 4; ++c) {         // the head, then half of every 32 bytes of codes
                    const uint4 q = rd16(ws + (c == 0 ? 0 : 32 * c - 16 + 16 * lh));
                    v[4 * c] = q.x, v[4 * c + 1] = q.y, v[4 * c + 2] = q.z, v[4 * c + 3] = q.w;
                }
                if constexpr (F == F_Q2_K) v[12] = *reinterpret_cast<const uint32_t *>(ws + 16 * FULL + 12);   // d, dmin end the super-block
            }
#pragma unroll
            for (uint32_t &x : v) asm volatile("" : "+v"(x));      // read now
        }
        // Mn of the tile's rows: the activation's 16 block sums against eight factors a lane half
        __device__ __forceinline__ v16f sums(const uint8_t *xl, const v8h &b) const {
            const uint4 u = rd16(xl + 256 + 16 * lh);
            const uint32_t s[4] = {u.x, u.y, u.z, u.w};
            v8h x;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[2 * e] = (_Float16)(int)(int16_t)(s[e] & 0xffffu);
                x[2 * e + 1] = (_Float16)(int)(int16_t)(s[e] >> 16);
            }
            const v16f z = {};
            return __builtin_amdgcn_mfma_f32_32x32x16_f16(x, b, z, 0, 0, 0);
        }
        __device__ __forceinline__ int scale6(int g) const { return (int)(int8_t)(v[24 + g / 4] >> (8 * (g & 3))); }

        __device__ __forceinline__ void work(const uint8_t *xs, int, int) {
            const int xrow = lane & (ROWS < 32 ? ROWS - 1 : 31);               // rows past the tile's LDS rows repeat them
            auto xl = [&](int t) { return xs + XROW * (xrow + 32 * t); };      // of MFMA tile t
            if (lane < 8 * FR) d8w[lane] = *reinterpret_cast<const float *>(xs + XROW * lane + 288);
            auto codes = [&](int kt, int t) {
                const uint4 c = rd16(xl(t) + 32 * kt + 16 * lh);
                return v4i{(int)c.x, (int)c.y, (int)c.z, (int)c.w};
            };
            v16f mn[NT];
            if constexpr (F == F_Q2_K) {
                const uint32_t scl[4] = {v[0], v[1], v[2], v[3]};
                v16i V[NT];
#pragma unroll
                for (int t = 0; t < NT; ++t) V[t] = bias;
#pragma unroll
                for (int kt = 0; kt < 8; ++kt) {
                    // K-step kt: group 2kt + lh, codes by a table of 0, sc, 2sc, 3sc
                    const int sft = 2 * (kt & 3);
                    const uint32_t sw = scl[kt >> 1] >> (16 * (kt & 1));
                    const uint32_t sc = (lh ? sw >> 8 : sw) & 15u, tab = sc * 0x03020100u;
                    v4i b;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t q = v[4 + 4 * (kt >> 2) + e];
                        b[e] = (int)__builtin_amdgcn_perm(0u, tab, (q >> sft) & 0x03030303u);
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t) V[t] = __builtin_amdgcn_mfma_i32_32x32x32_i8(codes(kt, t), b, V[t], 0, 0, 0);
                }
                const uint32_t mlo = lh ? v[2] : v[0], mhi = lh ? v[3] : v[1];        // groups 8h .. 8h + 7
                v8h bm;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    bm[e] = (_Float16)(int)((mlo >> (8 * e + 4)) & 15u);
                    bm[4 + e] = (_Float16)(int)((mhi >> (8 * e + 4)) & 15u);
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) mn[t] = sums(xl(t), bm);
                const uint32_t dd = v[12];
                float dw = half_lo(dd), ndm = -half_lo(dd >> 16);
                asm volatile("" : "+v"(dw), "+v"(ndm));
                const float nbw = dw * -es::kBias;         // exact: 11 + 2 significant bits
                fold([&](int r) {
                    const int e = V[r / 16][r % 16];
                    return fmaf(ndm, mn[r / 16][r % 16], fmaf(__int_as_float(e), dw, nbw));
                });
            } else if constexpr (F == F_Q4_K) {
                int sc[8], mm[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t sh = 8u * (uint32_t)(j & 3);
                    const uint32_t A = (v[1] >> sh) & 0xffu, B = (v[2] >> sh) & 0xffu, C = (v[3] >> sh) & 0xffu;
                    sc[j] = (int)(j < 4 ? A & 63u : (C & 15u) | ((A >> 6) << 4));
                    mm[j] = (int)(j < 4 ? B & 63u : (C >> 4) | ((B >> 6) << 4));
                }
                v16i A1[NT] = {}, A2[NT] = {};
#pragma unroll
                for (int kt = 0; kt < 8; ++kt) {
                    const uint32_t sft = 4u * (uint32_t)(kt & 1);
                    const unsigned short sh = (unsigned short)(sc[kt] >> 3), sl = (unsigned short)(sc[kt] & 7);
                    const u16x2 sh2 = {sh, sh}, sl2 = {sl, sl};
                    v4i b1, b2;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t q = v[4 + 4 * (kt >> 1) + e];
                        const u16x2 nib = __builtin_bit_cast(u16x2, (q >> sft) & 0x0f0f0f0fu);
                        b1[e] = __builtin_bit_cast(int, nib * sh2);
                        b2[e] = __builtin_bit_cast(int, nib * sl2);
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const v4i x = codes(kt, t);
                        A1[t] = __builtin_amdgcn_mfma_i32_32x32x32_i8(x, b1, A1[t], 0, 0, 0);
                        A2[t] = __builtin_amdgcn_mfma_i32_32x32x32_i8(x, b2, A2[t], 0, 0, 0);
                    }
                }
                v8h bm;                                    // groups 8h .. 8h + 7: sub-blocks 4h .. 4h + 3, two groups each
#pragma unroll
                for (int e = 0; e < 8; ++e) bm[e] = (_Float16)(lh ? mm[4 + (e >> 1)] : mm[e >> 1]);
#pragma unroll
                for (int t = 0; t < NT; ++t) mn[t] = sums(xl(t), bm);
                float dw = half_lo(v[0]), ndm = -half_lo(v[0] >> 16);
                asm volatile("" : "+v"(dw), "+v"(ndm));
                fold([&](int r) {
                    const int t = r / 16, k = r % 16;
                    return fmaf(ndm, mn[t][k], (float)(A1[t][k] * 8 + A2[t][k]) * dw);
                });
            } else {
                int V[4 * FR];
#pragma unroll
                for (int r = 0; r < 4 * FR; ++r) V[r] = 0;
                auto group = [](int t) { return 8 * (t >> 3) + 2 * (t & 3) + ((t >> 2) & 1); };
                uint32_t b0 = 0, b1 = 0;
                auto product = [&](int u) {                // step u = NT (4 (2hh + gg) + k) + MFMA tile
                    const int s = u / NT, t = u % NT, p = s >> 2, k = s & 3;
                    if (t == 0) {
                        const uint32_t nsh = 4u * (uint32_t)(k >> 1), hsh = 2u * (uint32_t)k;
                        const uint32_t l0 = v[6 * p + 2 * (k & 1)], l1 = v[6 * p + 2 * (k & 1) + 1];
                        b0 = ((l0 >> nsh) & 0x0f0f0f0fu) | (((v[6 * p + 4] >> hsh) & 0x03030303u) << 4);
                        b1 = ((l1 >> nsh) & 0x0f0f0f0fu) | (((v[6 * p + 5] >> hsh) & 0x03030303u) << 4);
                    }
                    const uint2 x = *reinterpret_cast<const uint2 *>(xl(t) + 16 * group(s) + 8 * lh);
                    const v16i z = {};
                    return __builtin_amdgcn_mfma_i32_32x32x16_i8((long)((uint64_t)x.y << 32 | x.x),
                                                                 (long)((uint64_t)b1 << 32 | b0), z, 0, 0, 0);
                };
                v16i I = product(0);
#pragma unroll
                for (int u = 0; u < 16 * NT; ++u) {
                    v16i next = I;
                    if (u + 1 < 16 * NT) next = product(u + 1);            // in flight while this group's is used
                    const int sc = scale6(group(u / NT)), t = u % NT;
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        if (16 * t + r >= 4 * FR) break;
                        const int e = I[r];
                        V[16 * t + r] = __mul24(sc, e) + V[16 * t + r];
                        asm volatile("" : "+v"(V[16 * t + r]));
                    }
                    __builtin_amdgcn_sched_barrier(0);
                    I = next;
                }
                v8h bm;
#pragma unroll
                for (int e = 0; e < 8; ++e) bm[e] = (_Float16)(32 * (lh ? scale6(8 + e) : scale6(e)));
#pragma unroll
                for (int t = 0; t < NT; ++t) mn[t] = sums(xl(t), bm);
                float dw = half_lo(v[28]);
                asm volatile("" : "+v"(dw));
                const float ndw = -dw;
                fold([&](int r) { return fmaf(ndw, mn[r / 16][r % 16], (float)V[r] * dw); });
            }
        }
        // acc += d8 * value of each of the tile's rows
        template <class Fn>
        __device__ __forceinline__ void fold(Fn &&value) {
#pragma unroll
            for (int i = 0; i < FR; ++i) {
                const float4 d8 = *reinterpret_cast<const float4 *>(d8w + 8 * i + 4 * lh);
                acc[4 * i] = fmaf(value(4 * i), d8.x, acc[4 * i]);
                acc[4 * i + 1] = fmaf(value(4 * i + 1), d8.y, acc[4 * i + 1]);
                acc[4 * i + 2] = fmaf(value(4 * i + 2), d8.z, acc[4 * i + 2]);
                acc[4 * i + 3] = fmaf(value(4 * i + 3), d8.w, acc[4 * i + 3]);
            }
        }
    };
};

hipError_t launch_experts_stream_k(int fmt, const ExpertArgs &a, hipStream_t st) {
    switch (fmt) {
        case F_Q2_K: return experts_stream<SuperBlocks<F_Q2_K>>(a, st);
        case F_Q4_K: return experts_stream<SuperBlocks<F_Q4_K>>(a, st);
        case F_Q6_K: return experts_stream<SuperBlocks<F_Q6_K>>(a, st);
    }
    return hipErrorInvalidValue;
}

}  // namespace qmm
