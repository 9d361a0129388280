// Experts' products of up to 64 rows a tile on MFMA: what the 32-value formats
// (experts_stream_32.hip) and the K-quants (experts_stream_k.hip) share.  The K-quants'
// products of many rows are here too: two workgroups a compute unit cover one another's
// start, which one of the prefill matmul's 128 x 256 tiles a compute unit does not (64
// experts of 1536 x 2048, 512 rows each: Q2_K 244 us, those tiles 259; Q4_K 320 / 349;
// Q6_K 580 / 567, of 2048 x 768 319 / 348).
//
// Bound by the weight stream, where an expert has few rows: every weight byte is used
// for little work, so what counts is how many bytes are on their way.
//   * A stage is 256 values of every row: a weight row's part (84 bytes of Q2_K ..
//     272 of Q8_0) is copied in 16-byte chunks, consecutive lanes on consecutive
//     chunks, and one barrier, one wait and one chain of LDS reads serve all of it.
//     Stages of two blocks, as the prefill tiles of the 32-value formats have them,
//     leave a workgroup that is nearly alone on its compute unit waiting for that
//     chain (1.8 TB/s of Q8_0 weights, whatever the depth of its ring).
//   * A wave copies its own 32 weight rows into one LDS buffer, empties it into
//     registers at the start of a step and at once copies the next stage into it:
//     a stage is on its way during all of a step, at half the LDS of two buffers,
//     and several workgroups share a compute unit (128 experts of 1536 x 2048, 8 a
//     token: Q4_0, 16 tokens 32.9 -> 25.0 us, 64 tokens 54.7 -> 44.7; Q8_0, 64 tokens
//     117 -> 71.5, which is 5.1 TB/s of weights).  Only the activations, which the
//     waves share, have two buffers.
//   * Tiles of 16 rows where an expert has few: less LDS, less of the fold.
//
// A workgroup: a tile's rows x 32 WPG weight rows, wave w of a group alone on weight
// rows 32 w .., one 32 x 32 MFMA tile a step of K (two, where there are rows 32 .. 63);
// G groups of WPG waves, each on its part of K, which join in LDS in a fixed order.
#pragma once

#include <type_traits>
#include <utility>

#include "moe.h"

namespace qmm {

namespace es {
constexpr float kBias = 12582912.0f;               // 1.5 * 2^23, bit pattern 0x4B400000

// LDS of a K group of WPG waves, for an activation row of XC chunks and a weight row
// of WC chunks a stage; XD bytes of a wave's own.
template <int ROWS, int WPG, int XC, int WC, int XD> struct Layout {
    static constexpr int WL = (32 * WC + kWave - 1) / kWave;  // wave loads of a wave's 32 weight rows
    static constexpr int XL = (ROWS * XC + kWave - 1) / kWave;       // of the activations
    static constexpr int XAREA = XL * 1024, WAREA = WL * 1024;
    static constexpr int WAT = 2 * XAREA, DXAT = WAT + WPG * WAREA, OWN = XD, LDS = DXAT + WPG * XD;
};
}  // namespace es

// A buffer's descriptor in scalar registers.
__device__ __forceinline__ v4i stream_buffer(const uint8_t *p, uint32_t bytes) {
    const uint64_t at = reinterpret_cast<uint64_t>(p);
    return v4i{uniform((int)(uint32_t)at), uniform((int)(uint32_t)(at >> 32) & 0xffff), uniform((int)bytes), 0x00020000};
}

// 16 bytes a lane from a buffer into LDS at m0base + 16 * lane; inline assembly, so
// that the compiler does not wait for the copies in flight before each LDS read.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void stream_to_lds(v4i r, uint32_t m0base, uint32_t voff, int soff) {
    asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :: "s"(m0base), "v"(voff), "s"(r), "s"(soff) : "memory", "m0");
}
#pragma clang diagnostic pop

// The loop over the stages of one tile.  C: the format's constants and its step,
//   C::XBYTES, WBYTES    bytes of a stage of an activation and of a weight row
//   C::XC, WC            chunks of them in LDS;  xchunk, wchunk: where chunk c starts
//   C::Step              empty() takes the weights out of LDS, work() uses them
//
// A row that is no whole number of stages (TAIL) ends with a stage of its last BLOCKS
// blocks, of which work() skips those that the stage before had.
//
// C::WLEAD, XLEAD, parts of 2 mod 4 bytes: every other one, along a row or down the rows,
// starts two bytes off the dword grid, where a copy takes four times as long (27 ns a wave
// against 7).  Such a part is copied from two bytes before and its LDS row starts with
// this lead; the chunk that brings the part's end (of Q6_K the last, of the others one
// more, MORE) is moved by two bytes, so that it too starts on the grid.
template <class C, int ROWS, int FR, int G, int WPG>
__device__ __forceinline__ void stream_tile(uint8_t *lds_all, const ExpertArgs &a, const uint8_t *w, int M,
                                            const TileRows &rows) {
    using namespace es;
    using L = typename C::template Lds<ROWS, WPG>;
    constexpr int BN = 32 * WPG;                           // weight rows of the workgroup
    const int lane = threadIdx.x & 63, wave = uniform((threadIdx.x >> 6) % WPG);
    const int grp = G == 1 ? 0 : uniform((threadIdx.x >> 6) / WPG);
    uint8_t *const lds = lds_all + grp * L::LDS;
    const int lr = lane & 31;
    const int n0 = rows.nt * BN, all = (a.nb + C::BLOCKS - 1) / C::BLOCKS;     // stages of a row; this group's are [s0, s1)
    const int s0 = all * grp / G, s1 = all * (grp + 1) / G;
    const int steps = (all + G - 1) / G;                   // every wave passes the same barriers
    constexpr int WB = C::WBYTES / C::BLOCKS, XB = C::XBYTES / C::BLOCKS;
    const uint32_t wrow = (uint32_t)a.nb * WB, xrow = (uint32_t)a.nb * XB;
    // up to two bytes past the last row, in its last dword
    const uint32_t x_bytes = C::XLEAD ? (rows.x_bytes + 3) & ~3u : rows.x_bytes;
    const uint32_t w_bytes = (uint32_t)min(a.N - n0, BN) * wrow;
    const v4i xr = stream_buffer(a.x, x_bytes);
    const v4i wr = stream_buffer(w + (int64_t)n0 * wrow, C::WLEAD ? (w_bytes + 3) & ~3u : w_bytes);
    // copies: rows past the matrix, and past the tile, repeat its last
    // (activations: the 8 FR rows that are worked out)
    constexpr int XL = (8 * FR * C::XC + kWave - 1) / kWave, NA = (XL + WPG - 1) / WPG;
    uint32_t xoff[NA], woff[L::WL], xat[NA];
    // what a stage that starts at an odd block adds: its scalar offset is two bytes less
    int xstep[C::XLEAD ? NA : 1], wstep[C::WLEAD ? L::WL : 1];
#pragma unroll
    for (int k = 0; k < NA; ++k) {
        const int q = min(wave + WPG * k, XL - 1), f = min(kWave * q + lane, 8 * FR * C::XC - 1), row = f / C::XC;
        const int c = f - C::XC * row;
        const uint32_t r = (uint32_t)rows.src[min(row, M - 1)];
        xoff[k] = r * xrow + (uint32_t)C::xchunk(c);
        xat[k] = 1024u * (uint32_t)q;
        if constexpr (C::XLEAD) {
            const bool off = r & a.nb & 1, more = c >= C::MORE * C::XBYTES / 16;
            xoff[k] += off ? (more ? 2 : -2) : 0;
            xstep[k] = off == more ? 0 : 4;
        }
    }
#pragma unroll
    for (int k = 0; k < L::WL; ++k) {
        const int f = min(kWave * k + lane, 32 * C::WC - 1), row = f / C::WC, c = f - C::WC * row;
        const int r = min(n0 + 32 * wave + row, a.N - 1);
        woff[k] = (uint32_t)(r - n0) * wrow + (uint32_t)C::wchunk(c);
        if constexpr (C::WLEAD) {
            const bool off = r & a.nb & 1, more = c >= C::MORE * C::WBYTES / 16;
            woff[k] += off ? (more ? 2 : -2) : 0;
            wstep[k] = off == more ? 0 : 4;
        }
    }
    const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>(lds);
    const uint32_t w0 = (uint32_t)uniform((int)(lds0 + L::WAT + L::WAREA * wave));
    // the stage's first block
    auto first = [&](int s) { return C::TAIL ? min(s * C::BLOCKS, a.nb - C::BLOCKS) : s * C::BLOCKS; };
    auto copy_weights = [&](int s) {
        const int at = first(s);
#pragma unroll
        for (int k = 0; k < L::WL; ++k)
            stream_to_lds(wr, w0 + 1024 * k, C::WLEAD && (at & 1) ? woff[k] + wstep[C::WLEAD ? k : 0] : woff[k],
                          C::WLEAD ? at * WB & ~3 : at * WB);
    };
    auto copy_rows = [&](int s, int buffer) {
        const int at = first(s);
#pragma unroll
        for (int k = 0; k < NA; ++k)
            stream_to_lds(xr, (uint32_t)uniform((int)(lds0 + buffer * L::XAREA + xat[k])),
                          C::XLEAD && (at & 1) ? xoff[k] + xstep[C::XLEAD ? k : 0] : xoff[k],
                          C::XLEAD ? at * XB & ~3 : at * XB);
    };
    typename C::template Step<ROWS, FR> step(lds + L::WAT + L::WAREA * wave + 16 * C::WC * lr,
                                             lds + L::DXAT + L::OWN * wave, lane);
    if constexpr (C::XLEAD || C::WLEAD) step.parities(min(n0 + 32 * wave + lr, a.N - 1) & a.nb, rows.src, M);
    if (s0 < s1) {
        copy_weights(s0);
        copy_rows(s0, 0);
    }
    // A step waits for its own copies of the stage, the barrier publishes every
    // wave's activations (and tells that the buffer of the stage before is free).
    for (int i = 0; i < steps; ++i) {
        asm volatile("s_waitcnt vmcnt(0)\n\ts_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        const int s = s0 + i;
        if (G > 1 && s >= s1) continue;                    // another group has one stage more
        if (s + 1 < s1) copy_rows(s + 1, (i + 1) & 1);
        step.empty(first(s));
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); // the weights are in registers
        if (s + 1 < s1) copy_weights(s + 1);
        step.work(lds + (i & 1) * L::XAREA, first(s), s * C::BLOCKS - first(s));
    }
    if constexpr (G > 1) {
        // the other groups hand their sums to group 0 through LDS, which adds them in
        // the groups' order
        constexpr int SUMS = 256 * FR;                     // of a wave
        static_assert((G - 1) * WPG * SUMS * 4 <= G * L::LDS, "the sums fit");
        float *sums = reinterpret_cast<float *>(lds_all) + SUMS * wave + lane;
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (grp > 0) {
#pragma unroll
            for (int r = 0; r < 4 * FR; ++r) sums[SUMS * WPG * (grp - 1) + 64 * r] = step.acc[r];
        }
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (grp > 0) return;
#pragma unroll
        for (int g = 1; g < G; ++g)
#pragma unroll
            for (int r = 0; r < 4 * FR; ++r) step.acc[r] += sums[SUMS * WPG * (g - 1) + 64 * r];
    }
    const int n = n0 + 32 * wave + lr;                     // lane l, register r: row 8 (r / 4) + 4 (l / 32) + r % 4
    if (n >= a.N) return;
#pragma unroll
    for (int r = 0; r < 4 * FR; ++r) {
        const int m = 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
        if (m < M) a.y[(int64_t)rows.pair[m] * a.N + n] = step.acc[r] * C::OUT_SCALE;
    }
}

template <class C, int ROWS, int G, int WPG>
__global__ __launch_bounds__(64 * G * WPG) void k_experts_stream(ExpertArgs a, int tiles_n, int parts) {
    using L = typename C::template Lds<ROWS, WPG>;
    extern __shared__ __attribute__((aligned(16))) uint8_t stream_lds[];
    int *pair = reinterpret_cast<int *>(stream_lds + G * L::LDS), *src = pair + ROWS;
    // parts: log2 of the workgroups that a tile's rows take
    const int part = (int)blockIdx.x / tiles_n, chunk = part >> parts;
    const Tile tile = expert_tile(a, chunk, pair, src, (part - (chunk << parts)) * ROWS, ROWS);
    if (tile.count == 0) return;
    __syncthreads();
    const TileRows rows = {pair, src, a.x_bytes, (int)blockIdx.x - part * tiles_n};
    if (tile.expert == a.E) {
        zero_tile(a, tile.count, rows, 32 * WPG);
        return;
    }
    const uint8_t *w = a.w + (int64_t)tile.expert * a.stride;
    if (tile.count <= 8)
        stream_tile<C, ROWS, 1, G, WPG>(stream_lds, a, w, tile.count, rows);
    else if (ROWS == 16 || tile.count <= 16)
        stream_tile<C, ROWS, 2, G, WPG>(stream_lds, a, w, tile.count, rows);
    else if (ROWS == 32 || tile.count <= 32)
        stream_tile<C, ROWS, 4, G, WPG>(stream_lds, a, w, tile.count, rows);
    else if (tile.count <= 48)
        stream_tile<C, ROWS, ROWS == 64 ? 6 : 4, G, WPG>(stream_lds, a, w, tile.count, rows);
    else
        stream_tile<C, ROWS, ROWS == 64 ? 8 : 4, G, WPG>(stream_lds, a, w, tile.count, rows);
}

template <class C, int ROWS, int G, int WPG>
static hipError_t launch_stream(const ExpertArgs &a, hipStream_t st) {
    constexpr int lds = G * C::template Lds<ROWS, WPG>::LDS + 8 * ROWS;
    static_assert(lds <= kMaxLdsBytes, "LDS of one CU");
    const void *k = (const void *)k_experts_stream<C, ROWS, G, WPG>;
    static int lds_ok[kLdsDevices] = {};
    const hipError_t e = allow_dynamic_lds(k, (size_t)lds, lds_ok);
    if (e != hipSuccess) return e;
    int tiles_n = (a.N + 32 * WPG - 1) / (32 * WPG), parts = 0;
    while (ROWS << parts < a.rows) ++parts;
    ExpertArgs args = a;
    void *argv[] = {(void *)&args, (void *)&tiles_n, (void *)&parts};
    return hipLaunchKernel(k, dim3((unsigned)((grid_tiles(a) << parts) * tiles_n)), dim3(64 * G * WPG), argv, (size_t)lds, st);
}

// Blocks of 128 weight rows that the call is likely to have, every expert in use.
constexpr int64_t kEnoughBlocks = 3 * kCUs / 2, kFewBlocks = kCUs / 2;       // for one group of waves each; for no two
inline int64_t stream_blocks(const ExpertArgs &a) {
    const int64_t tiles = (a.pairs < a.E ? a.pairs : a.E) + a.pairs / (a.rows < kNarrowRows ? a.rows : kNarrowRows);
    return tiles * ((a.N + 127) / 128);
}

template <class C, int ROWS>
static hipError_t pick_stream(const ExpertArgs &a, hipStream_t st) {
    // The workgroup that suits the call's blocks of 128 weight rows.  Few: K cut over
    // four groups of two waves, or two of two (us, Q4_0, one group of four waves / two
    // of two / four of two):
    //   40 blocks, 4 experts of 512 x 2048  17.1 / 10.8 / 8.9     114, 16 of 768 x 2048  11.3 / 9.0 / 8.5
    //   128, 64 of 1024 x 2048  9.8 / 7.6 / 7.6                   336, 8 of 3584 x 4096  33.0 / 24.8 / 29.3
    // Enough: one group, of two waves for the 32-value formats, whose smaller workgroups
    // spread more evenly over the compute units; of four for the K-quants, whose
    // activations are more bytes beside their weights, from 512 blocks on (one group of four
    // waves / of two):
    //   448 blocks, 8 of 3500 x 4096, 131 tokens  Q8_0 54 / 48  Q4_0 44 / 39  Q5_1 68 / 61  Q4_K 34 / 32  Q6_K 63 / 60
    //   560, 8 of 3584 x 4096, 200 tokens         Q8_0 57 / 56  Q4_0 44 / 44  Q5_1 70 / 67  Q4_K 35 / 36  Q6_K 64 / 78
    //   1900, 128 of 1536 x 2048, 500 tokens      Q8_0 135 / 131  Q4_0 93 / 96  Q5_1 152 / 146  Q4_K 78 / 87  Q6_K 141 / 146
    const int64_t blocks = stream_blocks(a);
    if (blocks >= kEnoughBlocks) {
        if constexpr (C::BLOCKS == 1)
            if (blocks >= 2 * kCUs) return launch_stream<C, ROWS, 1, 4>(a, st);
        return launch_stream<C, ROWS, 1, 2>(a, st);
    }
    if (blocks >= kFewBlocks) return launch_stream<C, ROWS, 2, 2>(a, st);
    return launch_stream<C, ROWS, 4, 2>(a, st);
}

template <class C>
static hipError_t experts_stream(const ExpertArgs &a, hipStream_t st) {
    if (a.rows <= kFewRows) return pick_stream<C, kFewRows>(a, st);
    // The K-quants' tiles of 128 in parts of 64 rows, or of 32: half of the weights' ways through LDS, half of the
    // workgroups (us, 32 / 64 rows: 128 experts of 1536 x 2048, 64 rows each Q4_K 125 / 118, Q6_K 233 / 202; 64 of 512 rows
    // each Q2_K 263 / 244, Q4_K 359 / 320, Q6_K 687 / 580; 8 of 3584 x 4096, 50 rows each, 560 blocks Q4_K 37 / 39, Q6_K
    // 64 / 77)
    if constexpr (C::HALF)
        if (a.rows == kFullRows && stream_blocks(a) >= 2 * kEnoughBlocks) return launch_stream<C, kHalfRows, 1, 4>(a, st);
    return pick_stream<C, kNarrowRows>(a, st);
}

}  // namespace qmm
