#pragma once
// Products of one token with its experts' weights, y[p] = W[id_p] x[p], and of any number
// of tokens with rows of one block of 32 values, which are no stage of the other kernels.
//
// Bound by the weight stream, as a decode step is: a token's experts are read once
// from HBM.  A workgroup takes a tile of an expert's rows (of one token nearly
// always one row) and four waves' weight rows: each wave copies the contiguous
// bytes of its rows into its own LDS slice and dots them with the activation rows
// in turn.  LPR lanes share a weight row, each holding one unit of it and of the
// activations (units as in the decode matvec), so that experts' short rows fill a
// wave too; rows of more than 64 units are walked in segments.  (8 of 128 experts of
// 1536 x 2048: Q4_0 4.8 us, 3.0 TB/s of weights; Q8_0 5.7 us, 4.7 TB/s; about 2 us of
// each are the launch and the chain from the ids to the first weight byte.)
#include "matvec_kernel.h"
#include "moe.h"

namespace qmm {

constexpr int kFewWaves = 4;
constexpr int kFewTiles = 32768;                       // of a launch at most: they lie along the grid's y, which holds 65535

template <int BIT>
__device__ __forceinline__ float sum_below(float v) {
    if constexpr (BIT >= 1) return sum_below<BIT / 2>(xsum<BIT>(v));
    return v;
}

template <int F, bool PAIRED, int LPR, int RI>
__global__ __launch_bounds__(64 * kFewWaves) void k_experts_few(ExpertArgs a, int tile0, int xs, int ss) {
    using FB = FmtBytes<F>;
    using UT = ::qmm::Unit<F, PAIRED>;
    extern __shared__ uint4 lds_dyn[];
    __shared__ int pairs[kFullRows], sources[kFullRows];
    constexpr int RW = kWave / LPR * RI;               // weight rows of a wave
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int64_t row0 = ((int64_t)blockIdx.x * kFewWaves + wave) * RW;
    const int nrows = (int)max((int64_t)0, min((int64_t)RW, (int64_t)a.N - row0));
    const Tile tile = expert_tile(a, tile0 + (int)blockIdx.y, pairs, sources, 0, a.rows);
    if (tile.count == 0) return;
    __syncthreads();
    if (tile.expert == a.E) {                          // no expert: zeros
        for (int i = 0; i < tile.count; ++i) {
            float *y = a.y + (int64_t)pairs[i] * a.N;
            for (int r = lane; r < nrows; r += kWave) y[row0 + r] = 0.0f;
        }
        return;
    }
    const uint8_t *w = a.w + (int64_t)tile.expert * a.stride;
    const int64_t RB = (int64_t)a.nb * FB::BB, xrow = (int64_t)a.nb * FB::XB;
    const int nu = (a.nb / UT::BPU) * UT::UPB;         // units of a row
    const int ul = lane % LPR, sub = lane / LPR;
    uint4 *slice = lds_dyn + xs / 16 + wave * (ss / 16);
    const uint8_t *xl8 = reinterpret_cast<const uint8_t *>(lds_dyn), *sl8 = reinterpret_cast<const uint8_t *>(slice);

    for (int i = 0; i < tile.count; ++i) {
        const int pair = uniform(pairs[i]);
        const int64_t xr = (int64_t)uniform(sources[i]) * xrow;
        float acc[RI];
#pragma unroll
        for (int r = 0; r < RI; ++r) acc[r] = 0.0f;
        for (int u0 = 0; u0 < nu; u0 += kWave) {
            const int u1 = min(nu, u0 + kWave);
            const int b0 = u0 / UT::UPB * UT::BPU, b1 = u1 / UT::UPB * UT::BPU;       // blocks of the segment
            const int64_t xlo = xr + (int64_t)b0 * FB::XB, xhi = xr + (int64_t)b1 * FB::XB;
            const int64_t lo = row0 * RB + (int64_t)b0 * FB::BB, A = lo & ~(int64_t)15;
            dma_span(a.x, xlo, xhi, lds_dyn, lane, wave, kFewWaves);
            if (nrows > 0 && (i == 0 || nu > kWave))   // whole rows stay for the next activation row
                dma_span<true>(w, lo, (row0 + nrows - 1) * RB + (int64_t)b1 * FB::BB, slice, lane, 0, 1);
            wait_vmcnt(0);
            __syncthreads();                           // the activations of every wave's copies
            const bool live = ul < u1 - u0;
            const int u = min(ul, u1 - u0 - 1);
            if (nrows > 0) {
                XU<F, PAIRED> xu;
                load_xu<F, PAIRED>(xl8, (uint32_t)(xlo & 15), u, xu);
#pragma unroll
                for (int r = 0; r < RI; ++r) {
                    const int row = min(r * (kWave / LPR) + sub, nrows - 1);
                    const uint32_t ro = (uint32_t)((row0 + row) * RB + (int64_t)b0 * FB::BB - A);
                    if (live)
                        acc[r] = unit_dot<F, PAIRED>(sl8, ro + (uint32_t)(u / UT::UPB * UT::BPU) * FB::BB, u0 + u, xu,
                                                     acc[r]);
                }
            }
            if (u1 < nu || i + 1 < tile.count) {       // the LDS is filled again
                wait_lds_reads();
                __syncthreads();
            }
        }
#pragma unroll
        for (int r = 0; r < RI; ++r) {
            const float s = sum_below<LPR / 2>(acc[r]);
            const int row = r * (kWave / LPR) + sub;
            if (ul == 0 && row < nrows) a.y[(int64_t)pair * a.N + row0 + row] = s;
        }
    }
}

template <int F, bool PAIRED, int LPR, int RI>
static hipError_t launch_few(const ExpertArgs &a, hipStream_t st) {
    using FB = FmtBytes<F>;
    using UT = ::qmm::Unit<F, PAIRED>;
    constexpr int RW = kWave / LPR * RI;
    const int nu = (a.nb / UT::BPU) * UT::UPB, segu = nu < kWave ? nu : kWave;
    const int64_t segb = (segu + UT::UPB - 1) / UT::UPB * UT::BPU;
    // whole 1 KB groups of chunks, up to 15 bytes of misalignment at each end
    const int64_t span = (int64_t)(RW - 1) * a.nb * FB::BB + segb * FB::BB;
    int ss = (int)((span + 32 + 1023) / 1024 * 1024), xs = (int)((segb * FB::XB + 32 + 1023) / 1024 * 1024);
    const size_t lds = (size_t)xs + (size_t)kFewWaves * ss;
    const void *k = (const void *)k_experts_few<F, PAIRED, LPR, RI>;
    if (a.rows > kFullRows) return hipErrorInvalidValue;          // the kernel's tables
    static int lds_ok[kLdsDevices] = {};
    const hipError_t e = allow_dynamic_lds(k, lds, lds_ok);
    if (e != hipSuccess) return e;
    const int row_blocks = (a.N + RW * kFewWaves - 1) / (RW * kFewWaves);
    ExpertArgs args = a;
    const int tiles = (int)grid_tiles(a);
    const int room = (1 << 23) / row_blocks, step = room < kFewTiles ? room : kFewTiles;       // 2^31 threads a launch
    for (int tile0 = 0; tile0 < tiles; tile0 += step) {
        void *argv[] = {(void *)&args, (void *)&tile0, (void *)&xs, (void *)&ss};
        const int y = tiles - tile0 < step ? tiles - tile0 : step;
        const hipError_t le = hipLaunchKernel(k, dim3((unsigned)row_blocks, (unsigned)y), dim3(64 * kFewWaves), argv, lds, st);
        if (le != hipSuccess) return le;
    }
    return hipSuccess;
}

template <int F, bool PAIRED>
static hipError_t pick_few(const ExpertArgs &a, hipStream_t st) {
    using UT = ::qmm::Unit<F, PAIRED>;
    const int nu = (a.nb / UT::BPU) * UT::UPB;
    if (nu <= 8) return launch_few<F, PAIRED, 8, 2>(a, st);
    if (nu <= 16) return launch_few<F, PAIRED, 16, 2>(a, st);
    if (nu <= 32) return launch_few<F, PAIRED, 32, 2>(a, st);
    return launch_few<F, PAIRED, 64, 1>(a, st);
}

template <int F>
static hipError_t experts_few(const ExpertArgs &a, hipStream_t st) {
    if constexpr (!kIsK<F>) {
        if (a.nb % 2 == 0) return pick_few<F, true>(a, st);
    }
    return pick_few<F, false>(a, st);
}

}  // namespace qmm
