#pragma once
// Products of a few rows with an expert's weights: y[p] = W[id_p] x[p].
//
// Bound by the weight stream, as a decode step is: every used expert's bytes
// come from HBM once.  A workgroup takes a tile of an expert's rows (or finds its
// rows from the ids, in calls of up to 64 pairs) and four waves' weight rows: each wave copies the
// contiguous bytes of its rows into its own LDS slice and dots them with up to
// TT activation rows in turn.  LPR lanes share a weight row, each holding one
// unit of it and of the activations (units as in the decode matvec), so that
// experts' short rows fill a wave too; rows of more than 64 units are walked in
// segments.
#include "matvec_kernel.h"
#include "moe.h"

namespace qmm {

constexpr int kFewWaves = 4;

template <int BIT>
__device__ __forceinline__ float sum_below(float v) {
    if constexpr (BIT >= 1) return sum_below<BIT / 2>(xsum<BIT>(v));
    return v;
}

template <int F, bool PAIRED, int LPR, int RI, int TT>
__global__ __launch_bounds__(64 * kFewWaves) void k_experts_few(ExpertArgs a, int xs, int ss) {
    using FB = FmtBytes<F>;
    using UT = ::qmm::Unit<F, PAIRED>;
    extern __shared__ uint4 lds_dyn[];
    constexpr int RW = kWave / LPR * RI;               // weight rows of a wave
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int chunk = blockIdx.y;
    const int64_t row0 = ((int64_t)blockIdx.x * kFewWaves + wave) * RW;
    const int nrows = (int)max((int64_t)0, min((int64_t)RW, (int64_t)a.N - row0));

    // the workgroup's expert and rows
    int e, count, start = 0;
    uint64_t members = 0;                              // from the ids: the pairs, one for each lane
    if (a.ids != nullptr) {
        const int id = lane < a.pairs ? a.ids[lane] : -1;
        e = __builtin_amdgcn_readlane(id, chunk);
        if ((unsigned)e >= (unsigned)a.E) {
            e = a.E;
            members = 1ull << chunk;
        } else {                                       // every TT-th pair of an expert takes the next TT
            members = __ballot(id == e && lane < a.pairs);
            if (__popcll(members & ((1ull << chunk) - 1)) % TT) return;
            members &= ~0ull << chunk;
        }
        count = min(__popcll(members), TT);
    } else {
        if (chunk >= *a.plan.count) return;
        const Tile tile = a.plan.tiles[chunk];
        e = uniform(tile.expert);
        count = uniform(tile.count);
        start = uniform(tile.start);
    }
    auto next = [&](int i) {                           // the i-th pair, in order
        if (a.ids == nullptr) return uniform(a.plan.pair[start + i]);
        const int p = __builtin_ctzll(members);
        members &= members - 1;
        return p;
    };
    if (e == a.E) {                                    // no expert: zeros
        for (int i = 0; i < count; ++i) {
            float *y = a.y + (int64_t)next(i) * a.N;
            for (int r = lane; r < nrows; r += kWave) y[row0 + r] = 0.0f;
        }
        return;
    }
    const uint8_t *w = a.w + (int64_t)e * a.stride;
    const int64_t RB = (int64_t)a.nb * FB::BB, xrow = (int64_t)a.nb * FB::XB;
    const int nu = (a.nb / UT::BPU) * UT::UPB;         // units of a row
    const int ul = lane % LPR, sub = lane / LPR;
    uint4 *slice = lds_dyn + TT * (xs / 16) + wave * (ss / 16);
    const uint8_t *xl8 = reinterpret_cast<const uint8_t *>(lds_dyn);
    const uint8_t *sl8 = reinterpret_cast<const uint8_t *>(slice);

    for (int i0 = 0; i0 < count; i0 += TT) {
        const int n = min(TT, count - i0);
        int pair[TT];
#pragma unroll
        for (int t = 0; t < TT; ++t) pair[t] = t < n ? next(i0 + t) : 0;
        float acc[RI][TT];
#pragma unroll
        for (int r = 0; r < RI; ++r)
#pragma unroll
            for (int t = 0; t < TT; ++t) acc[r][t] = 0.0f;
        for (int u0 = 0; u0 < nu; u0 += kWave) {
            const int u1 = min(nu, u0 + kWave);
            const int b0 = u0 / UT::UPB * UT::BPU, b1 = u1 / UT::UPB * UT::BPU;       // blocks of the segment
            uint32_t xoff[TT];
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                if (t >= n) break;
                const int64_t xr = (int64_t)(a.x_per_pair ? pair[t] : pair[t] / a.top) * xrow;
                const int64_t lo = xr + (int64_t)b0 * FB::XB, hi = xr + (int64_t)b1 * FB::XB;
                xoff[t] = (uint32_t)(lo & 15);
                dma_span(a.x, lo, hi, lds_dyn + t * (xs / 16), lane, wave, kFewWaves);
            }
            int64_t A = 0;
            if (nrows > 0) {
                const int64_t lo = row0 * RB + (int64_t)b0 * FB::BB;
                const int64_t hi = (row0 + nrows - 1) * RB + (int64_t)b1 * FB::BB;
                A = lo & ~(int64_t)15;
                dma_span<true>(w, lo, hi, slice, lane, 0, 1);
            }
            wait_vmcnt(0);
            __syncthreads();                           // the activations of every wave's copies
            if (nrows > 0) {
                const bool live = ul < u1 - u0;
                const int u = min(ul, u1 - u0 - 1);
                UnitW<F, PAIRED> wu[RI];
#pragma unroll
                for (int r = 0; r < RI; ++r) {
                    const int row = min(r * (kWave / LPR) + sub, nrows - 1);
                    const uint32_t ro = (uint32_t)((row0 + row) * RB + (int64_t)b0 * FB::BB - A);
                    wu[r].load(sl8, ro + (uint32_t)(u / UT::UPB * UT::BPU) * FB::BB, u0 + u);
                }
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    if (t >= n) break;
                    XU<F, PAIRED> xu;
                    load_xu<F, PAIRED>(xl8 + t * xs, xoff[t], u, xu);
#pragma unroll
                    for (int r = 0; r < RI; ++r)
                        if (live) acc[r][t] = wu[r].dot(xu, acc[r][t]);
                }
            }
            if (u1 < nu || i0 + TT < count) {          // the LDS is filled again
                wait_lds_reads();
                __syncthreads();
            }
        }
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            if (t >= n) break;
#pragma unroll
            for (int r = 0; r < RI; ++r) {
                const float s = sum_below<LPR / 2>(acc[r][t]);
                const int row = r * (kWave / LPR) + sub;
                if (ul == 0 && row < nrows) a.y[(int64_t)pair[t] * a.N + row0 + row] = s;
            }
        }
    }
}

template <int F, bool PAIRED, int LPR, int RI, int TT>
static hipError_t launch_few(const ExpertArgs &a, hipStream_t st) {
    using FB = FmtBytes<F>;
    using UT = ::qmm::Unit<F, PAIRED>;
    constexpr int RW = kWave / LPR * RI;
    const int nu = (a.nb / UT::BPU) * UT::UPB, segu = nu < kWave ? nu : kWave;
    const int64_t segb = (segu + UT::UPB - 1) / UT::UPB * UT::BPU;
    // whole 1 KB groups of chunks, up to 15 bytes of misalignment at each end
    const int64_t span = (int64_t)(RW - 1) * a.nb * FB::BB + segb * FB::BB;
    int ss = (int)((span + 32 + 1023) / 1024 * 1024), xs = (int)((segb * FB::XB + 32 + 1023) / 1024 * 1024);
    const size_t lds = (size_t)TT * xs + (size_t)kFewWaves * ss;
    const void *k = (const void *)k_experts_few<F, PAIRED, LPR, RI, TT>;
    static int lds_ok[kLdsDevices] = {};
    const hipError_t e = allow_dynamic_lds(k, lds, lds_ok);
    if (e != hipSuccess) return e;
    const int row_blocks = (a.N + RW * kFewWaves - 1) / (RW * kFewWaves);
    const int64_t chunks = a.ids != nullptr ? a.pairs : max_tiles(a.pairs, a.E, tile_rows(a.pairs, a.E));
    ExpertArgs args = a;
    void *argv[] = {(void *)&args, (void *)&xs, (void *)&ss};
    return hipLaunchKernel(k, dim3((unsigned)row_blocks, (unsigned)chunks), dim3(64 * kFewWaves), argv, lds, st);
}

template <int F, bool PAIRED, int TT>
static hipError_t pick_few(const ExpertArgs &a, hipStream_t st) {
    using UT = ::qmm::Unit<F, PAIRED>;
    const int nu = (a.nb / UT::BPU) * UT::UPB;
    if (nu <= 8) return launch_few<F, PAIRED, 8, 2, TT>(a, st);
    if (nu <= 16) return launch_few<F, PAIRED, 16, 2, TT>(a, st);
    if (nu <= 32) return launch_few<F, PAIRED, 32, 2, TT>(a, st);
    return launch_few<F, PAIRED, 64, 1, TT>(a, st);
}

template <int F>
static hipError_t experts_few(const ExpertArgs &a, hipStream_t st) {
    const bool one = a.pairs <= a.top;                 // one token
    if constexpr (!kIsK<F>) {
        if (a.nb % 2 == 0) return one ? pick_few<F, true, 1>(a, st) : pick_few<F, true, kFewRows>(a, st);
    }
    return one ? pick_few<F, false, 1>(a, st) : pick_few<F, false, kFewRows>(a, st);
}

}  // namespace qmm
