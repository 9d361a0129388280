// The plan of the experts' products, and the weighted sum of a token's experts.
#include "kv_layout.h"
#include "moe.h"

namespace qmm {

// ---------------------------------------------------------------------------
// Plan: a stable counting sort of the pairs by expert (an id outside [0, E)
// counts as expert E, whose rows the products fill with zeros), and the tiles.
// One workgroup; wave w takes the w-th stretch of the pairs, 64 at a time.  The
// lanes that hold the same expert find one another by a ballot for each bit of
// its number, so no atomic is needed and the order is that of the pairs.
// ---------------------------------------------------------------------------
constexpr int kPlanWaves = 16;

struct PlanArgs {
    const int *ids;
    Tile *tiles;
    int *pair, *token;
    int pairs, top, E, rows, most, bits;        // most: tiles that there is room for
};

__device__ __forceinline__ uint64_t same_lanes(int key, int bits, bool live) {
    uint64_t m = __ballot(live);
    for (int b = 0; b < bits; ++b) {
        const bool one = (key >> b) & 1;
        const uint64_t ones = __ballot(one);
        m &= one ? ones : ~ones;
    }
    return m;
}

__global__ __launch_bounds__(64 * kPlanWaves) void k_experts_plan(PlanArgs a) {
    extern __shared__ int plan_lds[];                     // [waves][E + 1] counts, then places; [E + 1] first rows; [waves]
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), n = a.E + 1;
    int *counts = plan_lds, *mine = counts + wave * n, *first = counts + kPlanWaves * n, *scan = first + n;
    for (int i = threadIdx.x; i < kPlanWaves * n; i += 64 * kPlanWaves) counts[i] = 0;
    __syncthreads();
    const int each = ((a.pairs + 64 * kPlanWaves - 1) / (64 * kPlanWaves)) * 64;
    const int lo = min(wave * each, a.pairs), hi = min(lo + each, a.pairs);
    auto key_of = [&](int p) {
        const int id = p < hi ? a.ids[p] : 0;
        return (unsigned)id < (unsigned)a.E ? id : a.E;
    };
    for (int p = lo + lane; p - lane < hi; p += 64) {
        const int key = key_of(p);
        const uint64_t m = same_lanes(key, a.bits, p < hi);
        if (p < hi && __builtin_ctzll(m) == lane) mine[key] += __popcll(m);
    }
    __syncthreads();
    // thread e sums expert e (E + 1 of them fit the workgroup): places inside the
    // expert for each wave, and the tiles before it
    const int e = threadIdx.x;
    int rows = 0;
    if (e < n) {
        for (int w = 0; w < kPlanWaves; ++w) {
            const int c = counts[w * n + e];
            counts[w * n + e] = rows;
            rows += c;
        }
    }
    const int tiles = (rows + a.rows - 1) / a.rows;
    int upto = tiles;                                     // inclusive sum in the wave, then the waves before
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(upto, d, kWave);
        if (lane >= d) upto += o;
    }
    if (lane == 63) scan[wave] = upto;
    __syncthreads();
    int before = upto - tiles, all = 0;
    for (int w = 0; w < kPlanWaves; ++w) {
        if (w < wave) before += scan[w];
        all += scan[w];
    }
    if (e < n) {
        first[e] = before * a.rows;
        for (int k = 0; k < tiles; ++k) a.tiles[before + k] = {e, min(a.rows, rows - k * a.rows)};
    }
    for (int k = all + threadIdx.x; k < a.most; k += 64 * kPlanWaves) a.tiles[k] = {0, 0};
    __syncthreads();
    for (int p = lo + lane; p - lane < hi; p += 64) {
        const int key = key_of(p);
        const uint64_t m = same_lanes(key, a.bits, p < hi);
        if (p < hi) {
            const int at = first[key] + mine[key] + __popcll(m & ((1ull << lane) - 1));
            a.pair[at] = p;
            a.token[at] = p / a.top;
        }
        if (p < hi && __builtin_ctzll(m) == lane) mine[key] += __popcll(m);
    }
}

static_assert(kMaxExperts + 1 <= 64 * kPlanWaves, "a thread for every expert");

hipError_t launch_experts_plan(const int *ids, void *plan, int pairs, int top, int E, hipStream_t st) {
    if (pairs <= kSelfPairs) return hipSuccess;
    const Plan p = plan_at(plan, pairs, E);
    const int rows = tile_rows(pairs, E);
    PlanArgs a = {ids, const_cast<Tile *>(p.tiles), const_cast<int *>(p.pair), const_cast<int *>(p.token), pairs, top, E,
                  rows, (int)max_tiles(pairs, E, rows), 32 - __builtin_clz((unsigned)E)};
    const size_t lds = (size_t)((kPlanWaves + 1) * (E + 1) + kPlanWaves) * 4;      // 35 KB at most
    void *args[] = {(void *)&a};
    return hipLaunchKernel((const void *)k_experts_plan, dim3(1), dim3(64 * kPlanWaves), args, lds, st);
}

// ---------------------------------------------------------------------------
// out[t] = residual[t] + sum_j weights[t][j] y[t top + j], f32, in the order of j,
// the residual last; one rounding to the rows' type.  Bound by memory.
// ---------------------------------------------------------------------------
struct CombineArgs {
    const float *y, *weights;
    const void *residual;       // NULL: none
    void *out;
    int64_t T, rs, os;          // strides in elements
    int top;
    uint32_t width;             // V-value pieces of a row
};

constexpr int kCombineThreads = 256;
constexpr int64_t kCombineGrid = 1 << 22;      // workgroups of a launch: a grid holds 2^32 threads

// V values a thread: 4, or 1 where N is no multiple of 4.
template <int RT, int V>
__global__ __launch_bounds__(kCombineThreads) void k_experts_combine(CombineArgs a) {
    const int64_t all = a.T * a.width;
    for (int64_t base = (int64_t)blockIdx.x * kCombineThreads; base < all;
         base += (int64_t)gridDim.x * kCombineThreads) {
        const int64_t row0 = base / a.width;
        const uint32_t at = (uint32_t)(base - row0 * a.width) + threadIdx.x;
        const int64_t t = row0 + at / a.width;
        const uint32_t c = at % a.width;
        if (t >= a.T) continue;
        const float *y = a.y + (t * a.top * a.width + c) * V, *w = a.weights + t * a.top;
        if constexpr (V == 4) {
            float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
            for (int j = 0; j < a.top; ++j) {
                const float4 v = *reinterpret_cast<const float4 *>(y + (int64_t)j * a.width * 4);
                s = make_float4(fmaf(w[j], v.x, s.x), fmaf(w[j], v.y, s.y), fmaf(w[j], v.z, s.z), fmaf(w[j], v.w, s.w));
            }
            if (a.residual != nullptr) {
                const float4 r = load4<RT>(a.residual, t * a.rs + 4 * (int64_t)c);
                s = make_float4(s.x + r.x, s.y + r.y, s.z + r.z, s.w + r.w);
            }
            store4<RT>(a.out, t * a.os + 4 * (int64_t)c, s);
        } else {
            float s = 0.0f;
            for (int j = 0; j < a.top; ++j) s = fmaf(w[j], y[(int64_t)j * a.width], s);
            if (a.residual != nullptr) s += load1<RT>(a.residual, t * a.rs + c);
            if constexpr (RT == R_F32)
                static_cast<float *>(a.out)[t * a.os + c] = s;
            else
                static_cast<uint16_t *>(a.out)[t * a.os + c] = (uint16_t)(pack2<RT>(s, 0.0f) & 0xffffu);
        }
    }
}

hipError_t launch_experts_combine(int rt, const float *y, const float *weights, const void *residual, void *out,
                                  int64_t T, int top, int64_t N, int64_t rs, int64_t os, hipStream_t st) {
    const bool four = N % 4 == 0;
    CombineArgs a = {y, weights, residual, out, T, rs, os, top, (uint32_t)(four ? N / 4 : N)};
    const int64_t grid = (T * a.width + kCombineThreads - 1) / kCombineThreads;
    const void *k = rt == R_F32   ? (four ? (const void *)k_experts_combine<R_F32, 4> : (const void *)k_experts_combine<R_F32, 1>)
                    : rt == R_F16 ? (four ? (const void *)k_experts_combine<R_F16, 4> : (const void *)k_experts_combine<R_F16, 1>)
                                  : (four ? (const void *)k_experts_combine<R_BF16, 4> : (const void *)k_experts_combine<R_BF16, 1>);
    void *args[] = {(void *)&a};
    return hipLaunchKernel(k, dim3((unsigned)(grid < kCombineGrid ? grid : kCombineGrid)), dim3(kCombineThreads), args,
                           0, st);
}

}  // namespace qmm
