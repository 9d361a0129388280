// The plan of the experts' products, and the weighted sum of a token's experts.
#include "kv_layout.h"
#include "moe.h"

namespace qmm {

// ---------------------------------------------------------------------------
// Plan: a stable counting sort of the pairs by expert (an id outside [0, E)
// counts as expert E, whose rows the products fill with zeros), and the tiles.
// A workgroup takes a segment of the pairs, wave w of it the w-th stretch, 64 at a
// time.  The lanes that hold the same expert find one another by a ballot for each
// bit of its number, so no atomic orders anything and the order is that of the pairs.
// More than one segment: a launch before it counts each segment's pairs, and every
// workgroup sums those of the segments before its own.  Bound by latency; one workgroup
// for all pairs would be bound by its compute unit's vector units (32768 pairs of 64
// experts: 48 us in one workgroup, 8.8 in 32 after a count).
// ---------------------------------------------------------------------------
constexpr int kPlanWaves = 16;

struct PlanArgs {
    const int *ids;
    Tile *tiles;
    int *pair, *token, *counts;                 // counts: [segments][E + 1]
    int pairs, top, E, rows, most, bits;        // most: tiles that there is room for
    int segment, segments;
};

__global__ __launch_bounds__(256) void k_experts_count(PlanArgs a) {
    extern __shared__ int count_lds[];
    const int n = a.E + 1, lo = blockIdx.x * a.segment, hi = min(lo + a.segment, a.pairs);
    for (int i = threadIdx.x; i < n; i += 256) count_lds[i] = 0;
    __syncthreads();
    for (int p = lo + threadIdx.x; p < hi; p += 256) {
        const int id = a.ids[p];
        atomicAdd(count_lds + ((unsigned)id < (unsigned)a.E ? id : a.E), 1);    // a sum of whole numbers: any order
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += 256) a.counts[(int64_t)blockIdx.x * n + i] = count_lds[i];
}

__device__ __forceinline__ uint64_t same_lanes(int key, int bits, bool live) {
    uint64_t m = __ballot(live);
    for (int b = 0; b < bits; ++b) {
        const bool one = (key >> b) & 1;
        const uint64_t ones = __ballot(one);
        m &= one ? ones : ~ones;
    }
    return m;
}

// HOLD ids a lane; longer segments (HOLD < 0) come in batches of -HOLD, twice.
template <int HOLD>
__global__ __launch_bounds__(64 * kPlanWaves) void k_experts_plan(PlanArgs a) {
    constexpr int N = HOLD < 0 ? -HOLD : HOLD;
    extern __shared__ int plan_lds[];                     // [waves][E + 1] counts, then places; [E + 1] first rows; [waves]
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), waves = blockDim.x >> 6, n = a.E + 1;
    int *counts = plan_lds, *mine = counts + wave * n, *first = counts + waves * n, *scan = first + n;
    const int from0 = blockIdx.x * a.segment, end = min(from0 + a.segment, a.pairs);
    const int each = (a.segment + 64 * waves - 1) / (64 * waves) * 64;
    const int lo = min(from0 + wave * each, end), hi = min(lo + each, end);
    int key[N];
    auto load = [&](int from) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int p = from + 64 * i + lane;
            key[i] = p < hi ? a.ids[p] : -1;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) key[i] = (unsigned)key[i] < (unsigned)a.E ? key[i] : a.E;
    };
    load(lo);
    for (int i = threadIdx.x; i < waves * n; i += blockDim.x) counts[i] = 0;
    __syncthreads();
    // fn(key, pair, lanes with the same key) of every 64 pairs of the wave, in order
    auto walk = [&](auto fn) {
        for (int from = lo; from < hi; from += 64 * N) {
            if (HOLD < 0) load(from);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int p = from + 64 * i + lane;
                if (p - lane >= hi) break;
                fn(key[i], p, same_lanes(key[i], a.bits, p < hi));
            }
        }
    };
    walk([&](int k, int p, uint64_t m) {
        if (p < hi && __builtin_ctzll(m) == lane) mine[k] += __popcll(m);
    });
    __syncthreads();
    // thread e sums expert e (E + 1 of them fit the workgroup): places inside the
    // expert for each wave, after the segments before this one, and the tiles before it
    const int e = threadIdx.x;
    int rows = 0;
    if (e < n) {
        int place = 0;
        if (a.segments > 1) {
#pragma unroll 8
            for (int s = 0; s < a.segments; ++s) {
                const int c = a.counts[(int64_t)s * n + e];
                rows += c;
                place += s < (int)blockIdx.x ? c : 0;
            }
        }
        for (int w = 0; w < waves; ++w) {
            const int c = counts[w * n + e];
            counts[w * n + e] = place;
            place += c;
        }
        if (a.segments == 1) rows = place;
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
    for (int w = 0; w < waves; ++w) {
        if (w < wave) before += scan[w];
        all += scan[w];
    }
    if (e < n) {
        first[e] = before * a.rows;
        // each workgroup writes some of the tiles
        for (int k = blockIdx.x; k < tiles; k += gridDim.x) a.tiles[before + k] = {e, min(a.rows, rows - k * a.rows)};
    }
    if (blockIdx.x == 0)
        for (int k = all + threadIdx.x; k < a.most; k += blockDim.x) a.tiles[k] = {0, 0};
    __syncthreads();
    walk([&](int k, int p, uint64_t m) {
        if (p < hi) {
            const int at = first[k] + mine[k] + __popcll(m & ((1ull << lane) - 1));
            a.pair[at] = p;
            a.token[at] = p / a.top;
        }
        if (p < hi && __builtin_ctzll(m) == lane) mine[k] += __popcll(m);
    });
}

static_assert(kMaxExperts + 1 <= 64 * kPlanWaves, "a thread for every expert");

hipError_t launch_experts_plan(const int *ids, void *plan, int pairs, int top, int E, hipStream_t st) {
    if (pairs <= kSelfPairs) return hipSuccess;
    const Plan p = plan_at(plan, pairs, E);
    const int rows = tile_rows(pairs, E);
    PlanArgs a = {ids, const_cast<Tile *>(p.tiles), const_cast<int *>(p.pair), const_cast<int *>(p.token),
                  const_cast<int *>(p.counts), pairs, top, E, rows, (int)max_tiles(pairs, E, rows),
                  32 - __builtin_clz((unsigned)E), (int)plan_segment(pairs), (int)plan_segments(pairs)};
    void *args[] = {(void *)&a};
    if (a.segments > 1) {
        const hipError_t e = hipLaunchKernel((const void *)k_experts_count, dim3((unsigned)a.segments), dim3(256), args,
                                             (size_t)(E + 1) * 4, st);
        if (e != hipSuccess) return e;
    }
    // a wave for every 64 pairs and for every 64 experts, 16 at most
    const int want = (a.segment + 63) / 64, least = (E + 64) / 64;
    const int waves = want < least ? least : want < kPlanWaves ? want : kPlanWaves;
    const size_t lds = (size_t)((waves + 1) * (E + 1) + waves) * 4;           // 35 KB at most
    const int each = (want + waves - 1) / waves;
    const void *k = each <= 1   ? (const void *)k_experts_plan<1>
                    : each <= 2 ? (const void *)k_experts_plan<2>
                                : (const void *)k_experts_plan<-16>;
    return hipLaunchKernel(k, dim3((unsigned)a.segments), dim3((unsigned)(64 * waves)), args, lds, st);
}

// ---------------------------------------------------------------------------
// out[t] = residual[t] + sum_j weights[t][j] y[t top + j], f32, in the order of j,
// the residual last; one rounding to the rows' type.  Bound by memory (4096 tokens of 8
// rows of 2048, bf16 out: 45 us, 6.7 TB/s).
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
