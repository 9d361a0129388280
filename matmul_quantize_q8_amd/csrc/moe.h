// What the mixture-of-experts kernels share: the plan that sorts (token, slot)
// pairs by expert, and the arguments of the experts' products.
#pragma once

#include "qmm_device.h"

namespace qmm {

constexpr int kMaxExperts = 512;
constexpr int kMaxTop = 64;
constexpr int64_t kMaxPairs = int64_t(1) << 26;

// Calls of up to this many pairs (one for each lane of a wave) need no plan:
// every workgroup of the product finds its rows from the ids by itself.
constexpr int64_t kSelfPairs = kWave;

// Rows of a tile of the plan: in what steps an expert's rows are cut, for products of
// any format and width.  Tiles of 128 are what the prefill matmul's workgroups take, or
// two of 64 or four of 32; all but those of 128 stream the weights (experts_stream.h).
// us, 128 experts of 1536 x 2048, 8 a token, tiles of 16 / 32 / 64 / 128 (of 16, and of
// 32 from 64 rows an expert on, in workgroups of four waves):
//   rows an expert   25                     32                     64                    128
//   Q4_0             90 / 89 / 96 / 127     105 / 102 / 108 / 133  - / 151 / 155 / 162   - / 263 / 256 / 231
//   Q8_0             131 / 119 / 122 / 147  154 / 130 / 132 / 157  - / 207 / 187 / 185   - / 347 / 299 / 251
//   Q5_1             156 / 130 / 139 / 175  180 / 146 / 157 / 180  - / 242 / 232 / 214   - / 426 / 390 / 305
//   Q4_K             91 / 70 / 75 / 86      105 / 81 / 80 / 95     - / 125 / 118 / 150   - / 210 / 193 / 225
// Below 4096 pairs the rule stays with 32: whole workgroups of 128 rows were too few there
// (8 experts of 1024 x 1024, 1400 pairs, Q4_0: 14.7 us in tiles of 32, 22 of 128).  Products
// have come to take a step of 128 in parts where columns are few, and with that steps of 128
// are the faster ones at 128 rows an expert and more, most of all of wide experts (2 of 8, in
// steps of 32 / 128, Q4_0, Q8_0, Q4_K, Q6_K: of 1024 x 1024, 1536 tokens 25 / 23, 30 / 23, 18 / 16,
// 33 / 26; of 14336 x 4096, 1024 tokens 546 / 399, 706 / 446, 415 / 360, 780 / 659).
constexpr int kFewRows = 16, kNarrowRows = 32, kHalfRows = 64, kFullRows = 128;

inline int tile_rows(int64_t pairs, int64_t experts) {
    const int64_t each = pairs / experts;
    return each < 20 ? kFewRows : each < 64 || pairs < 4096 ? kNarrowRows : kFullRows;
}

// Most tiles that `pairs` rows in experts + 1 groups (the last: pairs without
// an expert) can make.
inline int64_t max_tiles(int64_t pairs, int64_t experts, int rows) {
    const int64_t a = pairs / rows + experts + 1;
    return a < pairs ? a : pairs;
}

struct Tile {
    int expert;                 // E: pairs without an expert, whose rows are zeros
    int count;                  // its rows; 0: no tile
};

// Pairs that one workgroup of the plan sorts: all of them up to 2048, then 1024, or
// so many that there are at most 256 such segments.
inline int64_t plan_segment(int64_t pairs) {
    if (pairs <= 2048) return pairs;
    const int64_t s = (pairs + 255) / 256;
    return s <= 1024 ? 1024 : (s + 63) / 64 * 64;
}
inline int64_t plan_segments(int64_t pairs) {
    const int64_t s = plan_segment(pairs);
    return (pairs + s - 1) / s;
}

// The plan in memory: [most tiles][most tiles * rows pairs][their tokens][segments][E + 1
// pairs of each expert, where there are several segments].  A tile's rows are at its
// own place, so a workgroup loads them beside the tile.
struct Plan {
    const Tile *tiles;
    const int *pair, *token, *counts;
};

// Never less for more pairs, so that a buffer serves smaller calls too: room for the counts of 256
// segments wherever segments get longer (their number then falls where pairs grow).
inline int64_t plan_bytes(int64_t pairs, int64_t experts) {
    const int rows = tile_rows(pairs, experts);
    const int64_t most = (pairs + 1023) / 1024, segments = most < 256 ? most : 256;
    return max_tiles(pairs, experts, rows) * (8 + 8 * rows) + (plan_segments(pairs) > 1 ? segments * (experts + 1) * 4 : 0);
}

inline Plan plan_at(const void *plan, int64_t pairs, int64_t experts) {
    const int rows = tile_rows(pairs, experts);
    const int64_t tiles = max_tiles(pairs, experts, rows);
    const Tile *t = static_cast<const Tile *>(plan);
    const int *pair = reinterpret_cast<const int *>(t + tiles);
    return {t, pair, pair + tiles * rows, pair + 2 * tiles * rows};
}

// A product over experts.
struct ExpertArgs {
    const uint8_t *w;           // expert e's matrix at w + e * stride
    int64_t stride;
    const uint8_t *x;           // rows of activation blocks
    uint32_t x_bytes;           // all of them
    int x_per_pair;             // a row for each pair, otherwise for each token
    float *y;                   // [pairs][N]
    const int *ids;             // [pairs]; with it instead of the plan: kSelfPairs at most
    Plan plan;
    int pairs, top, E, N, nb;   // nb: blocks of a row
    int x_rows;                 // pairs, or tokens
    int rows;                   // rows of a tile
};

// s = round(x + residual), xq = Q8(y), y = s (offset + weight) / sqrt(mean(s^2) + eps).
struct NormArgs {
    const void *x, *residual;   // residual NULL: none
    void *sum, *y;              // either NULL: not wanted
    const float *weight;        // NULL: ones
    uint8_t *xq;
    int64_t T, xs, rs, ss, ys;  // strides in elements
    int64_t K;
    float eps, offset;
};

enum GluAct { G_SILU = 0, G_GELU = 1, G_GELU_TANH = 2 };

// xq = Q8(act(gate) up).
struct GluArgs {
    const void *gate, *up;
    uint8_t *xq;
    int64_t rows, gs, us;       // strides in elements
    int pieces;                 // of a row, 16 bytes each
};

// A token's top experts and their weights.
struct RouteArgs {
    const void *logits;
    const float *bias;          // NULL: none
    int *ids;
    float *weights;
    int64_t T, stride;
    int E, top, groups, kept, group_top;
    int softmax, renorm;
    float scale;
    int group_bits;             // set by the launch
};

// The rows of one tile, for the matrix-instruction kernels.
struct TileRows {
    const int *pair, *src;      // output rows and activation rows of the tile's rows (LDS)
    uint32_t x_bytes;
    int nt;                     // which columns of the output
};

// Rows from .. from + most - 1 of tile `chunk` of a product, into LDS tables of `most`
// entries: of the plan, or in a call without one (from 0, most a.rows) the pairs of pair
// `chunk`'s expert, if it is the first of every a.rows of them.  count: those that there
// are.  What the
// plan holds is kept inside the call's sizes: bytes that no plan of this size wrote
// give wrong rows, but no access outside the buffers.  The caller has a barrier before
// the tables are read.
__device__ __forceinline__ Tile expert_tile(const ExpertArgs &a, int chunk, int *pair, int *src, int from, int most) {
    Tile t;
    if (a.ids != nullptr) {
        const int lane = threadIdx.x & 63, id = lane < a.pairs ? a.ids[lane] : -1;
        const int e = __builtin_amdgcn_readlane(id, chunk);
        const bool none = (unsigned)e >= (unsigned)a.E;
        uint64_t m = none ? 1ull << chunk : __ballot(lane < a.pairs && id == e);
        const int before = __popcll(m & ((1ull << chunk) - 1));
        if (before % most) return {0, 0};
        m &= ~0ull << chunk;
        t = {none ? a.E : e, min((int)__popcll(m), most)};
        if (threadIdx.x < kWave && (m >> lane) & 1) {
            const int r = __popcll(m & ((1ull << lane) - 1));
            if (r < most) pair[r] = lane, src[r] = a.x_per_pair ? lane : lane / a.top;
        }
    } else {
        // loaded beside the tile: rows past its count are whatever the plan holds
        int p = 0, x = 0;
        if ((int)threadIdx.x < most) {
            const int64_t at = (int64_t)chunk * a.rows + from + threadIdx.x;
            p = a.plan.pair[at];
            x = a.x_per_pair ? p : a.plan.token[at];
        }
        t = a.plan.tiles[chunk];
        t.expert = uniform(t.expert);
        t.count = (unsigned)t.expert > (unsigned)a.E ? 0 : max(min(min(uniform(t.count), a.rows) - from, most), 0);
        p = (int)min((unsigned)p, (unsigned)a.pairs - 1), x = (int)min((unsigned)x, (unsigned)a.x_rows - 1);
        if ((int)threadIdx.x < t.count) pair[threadIdx.x] = p, src[threadIdx.x] = x;
    }
    return t;
}

// Zeros in the workgroup's columns of pairs without an expert.
__device__ __forceinline__ void zero_tile(const ExpertArgs &a, int count, const TileRows &rows, int columns) {
    const int n0 = rows.nt * columns, n = min(columns, a.N - n0);
    for (int i = threadIdx.x; i < count * n; i += blockDim.x) {
        const int r = i / n;
        a.y[(int64_t)rows.pair[r] * a.N + n0 + (i - r * n)] = 0.0f;
    }
}

// Tiles that a product's grid holds for its calls with and without a plan.
inline int64_t grid_tiles(const ExpertArgs &a) {
    return a.ids != nullptr ? a.pairs : max_tiles(a.pairs, a.E, a.rows);
}

}  // namespace qmm
