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

// Rows of a tile: what one workgroup of a product takes of an expert's rows.
constexpr int kFewRows = 8, kNarrowRows = 32, kFullRows = 128;

inline int tile_rows(int64_t pairs, int64_t experts) {
    const int64_t each = pairs / experts;
    return each < 8 ? kFewRows : each < 64 ? kNarrowRows : kFullRows;
}

// Most tiles that `pairs` rows in experts + 1 groups (the last: pairs without
// an expert) can make.
inline int64_t max_tiles(int64_t pairs, int64_t experts, int rows) {
    const int64_t a = pairs / rows + experts + 1;
    return a < pairs ? a : pairs;
}

struct Tile {
    int expert;                 // E: pairs without an expert, whose rows are zeros
    int start, count;           // its pairs: order[start .. start + count)
    int unused;
};

// The plan in memory: [1 int: number of tiles, padded to 16 bytes][tiles][pairs
// sorted by expert][their tokens].
struct Plan {
    const int *count;
    const Tile *tiles;
    const int *pair, *token;
};

inline int64_t plan_bytes(int64_t pairs, int64_t experts) {
    return 16 + 16 * max_tiles(pairs, experts, tile_rows(pairs, experts)) + 8 * pairs;
}

inline Plan plan_at(const void *plan, int64_t pairs, int64_t experts) {
    const char *p = static_cast<const char *>(plan);
    const int64_t tiles = 16 * max_tiles(pairs, experts, tile_rows(pairs, experts));
    const int *order = reinterpret_cast<const int *>(p + 16 + tiles);
    return {reinterpret_cast<const int *>(p), reinterpret_cast<const Tile *>(p + 16), order, order + pairs};
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
    int quads;                  // F / 4
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
};

// The rows of one tile, for the matrix-instruction kernels.
struct TileRows {
    const int *pair, *src;      // output rows and activation rows of the tile's rows
    uint32_t x_bytes;
    int nt;                     // which columns of the output
};

// Tile `chunk` of the plan and where its rows are.
__device__ __forceinline__ Tile expert_tile(const ExpertArgs &a, int chunk, int nt, TileRows &rows) {
    Tile t = a.plan.tiles[chunk];
    t.expert = uniform(t.expert);
    t.start = uniform(t.start);
    t.count = uniform(t.count);
    rows = {a.plan.pair + t.start, (a.x_per_pair ? a.plan.pair : a.plan.token) + t.start, a.x_bytes, nt};
    return t;
}

// Zeros in the workgroup's columns of pairs without an expert.
__device__ __forceinline__ void zero_tile(const ExpertArgs &a, const Tile &t, const TileRows &rows, int columns) {
    const int n0 = rows.nt * columns, n = min(columns, a.N - n0);
    for (int i = threadIdx.x; i < t.count * n; i += blockDim.x) {
        const int r = i / n;
        a.y[(int64_t)rows.pair[r] * a.N + n0 + (i - r * n)] = 0.0f;
    }
}

}  // namespace qmm
