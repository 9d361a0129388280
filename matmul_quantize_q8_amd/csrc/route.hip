// Routing to experts: the top-k experts of each token's logits, their weights.
// One wave a token; every lane holds the experts lane, lane + 64, ..
//
// What orders the experts is f64: scores that f32 would hold alike keep the
// order of the formula, and without a bias the order is that of the logits
// themselves, which softmax and sigmoid keep.  Scores are compared as unsigned
// keys: 0 for an expert that cannot be chosen (any more), NaN above all.
//
// Bound by latency for a few tokens (a chain of top_k reductions over the wave) and
// by the vector unit for many (an f64 exponential and a division an expert where a
// bias or groups need every score, nothing of the kind where the logits alone
// decide).  So a reduction is of 32 bits, in lane exchanges that are operand
// modifiers, and goes on to the low half and to the indices only where the high
// halves of several lanes are equal (8192 tokens, 4 of 8 groups of 32, 8 experts:
// 28.7 -> 17.7 us; one token, 8 of 128: 7.2 -> 3.9).
#include "kv_layout.h"
#include "moe.h"

namespace qmm {

constexpr int kRouteWaves = 4;

__device__ __forceinline__ uint64_t order_key(double v) {
    if (v != v) return ~0ull;
    const uint64_t u = __builtin_bit_cast(uint64_t, v + 0.0);       // -0 as +0
    return (u >> 63) ? ~u : u | (1ull << 63);
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
// Maximum over the wave, the same in every lane.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = max(v, dpp_u32<kDppQuadXor1>(v));
    v = max(v, dpp_u32<kDppQuadXor2>(v));
    v = max(v, dpp_u32<kDppHalfRowMirror>(v));
    v = max(v, dpp_u32<kDppRowRor8>(v));
    const uint32_t a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16);
    const uint32_t c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
    return max(max(a, b), max(c, d));
}
// The lanes that hold the largest key; none if all are 0.  (No key but 0 has a high half of 0.)
__device__ __forceinline__ uint64_t largest(uint64_t key) {
    const uint32_t hi = (uint32_t)(key >> 32), top = wave_max(hi);
    if (top == 0) return 0;
    uint64_t lanes = __ballot(hi == top);
    if (lanes & (lanes - 1)) {
        const uint32_t lo = hi == top ? (uint32_t)key : 0u, low = wave_max(lo);
        lanes = __ballot(hi == top && lo == low);
    }
    return lanes;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, kWave);
    return v;
}
__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v = fmax(v, __shfl_xor(v, m, kWave));
    return v;
}

// NE experts a lane; SCORES: every expert's score is needed, not its logit alone.
template <int RT, int NE, bool SCORES>
__global__ __launch_bounds__(kWave * kRouteWaves) void k_route(RouteArgs a) {
    extern __shared__ double lds[];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
    if (t >= a.T) return;                                 // the whole wave; no barrier follows
    const int64_t row = t * a.stride;
    const double inf = __builtin_inf();

    double x[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int e = lane + kWave * i;
        x[i] = e < a.E ? (double)load1<RT>(a.logits, row + e) : -inf;
    }
    // softmax over all of the row: its maximum and its sum
    double top = -inf, all = 1.0;
    if (a.softmax && (SCORES || !a.renorm)) {
#pragma unroll
        for (int i = 0; i < NE; ++i) top = fmax(top, x[i]);
        top = wave_max(top);
        all = 0.0;
#pragma unroll
        for (int i = 0; i < NE; ++i)
            if (x[i] != -inf) all += exp(x[i] - top);
        all = wave_sum(all);
    }
    uint64_t key[NE];
    if constexpr (!SCORES) {
#pragma unroll
        for (int i = 0; i < NE; ++i) key[i] = x[i] == -inf ? 0 : order_key(x[i]);
    } else {
        double c[NE];
        const double share = 1.0 / all;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int e = lane + kWave * i;
            c[i] = -inf;
            if (x[i] != -inf) {
                c[i] = a.softmax ? exp(x[i] - top) * share : 1.0 / (1.0 + exp(-x[i]));
                if (a.bias != nullptr) c[i] += (double)a.bias[e];
            }
            key[i] = c[i] == -inf ? 0 : order_key(a.bias == nullptr ? x[i] : c[i]);
        }
        if (a.groups > 1) {
            // 64 / groups lanes (a power of two) a group: the sum of its group_top largest scores
            double *scores = lds + (int64_t)wave * a.E;
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                const int e = lane + kWave * i;
                if (e < a.E) scores[e] = c[i];
            }
            wait_lds_reads();                             // this wave's own writes
            const int per = a.E / a.groups, sub = kWave >> a.group_bits;      // 2^group_bits >= groups
            const int group = lane / sub, from = lane & (sub - 1);
            double first = -inf, second = -inf;
            bool nan = false;
            if (group < a.groups) {
                for (int k = from; k < per; k += sub) {
                    const double v = scores[group * per + k];
                    nan |= v != v;
                    second = fmax(second, fmin(first, v));
                    first = fmax(first, v);
                }
            }
            for (int m = 1; m < sub; m <<= 1) {
                const double f = __shfl_xor(first, m, kWave), s = __shfl_xor(second, m, kWave);
                nan |= __shfl_xor((int)nan, m, kWave) != 0;
                second = fmax(fmax(second, s), fmin(first, f));
                first = fmax(first, f);
            }
            const double sum = nan ? __builtin_nan("") : a.group_top == 2 && second != -inf ? first + second : first;
            uint64_t mine = group < a.groups && from == 0 && sum != -inf ? order_key(sum) : 0;
            uint64_t keep = 0;                            // the first lanes of the groups that stay
            for (int k = 0; k < a.kept; ++k) {
                const uint64_t lanes = largest(mine);
                if (lanes == 0) break;
                const int g = __builtin_ctzll(lanes);     // of equal ones the lowest
                keep |= 1ull << g;
                if (lane == g) mine = 0;
            }
            const uint32_t inverse = (1u << 20) / (uint32_t)per + 1;          // e / per = e inverse >> 20 for e < 512
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                const int e = lane + kWave * i;
                const int g = (int)(((uint32_t)e * inverse) >> 20);
                if (e < a.E && !((keep >> (g * sub)) & 1)) key[i] = 0;
            }
        }
    }
    // the largest key, at its lowest index, a.top times; lane j keeps the j-th
    int id = -1;
    for (int j = 0; j < a.top; ++j) {
        uint64_t best = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const bool more = key[i] > best;
            best = more ? key[i] : best;
            at = more ? lane + kWave * i : at;
        }
        const uint64_t lanes = largest(best);
        if (lanes == 0) break;
        int e = __builtin_amdgcn_readlane(at, __builtin_ctzll(lanes));
        if (lanes & (lanes - 1)) e = (int)~wave_max((lanes >> lane) & 1 ? ~(uint32_t)at : 0u);
#pragma unroll
        for (int i = 0; i < NE; ++i)
            if (e == lane + kWave * i) key[i] = 0;
        if (lane == j) id = e;
    }
    // weights.  Renormalised ones are computed relative to the largest chosen
    // logit: chosen scores that all round to 0 keep their shares.
    const double l = id >= 0 ? (double)load1<RT>(a.logits, row + id) : -inf;
    double w = 0.0;
    if (a.renorm) {
        const double m = wave_max(l);
        if (id >= 0) {
            if (a.softmax)
                w = exp(l - m);
            else
                w = m < 0.0 ? exp(l - m) / (1.0 + exp(l)) : 1.0 / (1.0 + exp(-l));
        }
        const double sum = wave_sum(w);
        if (id >= 0) w /= sum;
    } else if (id >= 0) {
        w = a.softmax ? exp(l - top) / all : 1.0 / (1.0 + exp(-l));
    }
    if (lane < a.top) {
        a.ids[t * a.top + lane] = id;
        a.weights[t * a.top + lane] = (float)(w * (double)a.scale);
    }
}

template <int RT, bool SCORES>
static const void *kernel(int E) {
    return E <= 64    ? (const void *)k_route<RT, 1, SCORES>
           : E <= 128 ? (const void *)k_route<RT, 2, SCORES>
           : E <= 256 ? (const void *)k_route<RT, 4, SCORES>
                      : (const void *)k_route<RT, 8, SCORES>;
}

template <int RT>
static hipError_t launch(RouteArgs a, hipStream_t st) {
    const void *k = a.bias != nullptr || a.groups > 1 ? kernel<RT, true>(a.E) : kernel<RT, false>(a.E);
    while ((1 << a.group_bits) < a.groups) ++a.group_bits;
    const size_t lds = a.groups > 1 ? (size_t)kRouteWaves * a.E * 8 : 0;      // 16 KB at most
    void *args[] = {(void *)&a};
    return hipLaunchKernel(k, dim3((unsigned)((a.T + kRouteWaves - 1) / kRouteWaves)), dim3(kWave * kRouteWaves), args,
                           lds, st);
}

hipError_t launch_route(int rt, const RouteArgs &a, hipStream_t st) {
    return rt == R_F32 ? launch<R_F32>(a, st) : rt == R_F16 ? launch<R_F16>(a, st) : launch<R_BF16>(a, st);
}

}  // namespace qmm
