// Routing to experts: the top-k experts of each token's logits, their weights.
// One wave a token; every lane holds the experts lane, lane + 64, ..
//
// What orders the experts is f64: scores that f32 would hold alike keep the
// order of the formula, and without a bias the order is that of the logits
// themselves, which softmax and sigmoid keep.  Scores are compared as unsigned
// keys: 0 for an expert that cannot be chosen (any more), NaN above all.
#include "kv_layout.h"
#include "moe.h"

namespace qmm {

constexpr int kRouteWaves = 4;

__device__ __forceinline__ uint64_t order_key(double v) {
    if (v != v) return ~0ull;
    const uint64_t u = __builtin_bit_cast(uint64_t, v + 0.0);       // -0 as +0
    return (u >> 63) ? ~u : u | (1ull << 63);
}

__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) {
        const uint64_t o = __shfl_xor((unsigned long long)v, m, kWave);
        v = o > v ? o : v;
    }
    return v;
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
__device__ __forceinline__ int wave_min(int v) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v = min(v, __shfl_xor(v, m, kWave));
    return v;
}

// NE experts a lane.
template <int RT, int NE>
__global__ __launch_bounds__(kWave * kRouteWaves) void k_route(RouteArgs a) {
    extern __shared__ double lds[];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
    if (t >= a.T) return;                                 // the whole wave; no barrier follows
    const int64_t row = t * a.stride;
    const double inf = __builtin_inf();

    double x[NE];
    bool there[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int e = lane + kWave * i;
        x[i] = e < a.E ? (double)load1<RT>(a.logits, row + e) : -inf;
        there[i] = x[i] != -inf;
    }
    // softmax over all of the row: its maximum and its sum
    double top = -inf, all = 1.0;
    if (a.softmax) {
#pragma unroll
        for (int i = 0; i < NE; ++i) top = fmax(top, x[i]);
        top = wave_max(top);
        all = 0.0;
#pragma unroll
        for (int i = 0; i < NE; ++i)
            if (there[i]) all += exp(x[i] - top);
        all = wave_sum(all);
    }
    uint64_t key[NE];
    if (a.bias == nullptr && a.groups == 1) {
#pragma unroll
        for (int i = 0; i < NE; ++i) key[i] = there[i] ? order_key(x[i]) : 0;
    } else {
        double c[NE];
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int e = lane + kWave * i;
            c[i] = -inf;
            if (there[i]) c[i] = a.softmax ? exp(x[i] - top) / all : 1.0 / (1.0 + exp(-x[i]));
            if (a.bias != nullptr && there[i]) c[i] += (double)a.bias[e];
            key[i] = c[i] == -inf ? 0 : order_key(a.bias == nullptr ? x[i] : c[i]);
        }
        if (a.groups > 1) {
            // a lane a group: the sum of its group_top largest scores
            double *scores = lds + (int64_t)wave * a.E;
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                const int e = lane + kWave * i;
                if (e < a.E) scores[e] = c[i];
            }
            wait_lds_reads();                             // this wave's own writes
            const int per = a.E / a.groups;
            uint64_t mine = 0;
            if (lane < a.groups) {
                double first = -inf, second = -inf;
                bool nan = false, any = false;
                for (int k = 0; k < per; ++k) {
                    const double v = scores[lane * per + k];
                    nan |= v != v;
                    any |= v != -inf;
                    second = fmax(second, fmin(first, v));
                    first = fmax(first, v);
                }
                const double sum = nan ? __builtin_nan("") : a.group_top == 2 && second != -inf ? first + second : first;
                mine = any ? order_key(sum) : 0;
            }
            int before = 0;                               // groups that come before the lane's
            for (int g = 0; g < a.groups; ++g) {
                const uint64_t o = __shfl((unsigned long long)mine, g, kWave);
                before += o > mine || (o == mine && g < lane);
            }
            const uint64_t keep = __ballot(lane < a.groups && mine != 0 && before < a.kept);
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                const int e = lane + kWave * i;
                if (e < a.E && !((keep >> (e / per)) & 1)) key[i] = 0;
            }
        }
    }
    // the largest key, at its lowest index, a.top times; lane j keeps the j-th
    int id = -1;
    for (int j = 0; j < a.top; ++j) {
        uint64_t best = 0;
#pragma unroll
        for (int i = 0; i < NE; ++i) best = key[i] > best ? key[i] : best;
        best = wave_max(best);
        if (best == 0) break;
        int at = 0x7fffffff;
#pragma unroll
        for (int i = NE - 1; i >= 0; --i)
            if (key[i] == best) at = lane + kWave * i;
        at = wave_min(at);
#pragma unroll
        for (int i = 0; i < NE; ++i)
            if (at == lane + kWave * i) key[i] = 0;
        if (lane == j) id = at;
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

template <int RT>
static hipError_t launch(RouteArgs a, hipStream_t st) {
    const void *k = a.E <= 64    ? (const void *)k_route<RT, 1>
                    : a.E <= 128 ? (const void *)k_route<RT, 2>
                    : a.E <= 256 ? (const void *)k_route<RT, 4>
                    : a.E <= 512 ? (const void *)k_route<RT, 8>
                                 : (const void *)k_route<RT, 16>;
    const size_t lds = a.groups > 1 ? (size_t)kRouteWaves * a.E * 8 : 0;      // 32 KB at most
    void *args[] = {(void *)&a};
    return hipLaunchKernel(k, dim3((unsigned)((a.T + kRouteWaves - 1) / kRouteWaves)), dim3(kWave * kRouteWaves), args,
                           lds, st);
}

hipError_t launch_route(int rt, const RouteArgs &a, hipStream_t st) {
    return rt == R_F32 ? launch<R_F32>(a, st) : rt == R_F16 ? launch<R_F16>(a, st) : launch<R_BF16>(a, st);
}

}  // namespace qmm
