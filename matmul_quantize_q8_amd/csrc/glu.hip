// Gated activation and quantization of rows: xq = Q8(act(gate) up).
// Bound by memory: 4 or 8 bytes read and about one written for every value, sixteen
// bytes a lane (32768 rows of 768 f32 to Q8_0: 43.8 us in a loop over three inputs,
// 5.2 TB/s; 128 rows 2.3 us).
#include "moe.h"
#include "q8_rows.h"

namespace qmm {

// In f32, each within a few units of its last place, but for the GELUs' far negative
// tail: e^(-z^2) with z^2 < 104 of a z rounded to 2^-24 of itself is off by up to 2 z^2
// 2^-24 = 2^-16 of itself.  The result is held in 8 bits.
template <int ACT>
__device__ __forceinline__ float activation(float g) {
    if constexpr (ACT == G_SILU) return g / (1.0f + expf(-g));
    if constexpr (ACT == G_GELU) return 0.5f * g * erfcf(-0.70710678118654752f * g);
    // 0.5 (1 + tanh z) = 1 / (1 + e^(-2z))
    const float z2 = 1.5957691216057308f * (g + 0.044715f * g * g * g);
    return g / (1.0f + expf(-z2));
}

// Gates below this have an activation of less than 2^-120, where e^-g and e^(-2z) overflow
// soon and erfc falls below the normal values: activation() is 0 or coarse there while the
// activation, and still more its product with `up`, is a number that f32 holds.
template <int ACT> constexpr float kFarGate = ACT == G_SILU ? -88.0f : ACT == G_GELU ? -13.0f : -10.0f;

// act(g) u there: g e^z u, z = g or the 2z above (1 + e^z rounds to 1), or with erfc's
// scaled form g/2 erfcx(-g / sqrt 2) e^(-g^2 / 2) u; e^z in two halves around u, so that
// neither is far below the normal values before the product is.
template <int ACT>
__device__ __forceinline__ float far_gated(float g, float u) {
    float s = g, z = g;
    if constexpr (ACT == G_GELU) {
        s = 0.5f * g * erfcxf(-0.70710678118654752f * g);
        z = -0.5f * g * g;
    }
    if constexpr (ACT == G_GELU_TANH) z = 1.5957691216057308f * (g + 0.044715f * g * g * g);
    const float h = expf(0.5f * z);
    return s * h * u * h;
}

constexpr int kGluThreads = 256;
constexpr int64_t kGluGrid = 1 << 22;          // workgroups of a launch: a grid holds 2^32 threads

template <int RT, int FMT, int ACT>
__global__ __launch_bounds__(kGluThreads) void k_glu(GluArgs a) {
    constexpr int V = row_values(RT);                     // 16 bytes a lane
    const int64_t row_bytes = (int64_t)(a.pieces / (act_values(FMT) / V)) * act_bytes(FMT);
    const int64_t all = a.rows * a.pieces;
    for (int64_t base = (int64_t)blockIdx.x * kGluThreads; base < all; base += (int64_t)gridDim.x * kGluThreads) {
        const int64_t row0 = base / a.pieces;
        const uint32_t at = (uint32_t)(base - row0 * a.pieces) + threadIdx.x;
        const int64_t row = row0 + at / (uint32_t)a.pieces;
        const int c = (int)(at % (uint32_t)a.pieces);
        if (row >= a.rows) continue;
        float g[V], u[V], v[V];
        load_row<RT, V>(a.gate, row * a.gs + V * c, g);
        load_row<RT, V>(a.up, row * a.us + V * c, u);
        uint32_t least = 0;                               // the bits of negative numbers grow as they fall
#pragma unroll
        for (int k = 0; k < V; ++k) least = max(least, __builtin_bit_cast(uint32_t, g[k]));
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = activation<ACT>(g[k]) * u[k];
        if (__builtin_expect(least > __builtin_bit_cast(uint32_t, kFarGate<ACT>), 0)) {
            // value by value, the arrays going round: little code beside the usual path's
#pragma unroll 1
            for (int i = 0; i < V; ++i) {
                const float g0 = g[0], u0 = u[0], v0 = v[0];
#pragma unroll
                for (int k = 0; k + 1 < V; ++k) g[k] = g[k + 1], u[k] = u[k + 1], v[k] = v[k + 1];
                g[V - 1] = g0, u[V - 1] = u0, v[V - 1] = g0 < kFarGate<ACT> ? far_gated<ACT>(g0, u0) : v0;
            }
        }
        store_quantized<FMT, V>(a.xq + row * row_bytes, c, v);
    }
}

template <int RT, int FMT>
static hipError_t launch(int act, GluArgs a, hipStream_t st) {
    const void *k = act == G_SILU   ? (const void *)k_glu<RT, FMT, G_SILU>
                    : act == G_GELU ? (const void *)k_glu<RT, FMT, G_GELU>
                                    : (const void *)k_glu<RT, FMT, G_GELU_TANH>;
    const int64_t grid = (a.rows * a.pieces + kGluThreads - 1) / kGluThreads;
    void *args[] = {(void *)&a};
    return hipLaunchKernel(k, dim3((unsigned)(grid < kGluGrid ? grid : kGluGrid)), dim3(kGluThreads), args, 0, st);
}

hipError_t launch_glu(int rt, int fmt, int act, const GluArgs &a, hipStream_t st) {
    switch (rt * 2 + fmt) {
        case R_F32 * 2 + A_Q8_0: return launch<R_F32, A_Q8_0>(act, a, st);
        case R_F32 * 2 + A_Q8_K: return launch<R_F32, A_Q8_K>(act, a, st);
        case R_F16 * 2 + A_Q8_0: return launch<R_F16, A_Q8_0>(act, a, st);
        case R_F16 * 2 + A_Q8_K: return launch<R_F16, A_Q8_K>(act, a, st);
        case R_BF16 * 2 + A_Q8_0: return launch<R_BF16, A_Q8_0>(act, a, st);
        case R_BF16 * 2 + A_Q8_K: return launch<R_BF16, A_Q8_K>(act, a, st);
    }
    return hipErrorInvalidValue;
}

}  // namespace qmm
