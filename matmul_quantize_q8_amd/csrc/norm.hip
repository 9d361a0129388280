// Residual addition, root-mean-square norm and quantization of rows:
//   s = round(x + residual),  y = s (offset + weight) / sqrt(mean(s^2) + eps),  xq = Q8(y)
// One pass over memory: a workgroup holds its row in registers between the sum
// of squares and the norm.  The sum of squares and the norm's factors are f64
// (a sum of f32 squares overflows from 1.8e19 on; f64 also makes every y the
// exact one rounded once, so the codes do not depend on the order of the sum).
#include "moe.h"
#include "q8_rows.h"

namespace qmm {

// Sum over the workgroup, the same in every thread; `part` holds a value for
// each wave.
__device__ __forceinline__ double workgroup_sum(double v, double *part) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, kWave);
    const int wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    if ((threadIdx.x & 63) == 0) part[wave] = v;
    __syncthreads();
    double s = 0.0;
    for (int i = 0; i < waves; ++i) s += part[i];
    return s;
}

template <int RT>
__device__ __forceinline__ float4 norm_input(const NormArgs &a, int64_t t, int c) {
    float4 v = load4<RT>(a.x, t * a.xs + 4 * c);
    if (a.residual != nullptr) {
        const float4 r = load4<RT>(a.residual, t * a.rs + 4 * c);
        v = make_float4(v.x + r.x, v.y + r.y, v.z + r.z, v.w + r.w);
        if constexpr (RT != R_F32) {                      // the norm is of what the stream holds
            const uint32_t lo = pack2<RT>(v.x, v.y), hi = pack2<RT>(v.z, v.w);
            v = RT == R_F16 ? make_float4(f16_bits_to_f32(lo), f16_bits_to_f32(lo >> 16), f16_bits_to_f32(hi),
                                          f16_bits_to_f32(hi >> 16))
                            : make_float4(__builtin_bit_cast(float, lo << 16),
                                          __builtin_bit_cast(float, lo & 0xffff0000u),
                                          __builtin_bit_cast(float, hi << 16),
                                          __builtin_bit_cast(float, hi & 0xffff0000u));
        }
    }
    return v;
}

__device__ __forceinline__ double square_sum(float4 v) {
    return fma((double)v.x, (double)v.x, fma((double)v.y, (double)v.y, fma((double)v.z, (double)v.z,
                                                                            (double)v.w * (double)v.w)));
}

template <int RT, int FMT>
__device__ __forceinline__ void norm_output(const NormArgs &a, int64_t t, int c, float4 v, double r, uint8_t *xq) {
    const float4 w = a.weight == nullptr ? make_float4(1.0f, 1.0f, 1.0f, 1.0f) : load4<R_F32>(a.weight, 4 * c);
    const double o = a.offset;
    const float4 y = make_float4((float)((double)v.x * r * (o + (double)w.x)), (float)((double)v.y * r * (o + (double)w.y)),
                                 (float)((double)v.z * r * (o + (double)w.z)), (float)((double)v.w * r * (o + (double)w.w)));
    if (a.y != nullptr) store4<RT>(a.y, t * a.ys + 4 * c, y);
    store_quantized<FMT>(xq, c, y);
}

// Workgroups of a launch: a grid holds 2^32 threads.
constexpr int64_t kMaxGrid = 1 << 20;

// V pieces of four values a thread; longer rows (V = 0) are walked twice.
template <int RT, int FMT, int V>
__global__ __launch_bounds__(1024) void k_rms_norm(NormArgs a) {
    __shared__ double part[16];
    const int n = (int)(a.K / 4), step = blockDim.x;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        uint8_t *xq = a.xq + t * (a.K / act_values(FMT)) * act_bytes(FMT);
        double s = 0.0;
        float4 v[V ? V : 1];
        if constexpr (V > 0) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = threadIdx.x + i * step;
                if (c < n) v[i] = norm_input<RT>(a, t, c);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = threadIdx.x + i * step;
                if (c >= n) continue;
                if (a.sum != nullptr) store4<RT>(a.sum, t * a.ss + 4 * c, v[i]);
                s += square_sum(v[i]);
            }
        } else {
            for (int c = threadIdx.x; c < n; c += step) s += square_sum(norm_input<RT>(a, t, c));
        }
        const double r = 1.0 / sqrt(workgroup_sum(s, part) / (double)a.K + (double)a.eps);
        if constexpr (V > 0) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = threadIdx.x + i * step;
                if (c < n) norm_output<RT, FMT>(a, t, c, v[i], r, xq);
            }
        } else {
            for (int c = threadIdx.x; c < n; c += step) {
                const float4 u = norm_input<RT>(a, t, c);
                if (a.sum != nullptr) store4<RT>(a.sum, t * a.ss + 4 * c, u);
                norm_output<RT, FMT>(a, t, c, u, r, xq);
            }
        }
        __syncthreads();                                  // `part` is free again
    }
}

template <int RT, int FMT>
static hipError_t launch(NormArgs a, hipStream_t st) {
    const int64_t n = a.K / 4;
    // short rows: the fewest whole waves that hold a row; long ones: 1024 threads
    const int threads = n <= 1024 ? (int)((n + 63) / 64 * 64) : 1024;
    const void *k = n <= 1024   ? (const void *)k_rms_norm<RT, FMT, 1>
                    : n <= 4096 ? (const void *)k_rms_norm<RT, FMT, 4>
                                : (const void *)k_rms_norm<RT, FMT, 0>;
    void *args[] = {(void *)&a};
    return hipLaunchKernel(k, dim3((unsigned)(a.T < kMaxGrid ? a.T : kMaxGrid)), dim3((unsigned)threads), args, 0, st);
}

hipError_t launch_rms_norm(int rt, int fmt, const NormArgs &a, hipStream_t st) {
    switch (rt * 2 + fmt) {
        case R_F32 * 2 + A_Q8_0: return launch<R_F32, A_Q8_0>(a, st);
        case R_F32 * 2 + A_Q8_K: return launch<R_F32, A_Q8_K>(a, st);
        case R_F16 * 2 + A_Q8_0: return launch<R_F16, A_Q8_0>(a, st);
        case R_F16 * 2 + A_Q8_K: return launch<R_F16, A_Q8_K>(a, st);
        case R_BF16 * 2 + A_Q8_0: return launch<R_BF16, A_Q8_0>(a, st);
        case R_BF16 * 2 + A_Q8_K: return launch<R_BF16, A_Q8_K>(a, st);
    }
    return hipErrorInvalidValue;
}

}  // namespace qmm
