// Residual addition, root-mean-square norm and quantization of rows:
//   s = round(x + residual),  y = s (offset + weight) / sqrt(mean(s^2) + eps),  xq = Q8(y)
//
// Bound by memory: one pass, a workgroup holds its row in registers between the sum
// of squares and the norm.  Sixteen-byte loads, a few of them in flight a lane, and
// 256 threads a row of up to 8192 16-bit values, so that a compute unit has rows in
// every phase (4096 rows of 4096 bf16 with every output: 32.7 us; 1024 threads
// and eight bytes a lane 53).  Fewer rows than compute units take more threads each.
// The sum of squares and the norm's factors are f64: a sum of f32 squares overflows
// from 1.8e19 on, and every y is the exact one rounded once, so the codes do not
// depend on the order of the sum.
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

// Values V c .. of x, and of the residual; s of both.
template <int RT, int V>
__device__ __forceinline__ void norm_load(const NormArgs &a, int64_t t, int c, float (&x)[V], float (&r)[V]) {
    load_row<RT, V>(a.x, t * a.xs + V * c, x);
    if (a.residual != nullptr) load_row<RT, V>(a.residual, t * a.rs + V * c, r);
}
template <int RT, int V>
__device__ __forceinline__ void norm_add(const NormArgs &a, int64_t t, int c, float (&x)[V], const float (&r)[V]) {
    if (a.residual != nullptr) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            x[k] += r[k];
            if constexpr (RT == R_F16) x[k] = f16_bits_to_f32(f32_to_f16_bits(x[k]));        // what the stream holds
            if constexpr (RT == R_BF16) x[k] = __builtin_bit_cast(float, f32_to_bf16_bits(x[k]) << 16);
        }
    }
    if (a.sum != nullptr) store_row<RT, V>(a.sum, t * a.ss + V * c, x);
}
template <int V>
__device__ __forceinline__ double square_sum(const float (&x)[V]) {
    double s = 0.0;
#pragma unroll
    for (int k = 0; k < V; ++k) s = fma((double)x[k], (double)x[k], s);
    return s;
}
template <int RT, int FMT, int V>
__device__ __forceinline__ void norm_output(const NormArgs &a, int64_t t, int c, const float (&x)[V], double r,
                                            uint8_t *xq) {
    float y[V];
    const double o = a.offset;
#pragma unroll
    for (int k = 0; k < V; k += 4) {
        const float4 w = a.weight == nullptr ? make_float4(1.0f, 1.0f, 1.0f, 1.0f) : load4<R_F32>(a.weight, V * c + k);
        y[k] = (float)((double)x[k] * r * (o + (double)w.x));
        y[k + 1] = (float)((double)x[k + 1] * r * (o + (double)w.y));
        y[k + 2] = (float)((double)x[k + 2] * r * (o + (double)w.z));
        y[k + 3] = (float)((double)x[k + 3] * r * (o + (double)w.w));
    }
    if (a.y != nullptr) store_row<RT, V>(a.y, t * a.ys + V * c, y);
    store_quantized<FMT, V>(xq, c, y);
}

// Workgroups of a launch: a grid holds 2^32 threads.
constexpr int64_t kNormGrid = 1 << 20;

// P pieces of V values a thread; longer rows (P = 0) are walked twice.
template <int RT, int FMT, int V, int P>
__global__ __launch_bounds__(1024) void k_rms_norm(NormArgs a) {
    __shared__ double part[16];
    const int n = (int)(a.K / V), step = blockDim.x;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        uint8_t *xq = a.xq + t * (a.K / act_values(FMT)) * act_bytes(FMT);
        double s = 0.0;
        float x[P ? P : 1][V], r[P ? P : 1][V];
        if constexpr (P > 0) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int c = threadIdx.x + i * step;
                if (c < n) norm_load<RT, V>(a, t, c, x[i], r[i]);
            }
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int c = threadIdx.x + i * step;
                if (c >= n) continue;
                norm_add<RT, V>(a, t, c, x[i], r[i]);
                s += square_sum<V>(x[i]);
            }
        } else {
            for (int c = threadIdx.x; c < n; c += step) {
                NormArgs only = a;
                only.sum = nullptr;                       // written on the second walk: it may be x or the residual
                norm_load<RT, V>(a, t, c, x[0], r[0]);
                norm_add<RT, V>(only, t, c, x[0], r[0]);
                s += square_sum<V>(x[0]);
            }
        }
        const double f = 1.0 / sqrt(workgroup_sum(s, part) / (double)a.K + (double)a.eps);
        if constexpr (P > 0) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int c = threadIdx.x + i * step;
                if (c < n) norm_output<RT, FMT, V>(a, t, c, x[i], f, xq);
            }
        } else {
            for (int c = threadIdx.x; c < n; c += step) {
                norm_load<RT, V>(a, t, c, x[0], r[0]);
                norm_add<RT, V>(a, t, c, x[0], r[0]);
                norm_output<RT, FMT, V>(a, t, c, x[0], f, xq);
            }
        }
        __syncthreads();                                  // `part` is free again
    }
}

template <int RT, int FMT>
static hipError_t launch(NormArgs a, hipStream_t st) {
    constexpr int V = row_values(RT);
    const int64_t n = a.K / V, waves = (n + 63) / 64;     // pieces of a row; waves that hold one each
    // few rows: as many threads as pieces; otherwise four waves that hold up to four each
    const int64_t most = a.T < kCUs ? 16 : 4;
    int64_t threads = 64 * (waves < most ? waves : most);
    if (n > 4 * threads) threads = n <= 2048 ? 512 : 1024;
    const int64_t each = (n + threads - 1) / threads;
    const void *k = each <= 1   ? (const void *)k_rms_norm<RT, FMT, V, 1>
                    : each <= 2 ? (const void *)k_rms_norm<RT, FMT, V, 2>
                    : each <= 4 ? (const void *)k_rms_norm<RT, FMT, V, 4>
                                : (const void *)k_rms_norm<RT, FMT, V, 0>;
    void *args[] = {(void *)&a};
    return hipLaunchKernel(k, dim3((unsigned)(a.T < kNormGrid ? a.T : kNormGrid)), dim3((unsigned)threads), args, 0, st);
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
