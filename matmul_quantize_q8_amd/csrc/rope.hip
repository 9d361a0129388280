// Rotary positions: y = R(p) x, a rotation of each pair of a row's values by
// the angle p * f_i (include/qmm.h states the formula and its roundings).
//
// One workgroup takes one token and, where there are few tokens, a part of its
// heads: the token's rot/2 cosines and sines are computed once, in f64, into
// LDS, and every wave then turns whole rows, 16 bytes a lane (8 of 16-bit rows
// whose length is no multiple of eight).  A wave loads the rows it works on
// before it stores any of them, so y may be x.
//
// Bound by memory: 4096 tokens of 32 heads of 128 in bf16 (67 MB) take 16 us,
// 4.2 TB/s of the 4.9 of a large copy; one token of 40 heads 2.5 us, a launch.
#include "kv_layout.h"

namespace qmm {

constexpr int kRopeThreads = 256;

template <int RT, int V>
__global__ __launch_bounds__(kRopeThreads) void k_rope(Rope r, const void *x, void *y, const int32_t *positions,
                                                       int H, int D, Strides xs, Strides ys) {
    __shared__ float2 cs[kMaxHeadDim / 2];
    const int64_t t = blockIdx.x;
    rope_table(r, positions[t], cs, threadIdx.x, kRopeThreads);
    __syncthreads();
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int lanes = D / V, per_wave = 64 / lanes, sub = lane / lanes, n = V * (lane - sub * lanes);
    if (sub >= per_wave) return;
    const int step = gridDim.y * (kRopeThreads / 64) * per_wave;
    int h = (blockIdx.y * (kRopeThreads / 64) + wave) * per_wave + sub;
    float v[V];
    for (; h + step < H; h += 2 * step) {                 // two rows' loads in flight: neither store may pass them
        float w[V];
        rotate<RT, V>(x, t * xs.token + h * xs.head, n, r, cs, v);
        rotate<RT, V>(x, t * xs.token + (h + step) * xs.head, n, r, cs, w);
        store_row<RT, V>(y, t * ys.token + h * ys.head + n, v);
        store_row<RT, V>(y, t * ys.token + (h + step) * ys.head + n, w);
    }
    if (h < H) {
        rotate<RT, V>(x, t * xs.token + h * xs.head, n, r, cs, v);
        store_row<RT, V>(y, t * ys.token + h * ys.head + n, v);
    }
}

// Parts of a token's rows: as many workgroups as give the chip four a compute
// unit, at least one row for every wave.
int row_parts(int64_t T, int64_t rows, int rows_per_workgroup) {
    const int64_t most = (rows + rows_per_workgroup - 1) / rows_per_workgroup, want = (4 * kCUs + T - 1) / T;
    return (int)(want < most ? want : most);
}

hipError_t launch_rope(int rt, Rope r, const void *x, void *y, const int32_t *positions, int64_t T, int H, int D,
                       Strides xs, Strides ys, hipStream_t st) {
    const bool wide = row_values(rt) == 8 && D % 8 == 0;
    const dim3 grid((unsigned)T, (unsigned)row_parts(T, H, kRopeThreads / 64 * (64 / (D / (wide ? 8 : 4)))));
    void *args[] = {(void *)&r, (void *)&x, (void *)&y, (void *)&positions, (void *)&H, (void *)&D,
                    (void *)&xs, (void *)&ys};
    const void *k = rt == R_F32   ? (const void *)k_rope<R_F32, 4>
                    : rt == R_F16 ? (wide ? (const void *)k_rope<R_F16, 8> : (const void *)k_rope<R_F16, 4>)
                                  : (wide ? (const void *)k_rope<R_BF16, 8> : (const void *)k_rope<R_BF16, 4>);
    return hipLaunchKernel(k, grid, dim3(kRopeThreads), args, 0, st);
}

}  // namespace qmm
