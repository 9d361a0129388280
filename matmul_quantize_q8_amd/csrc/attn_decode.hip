// Decode attention: how the work is split, and the joining of the chunks
// (attn_chunk.h has the first launch, a chunk of positions to a workgroup).
#include "kv_layout.h"

namespace qmm {

hipError_t launch_attn_f16(int nb, int rt, const AttnArgs &a, int64_t B, hipStream_t st);
hipError_t launch_attn_q8_0(int nb, int rt, const AttnArgs &a, int64_t B, hipStream_t st);
hipError_t launch_attn_q4_0(int nb, int rt, const AttnArgs &a, int64_t B, hipStream_t st);

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kHeadTile = 16;                   // query heads of a workgroup

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// ---------------------------------------------------------------------------
// The chunks of a query head, one workgroup a head: each with its sums and the
// reference, in log2 units, that they are relative to.
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 256;

template <int RT>
__global__ __launch_bounds__(kJoinThreads) void k_attn_join(AttnArgs a, int D) {
    __shared__ float4 sums[kJoinThreads];
    __shared__ float red[4], ls[kJoinThreads];
    const int64_t head = blockIdx.x;
    const int tid = threadIdx.x, quads = D >> 2, rows = kJoinThreads / quads;
    const float2 *ml = a.part_ml + head * a.splits;
    float m = -INFINITY;
    for (int i = tid; i < a.splits; i += kJoinThreads) m = fmaxf(m, ml[i].x);
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) m = fmaxf(m, xor_shfl(m, k));
    if ((tid & 63) == 0) red[tid >> 6] = m;
    __syncthreads();
    m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const float base = m == -INFINITY ? 0.0f : m;

    const int row = tid / quads, quad = tid - row * quads;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.0f;
    if (row < rows) {
        for (int i = row; i < a.splits; i += rows) {
            const float2 x = ml[i];
            const float w = exp2_fast(x.x - base);
            const float4 v = reinterpret_cast<const float4 *>(a.part + (head * a.splits + i) * D)[quad];
            l = fmaf(w, x.y, l);
            o.x = fmaf(w, v.x, o.x);
            o.y = fmaf(w, v.y, o.y);
            o.z = fmaf(w, v.z, o.z);
            o.w = fmaf(w, v.w, o.w);
        }
    }
    sums[tid] = o;
    ls[tid] = l;
    __syncthreads();
    if (tid >= quads) return;
    for (int k = 1; k < rows; ++k) {
        const float4 v = sums[k * quads + tid];
        o.x += v.x;
        o.y += v.y;
        o.z += v.z;
        o.w += v.w;
        l += ls[k * quads + tid];
    }
    const float r = l == 0.0f ? 0.0f : 1.0f / l;
    const int64_t b = head / a.Hq, h = head - b * a.Hq;
    store4<RT>(a.out, b * a.os.token + h * a.os.head + 4 * quad, make_float4(o.x * r, o.y * r, o.z * r, o.w * r));
    if (a.lse && tid == 0) a.lse[head] = base / kLog2e + logf(l);
}

struct AttnSplit {
    int chunk, splits;
};

// Chunks of a multiple of 256 positions (a tile for each wave, of up to 64).
static AttnSplit attn_split(int64_t B, int64_t Hq, int64_t heads, int64_t max_len, int64_t window) {
    // a window starts anywhere in a group of 16
    const int64_t span = window > 0 && window < max_len ? window + kGroup - 1 : max_len;
    const int64_t group = Hq / heads, columns = B * heads * ((group + kHeadTile - 1) / kHeadTile);
    const int64_t want = (2 * kCUs + columns - 1) / columns;
    int64_t chunk = (span + want - 1) / want;
    chunk = (chunk + 255) / 256 * 256;
    return {(int)chunk, (int)((span + chunk - 1) / chunk)};
}

int64_t attn_workspace(int64_t B, int64_t Hq, int64_t heads, int64_t D, int64_t max_len, int64_t window) {
    const AttnSplit s = attn_split(B, Hq, heads, max_len, window);
    return B * Hq * s.splits * (D + 2) * 4;
}

hipError_t launch_attn(int fmt, int nb, int rt, AttnArgs a, int64_t B, void *workspace, hipStream_t st) {
    const AttnSplit s = attn_split(B, a.Hq, a.c.heads, a.max_len, a.window);
    int D = 32 * nb;
    a.splits = s.splits;
    a.chunk = s.chunk;
    a.part = static_cast<float *>(workspace);
    a.part_ml = reinterpret_cast<float2 *>(a.part + B * a.Hq * s.splits * D);
    const hipError_t e = fmt == KV_F16    ? launch_attn_f16(nb, rt, a, B, st)
                         : fmt == KV_Q8_0 ? launch_attn_q8_0(nb, rt, a, B, st)
                                          : launch_attn_q4_0(nb, rt, a, B, st);
    if (e != hipSuccess || s.splits == 1) return e;
    void *args[] = {(void *)&a, (void *)&D};
    const void *j = rt == R_F32 ? (const void *)k_attn_join<R_F32>
                    : rt == R_F16 ? (const void *)k_attn_join<R_F16> : (const void *)k_attn_join<R_BF16>;
    return hipLaunchKernel(j, dim3((unsigned)(B * a.Hq)), dim3(kJoinThreads), args, 0, st);
}

}  // namespace qmm
