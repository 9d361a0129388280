// Attention of one new token over the paged key-value cache (include/qmm.h
// states the formula).  The sequence is cut into chunks of positions; every
// chunk's maximum m, sum l of exp(s - m) and sum o of exp(s - m) v are joined
// by a second, small launch:
//   M = max m,  l = sum l_i exp(m_i - M),  out = sum o_i exp(m_i - M) / l.
#include "kv_layout.h"

namespace qmm {

constexpr int kAttnThreads = 256;
constexpr int kChunk = 256;

// Value n of the row of position t at `side`.
template <int F, int NB>
__device__ __forceinline__ float kv_value(const uint8_t *side, int page, int t, int n, bool values) {
    using K = Kv<F, NB>;
    const int b = n >> 5, r = n & 31;
    const int v = values ? (t & 3) * 2 * NB + 2 * b + (r & 1) : 8 * b + (r & 7);
    const int byte = values ? K::at((t & 15) >> 2, r >> 1, K::byte_of(v)) : K::at(r >> 3, t & 15, K::byte_of(v));
    const uint8_t *p = side + (t >> 4) * K::kGroupBytes + byte;
    if constexpr (F == KV_F16) return f16_bits_to_f32(*reinterpret_cast<const uint16_t *>(p));
    const float d = f16_bits_to_f32(
        reinterpret_cast<const uint16_t *>(side + (page >> 4) * K::kGroupBytes)[t * NB + b]);
    if constexpr (F == KV_Q8_0) return d * (float)((int)*p - 128);
    return d * (float)((int)((*p >> (4 * (v & 1))) & 15) - 8);
}

template <int F, int NB, int RT>
__global__ __launch_bounds__(kAttnThreads) void k_attn_chunk(AttnArgs a) {
    constexpr int D = 32 * NB;
    __shared__ float q[D], p[kAttnThreads], red[4];
    const int tid = threadIdx.x, split = blockIdx.x, hq = blockIdx.y, b = blockIdx.z;
    const int len = a.lens[b], page = 1 << a.c.page_shift;
    const bool bad_len = len < 0 || len > a.max_len;
    const int lo = a.window && !bad_len ? max(0, len - a.window) : 0;
    const int from = lo + split * a.chunk, to = bad_len ? from : min(len, from + a.chunk);
    const int64_t side = Kv<F, NB>::side_bytes(page);
    const int h = hq / (a.Hq / a.c.heads);
    const int64_t head = (int64_t)b * a.Hq + hq;
    for (int i = tid; i < D; i += kAttnThreads) q[i] = load1<RT>(a.q, b * a.qs.token + hq * a.qs.head + i);
    __syncthreads();
    float m = -INFINITY, l = 0.0f, o = 0.0f;
    for (int t0 = from; t0 < to; t0 += kAttnThreads) {
        const int t = t0 + tid;
        float s = -INFINITY;
        if (t < to) {
            const int64_t pg = a.pages[b * a.pages_stride + (t >> a.c.page_shift)];
            if (!a.c.has_page(pg)) {
                s = NAN;
            } else {
                const uint8_t *ks = a.c.page_at(pg, side) + 2 * h * side;
                float acc = 0.0f;
                for (int i = 0; i < D; ++i)
                    acc = fmaf(q[i], kv_value<F, NB>(ks, page, t & (page - 1), i, false), acc);
                s = acc * a.scale;
                if (a.softcap > 0.0f) s = a.softcap * tanhf(s / a.softcap);
                if (a.mask) {
                    const float x = a.mask[b * a.mask_stride + t];
                    s = x == -INFINITY ? -INFINITY : s + x;
                }
            }
        }
        float mx = s;
        for (int k = 1; k < 64; k <<= 1) mx = fmaxf(mx, xor_shfl(mx, k));
        if ((tid & 63) == 0) red[tid >> 6] = mx;
        __syncthreads();
        mx = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), m);
        const float base = mx == -INFINITY ? 0.0f : mx;
        p[tid] = expf(s - base);
        const float alpha = expf(m - base);
        m = mx;
        l *= alpha;
        o *= alpha;
        __syncthreads();
        for (int k = 0; k < min(kAttnThreads, to - t0); ++k) {
            const int tk = t0 + k;
            const float w = p[k];
            const int64_t pg = a.pages[b * a.pages_stride + (tk >> a.c.page_shift)];
            const bool bad = !a.c.has_page(pg);
            if (a.mask && a.mask[b * a.mask_stride + tk] == -INFINITY) continue;
            l += w;
            if (tid < D)
                o = fmaf(w, bad ? 0.0f
                                : kv_value<F, NB>(a.c.page_at(pg, side) + (2 * h + 1) * side, page,
                                                  tk & (page - 1), tid, true), o);
        }
        __syncthreads();
    }
    if (bad_len) l = o = NAN;
    if (tid < D) a.part[(head * a.splits + split) * D + tid] = o;
    if (tid == 0) a.part_ml[head * a.splits + split] = make_float2(m, l);
}

// One wave a query head.
template <int RT>
__global__ __launch_bounds__(64) void k_attn_join(AttnArgs a, int D) {
    const int64_t head = blockIdx.x;
    const int lane = threadIdx.x;
    const float2 *ml = a.part_ml + head * a.splits;
    float m = -INFINITY;
    for (int i = 0; i < a.splits; ++i) m = fmaxf(m, ml[i].x);
    const float base = m == -INFINITY ? 0.0f : m;
    float l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int i = 0; i < a.splits; ++i) {
        const float w = expf(ml[i].x - base);
        if (ml[i].y == 0.0f) continue;
        l = fmaf(w, ml[i].y, l);
        if (4 * lane < D) {
            const float4 v = *reinterpret_cast<const float4 *>(a.part + (head * a.splits + i) * D + 4 * lane);
            o[0] = fmaf(w, v.x, o[0]);
            o[1] = fmaf(w, v.y, o[1]);
            o[2] = fmaf(w, v.z, o[2]);
            o[3] = fmaf(w, v.w, o[3]);
        }
    }
    const float r = l == 0.0f ? 0.0f : 1.0f / l;
    const int64_t b = head / a.Hq, h = head - b * a.Hq;
    if (4 * lane < D)
        store4<RT>(a.out, b * a.os.token + h * a.os.head + 4 * lane, make_float4(o[0] * r, o[1] * r, o[2] * r, o[3] * r));
    if (a.lse && lane == 0) a.lse[head] = base + logf(l);
}

struct AttnSplit {
    int chunk, splits;
};

static AttnSplit attn_split(int64_t max_len, int64_t window) {
    const int64_t span = window > 0 && window < max_len ? window : max_len;
    return {kChunk, (int)((span + kChunk - 1) / kChunk)};
}

int64_t attn_workspace(int64_t B, int64_t Hq, int64_t D, int64_t max_len, int64_t window) {
    const AttnSplit s = attn_split(max_len, window);
    return B * Hq * s.splits * (D + 2) * 4;
}

template <int F, int NB>
static hipError_t launch_attn_f(int rt, AttnArgs a, int64_t B, void *workspace, hipStream_t st) {
    const AttnSplit s = attn_split(a.max_len, a.window);
    int D = 32 * NB;
    a.splits = s.splits;
    a.chunk = s.chunk;
    a.part = static_cast<float *>(workspace);
    a.part_ml = reinterpret_cast<float2 *>(a.part + B * a.Hq * s.splits * D);
    void *args[] = {(void *)&a};
    const void *k = rt == R_F32   ? (const void *)k_attn_chunk<F, NB, R_F32>
                    : rt == R_F16 ? (const void *)k_attn_chunk<F, NB, R_F16>
                                  : (const void *)k_attn_chunk<F, NB, R_BF16>;
    hipError_t e = hipLaunchKernel(k, dim3((unsigned)s.splits, (unsigned)a.Hq, (unsigned)B), dim3(kAttnThreads),
                                   args, 0, st);
    if (e != hipSuccess) return e;
    void *jargs[] = {(void *)&a, (void *)&D};
    const void *j = rt == R_F32 ? (const void *)k_attn_join<R_F32>
                    : rt == R_F16 ? (const void *)k_attn_join<R_F16> : (const void *)k_attn_join<R_BF16>;
    return hipLaunchKernel(j, dim3((unsigned)(B * a.Hq)), dim3(64), jargs, 0, st);
}

hipError_t launch_attn(int fmt, int nb, int rt, AttnArgs a, int64_t B, void *workspace, hipStream_t st) {
    QMM_KV_DISPATCH(launch_attn_f, rt, a, B, workspace, st);
}

}  // namespace qmm
