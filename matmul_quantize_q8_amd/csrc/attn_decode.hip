// Decode attention: how the work is split, and the joining of its chunks
// (attn_chunk.h has the first launch, a chunk of positions to a workgroup).
#include "attn_chunk.h"

namespace qmm {

hipError_t launch_attn_f16(int nb, int rt, const AttnArgs &a, int64_t B, hipStream_t st);
hipError_t launch_attn_q8_0(int nb, int rt, const AttnArgs &a, int64_t B, hipStream_t st);
hipError_t launch_attn_q4_0(int nb, int rt, const AttnArgs &a, int64_t B, hipStream_t st);

// ---------------------------------------------------------------------------
// The chunks of a query head, one workgroup a head.  Each chunk has, relative to
// a reference r of its own in log2 units, the sum l of the weights 2^(s - r) and
// the sum o of the weighted values:
//   R = max r,  l = sum l_i 2^(r_i - R),  out = sum o_i 2^(r_i - R) / l,
//   lse = R ln 2 + ln l.
// (The workgroup that finishes a head's last chunk could do this in the first
// launch.  That was built: the release that makes its sums visible across XCDs
// writes back a whole L2 for every workgroup, and 16 ragged sequences of up to
// 4096 took 47 us in one launch against 22 + 4 in two.)
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 256, kJoinAhead = 4;

// Adds (r2, l2, o2) to (r, l, o): both relative to their references.
__device__ __forceinline__ void join_parts(float &r, float &l, float4 &o, float r2, float l2, float4 o2) {
    const float top = fmaxf(r, r2), base = top == -INFINITY ? 0.0f : top;
    const float w1 = exp2_fast(r - base), w2 = exp2_fast(r2 - base);
    r = top;
    l = l * w1 + l2 * w2;
    o = make_float4(o.x * w1 + o2.x * w2, o.y * w1 + o2.y * w2, o.z * w1 + o2.z * w2, o.w * w1 + o2.w * w2);
}

// D/4 threads take a row of chunks each, row, row + rows, ...; then the rows are
// joined.  A thread's sums and their references are loaded together (four chunks
// at a time), so that the whole is two trips to memory and not three.
template <int RT>
__global__ __launch_bounds__(kJoinThreads) void k_attn_join(AttnArgs a, int D) {
    __shared__ float4 sums[kJoinThreads];
    __shared__ float2 refs[kJoinThreads];
    const int64_t head = blockIdx.x;
    const int tid = threadIdx.x, quads = D >> 2, rows = kJoinThreads / quads;
    const int row = tid / quads, quad = tid - row * quads;
    const float2 *ml = a.part_ml + head * a.splits;
    const float4 *part = reinterpret_cast<const float4 *>(a.part + head * a.splits * D) + quad;
    float r = -INFINITY, l = 0.0f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row < rows) {
        for (int i = row; i < a.splits; i += kJoinAhead * rows) {
            float2 x[kJoinAhead];
            float4 v[kJoinAhead];
#pragma unroll
            for (int k = 0; k < kJoinAhead; ++k) {
                const int j = min(i + k * rows, a.splits - 1);
                x[k] = ml[j];
                v[k] = part[(int64_t)j * quads];
            }
#pragma unroll
            for (int k = 0; k < kJoinAhead; ++k)
                if (i + k * rows < a.splits) join_parts(r, l, o, x[k].x, x[k].y, v[k]);
        }
    }
    sums[tid] = o;
    refs[tid] = make_float2(r, l);
    __syncthreads();
    if (tid >= quads) return;
    for (int k = 1; k < rows; ++k) {
        const float2 x = refs[k * quads + tid];
        join_parts(r, l, o, x.x, x.y, sums[k * quads + tid]);
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int64_t b = head / a.Hq, h = head - b * a.Hq;
    store4<RT>(a.out, b * a.os.token + h * a.os.head + 4 * quad,
               make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
    if (a.lse && tid == 0) a.lse[head] = log_sum(r, l);
}

struct AttnSplit {
    int chunk, splits;
};

// Work is split until there are two workgroups a CU; a column (one sequence, one
// key head, up to 16 of its query heads) is one chunk when there are as many of
// those.  Of 128 to 2048 positions a chunk, the rule's is the fastest or within 14 %
// of it from 1200 to 40000 positions and 1 to 64 sequences, and within 8 % in 28 of 35 such
// cases; 40000 positions of 8 key heads (q8_0): 24.5 us, with chunks of 256 28.1, of 1024
// 26.7.  It does not know the join's 2 to 4 us: 64 sequences of 1200 of 2 key heads of 64
// take 13.2 us and 11.6 whole, 16 of 1200 of 8 of 128 17.5 and 15.7; and 10000 positions of
// 8 key heads 15.2, with chunks of 384 13.5.
constexpr int kSplitColumns = 2 * (int)kCUs;
constexpr int kMinChunk = 256;                  // positions: a tile of 64 for each wave

static int64_t attn_span(int64_t max_len, int64_t window) {
    // a window starts anywhere in a group of 16, and ends no later than the longest sequence
    return window > 0 && window < max_len - kGroup + 1 ? window + kGroup - 1 : max_len;
}
static int64_t head_tiles(int64_t Hq, int64_t heads) {
    return heads * ((Hq / heads + kHeadTile - 1) / kHeadTile);
}

static AttnSplit attn_split(int64_t B, int64_t Hq, int64_t heads, int64_t max_len, int64_t window) {
    const int64_t span = attn_span(max_len, window), columns = B * head_tiles(Hq, heads);
    // up to 512 positions, one chunk: 300 positions of 2 key heads take 7.0 us whole and
    // 8.8 us split and joined, 1200 take 11.3 and 9.0
    const int64_t want = span <= 2 * kMinChunk ? 1 : (kSplitColumns + columns - 1) / columns;
    int64_t chunk = (span + want - 1) / want;
    chunk = (chunk + kMinChunk - 1) / kMinChunk * kMinChunk;
    return {(int)chunk, (int)((span + chunk - 1) / chunk)};
}

// The workspace: the chunks' sums, then their references.  The size is a bound
// over every smaller batch and length too, which may be split further: a batch of
// B has at most B + kSplitColumns / (columns of a sequence) chunks for each of a
// sequence's columns, and at most one for kMinChunk positions.
static int64_t part_bytes(int64_t B, int64_t Hq, int64_t splits, int64_t D) { return B * Hq * splits * (D + 2) * 4; }

int64_t attn_workspace(int64_t B, int64_t Hq, int64_t heads, int64_t D, int64_t max_len, int64_t window) {
    const int64_t per = head_tiles(Hq, heads), span = attn_span(max_len, window);
    const int64_t by_columns = B + (kSplitColumns + per - 1) / per, by_length = B * ((span + kMinChunk - 1) / kMinChunk);
    return (by_columns < by_length ? by_columns : by_length) * Hq * (D + 2) * 4;
}

hipError_t launch_attn(int fmt, int nb, int rt, AttnArgs a, int64_t B, void *workspace, int64_t workspace_bytes,
                       hipStream_t st) {
    const AttnSplit s = attn_split(B, a.Hq, a.c.heads, a.max_len, a.window);
    int D = 32 * nb;
    if (s.splits > 1 && part_bytes(B, a.Hq, s.splits, D) > workspace_bytes) return hipErrorInvalidValue;
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
