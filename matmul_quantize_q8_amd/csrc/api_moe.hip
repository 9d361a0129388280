// C ABI of the mixture-of-experts operators: argument checks, launch.
// Declarations and contracts are in include/qmm.h.
#include <cmath>

#include "api_check.h"
#include "moe.h"
#include "q8_rows.h"

namespace qmm {
hipError_t launch_rms_norm(int rt, int fmt, const NormArgs &a, hipStream_t st);
hipError_t launch_glu(int rt, int fmt, int act, const GluArgs &a, hipStream_t st);
hipError_t launch_route(int rt, const RouteArgs &a, hipStream_t st);
hipError_t launch_experts_plan(const int *ids, void *plan, int pairs, int top, int E, hipStream_t st);
hipError_t launch_experts_combine(int rt, const float *y, const float *weights, const void *residual, void *out,
                                  int64_t T, int top, int64_t N, int64_t rs, int64_t os, hipStream_t st);
hipError_t launch_experts_few_q4_0(const ExpertArgs &a, hipStream_t st);
hipError_t launch_experts_few_q8_0(const ExpertArgs &a, hipStream_t st);
hipError_t launch_experts_few_q4_1(const ExpertArgs &a, hipStream_t st);
hipError_t launch_experts_few_q5_0(const ExpertArgs &a, hipStream_t st);
hipError_t launch_experts_few_q5_1(const ExpertArgs &a, hipStream_t st);
hipError_t launch_experts_few_q2_k(const ExpertArgs &a, hipStream_t st);
hipError_t launch_experts_few_q4_k(const ExpertArgs &a, hipStream_t st);
hipError_t launch_experts_few_q6_k(const ExpertArgs &a, hipStream_t st);
hipError_t launch_experts_stream_32(int fmt, const ExpertArgs &a, hipStream_t st);
bool experts_stream_32_suits(int fmt, const ExpertArgs &a);
hipError_t launch_experts_stream_k(int fmt, const ExpertArgs &a, hipStream_t st);
hipError_t launch_experts_32(int fmt, const ExpertArgs &a, hipStream_t st);
hipError_t launch_experts_q6_k(const ExpertArgs &a, hipStream_t st);
int64_t matmul_q4_0_max_blocks();
int64_t matmul_k_max_blocks();
}  // namespace qmm

namespace {

using namespace qmm;

constexpr int64_t kMaxOutputs = int64_t(1) << 35;      // values of a product: its grid holds less than 2^32 threads
constexpr int64_t kMaxRows = int64_t(1) << 18;         // weight rows of an expert

bool act_shape_ok(int fmt, int64_t T, int64_t K) {
    if (T < 1 || T > kMaxDim || K < act_values(fmt) || K > kMaxDim || K % act_values(fmt) != 0) return false;
    return T <= kMaxBytes / (K / act_values(fmt) * act_bytes(fmt)) && T <= kMaxBytes / 4 / K;
}

qmm_status check_in(const void *p, int dt, int64_t T, int64_t K, int64_t stride) {
    return check_rows(p, dt, T, 1, K, T > 1 ? stride : 0, 0);
}
qmm_status check_written(const void *p, int dt, int64_t T, int64_t K, int64_t stride) {
    return check_out(p, dt, T, 1, K, T > 1 ? stride : 0, 0);
}

qmm_status rms_norm(int fmt, const void *x, const void *residual, void *sum, const float *weight, void *xq, void *y,
                    int dtype, int64_t T, int64_t K, int64_t xs, int64_t rs, int64_t ss, int64_t ys, float eps,
                    float offset, void *stream) {
    if (!dtype_ok(dtype) || !act_shape_ok(fmt, T, K)) return QMM_E_SHAPE;
    if (!(eps >= 0.0f) || std::isinf(eps) || std::isnan(offset) || std::isinf(offset)) return QMM_E_SHAPE;
    QMM_TRY(check_in(x, dtype, T, K, xs));
    if (residual != nullptr) QMM_TRY(check_in(residual, dtype, T, K, rs));
    if (sum != nullptr) QMM_TRY(check_written(sum, dtype, T, K, ss));
    if (y != nullptr) QMM_TRY(check_written(y, dtype, T, K, ys));
    QMM_TRY(check_ptrs({xq}));
    if (weight != nullptr && !aligned16(weight)) return QMM_E_ALIGN;
    QMM_TRY(check_device());
    const NormArgs a = {x, residual, sum, y, weight, static_cast<uint8_t *>(xq), T, xs, rs, ss, ys, K, eps, offset};
    return launched(launch_rms_norm(dtype, fmt, a, static_cast<hipStream_t>(stream)));
}

qmm_status glu(int fmt, const void *gate, const void *up, void *xq, int dtype, int act, int64_t rows, int64_t F,
               int64_t gs, int64_t us, void *stream) {
    if (!dtype_ok(dtype) || act < QMM_GLU_SILU || act > QMM_GLU_GELU_TANH || !act_shape_ok(fmt, rows, F))
        return QMM_E_SHAPE;
    QMM_TRY(check_in(gate, dtype, rows, F, gs));
    QMM_TRY(check_in(up, dtype, rows, F, us));
    QMM_TRY(check_ptrs({xq}));
    QMM_TRY(check_device());
    const GluArgs a = {gate, up, static_cast<uint8_t *>(xq), rows, gs, us, (int)(F / row_values(dtype))};
    return launched(launch_glu(dtype, fmt, act, a, static_cast<hipStream_t>(stream)));
}

bool pairs_ok(int64_t T, int64_t top_k, int64_t E) {
    return T >= 1 && top_k >= 1 && top_k <= kMaxTop && E >= 1 && E <= kMaxExperts && T <= kMaxPairs / top_k;
}

// A plan's tiles of 128 rows as four of 32 each, where workgroups of 128 x 128 leave
// compute units idle (us, whole / in parts, K = 1024):
//   8192 rows, 1 expert of 256      128 blocks  Q4_0 23 / 16, Q8_0 23 / 19, Q5_1 28 / 23
//   16384 rows, 64 experts of 104   192         Q4_0 23 / 21, Q8_0 23 / 29, Q5_1 28 / 35
//   8192 rows, 1 expert of 512      256         Q4_0 25 / 27, Q8_0 25 / 33, Q5_1 31 / 41
bool in_parts(const ExpertArgs &a) {
    const int64_t tiles = a.pairs / kFullRows + (a.pairs < a.E ? a.pairs : a.E) / 2;      // experts end in the middle of one
    return tiles * ((a.N + 127) / 128) <= kCUs / 2;
}

typedef hipError_t (*few_launch)(const ExpertArgs &, hipStream_t);

qmm_status experts_matmul(int fmt, few_launch few, const void *w, int64_t stride, const void *xq, int64_t x_rows,
                          const int32_t *ids, const void *plan, int64_t bytes, float *y, int64_t T, int64_t top_k,
                          int64_t E, int64_t N, int64_t K, int64_t blk, int64_t wbytes, void *stream) {
    const bool k = blk == 256;
    const int64_t xbytes = k ? kQ8KBytes : kQ80Bytes;
    if (!pairs_ok(T, top_k, E) || N < 1 || N > kMaxRows || K < blk || K > kMaxDim || K % blk != 0) return QMM_E_SHAPE;
    const int64_t nb = K / blk, pairs = T * top_k;
    if (nb > (k ? matmul_k_max_blocks() : matmul_q4_0_max_blocks()) || pairs > kMaxOutputs / N) return QMM_E_SHAPE;
    if (x_rows != T && x_rows != pairs) return QMM_E_SHAPE;
    if (x_rows * nb * xbytes > 0xffffffffll) return QMM_E_SHAPE;            // 32-bit buffer offsets
    if (N * nb * wbytes > kMaxBytes || stride < N * nb * wbytes || stride > kMaxBytes / E) return QMM_E_SHAPE;
    if (bytes < plan_bytes(pairs, E)) return QMM_E_SHAPE;
    QMM_TRY(check_ptrs({w, xq, y}));
    if (stride % 16 != 0) return QMM_E_ALIGN;
    QMM_TRY(check_index(ids, 4));
    QMM_TRY(check_ptrs({plan}));
    QMM_TRY(check_device());
    ExpertArgs a = {static_cast<const uint8_t *>(w), stride, static_cast<const uint8_t *>(xq),
                    (uint32_t)(x_rows * nb * xbytes), x_rows == pairs, y, nullptr, {}, (int)pairs, (int)top_k, (int)E,
                    (int)N, (int)nb, (int)x_rows, tile_rows(pairs, E)};
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (pairs <= kSelfPairs)
        a.ids = ids;
    else
        a.plan = plan_at(plan, pairs, E);
    // one token's experts have a row each: the decode product's way; a single block of 32
    // values is no stage of any other
    if (T == 1 || (!k && nb < 2)) return launched(few(a, st));
    // Q6_K, 64 experts of 1536 x 2048 with 192 / 256 / 512 / 1024 rows each, in tiles of 64 249 / 314 / 580 / 1112 us, of 128
    // 263 / 325 / 567 / 1045; of a plan in steps of 32, most of those would be empty (8 experts of 4096 x 2048, 500 rows each
    // 433 us, streamed 234; 4 of 1048 x 2048 81 / 53)
    if (fmt == F_Q6_K && a.rows == kFullRows && pairs / E >= 384 && !in_parts(a)) return launched(launch_experts_q6_k(a, st));
    if (k) return launched(launch_experts_stream_k(fmt, a, st));
    const bool stages = (a.rows < kFullRows || in_parts(a)) && experts_stream_32_suits(fmt, a);
    return launched(stages ? launch_experts_stream_32(fmt, a, st) : launch_experts_32(fmt, a, st));
}

}  // namespace

extern "C" {

#define QMM_ACT_ENTRY_POINTS(name, fmt)                                                                             \
    qmm_status qmm_rms_norm_##name(const void *x, const void *residual, void *sum, const float *weight, void *xq,   \
                                   void *y, int dtype, int64_t T, int64_t K, int64_t x_stride,                      \
                                   int64_t residual_stride, int64_t sum_stride, int64_t y_stride, float eps,        \
                                   float weight_offset, void *stream) {                                             \
        return rms_norm(fmt, x, residual, sum, weight, xq, y, dtype, T, K, x_stride, residual_stride, sum_stride,   \
                        y_stride, eps, weight_offset, stream);                                                      \
    }                                                                                                               \
    qmm_status qmm_glu_##name(const void *gate, const void *up, void *xq, int dtype, int act, int64_t rows,         \
                              int64_t F, int64_t gate_stride, int64_t up_stride, void *stream) {                    \
        return glu(fmt, gate, up, xq, dtype, act, rows, F, gate_stride, up_stride, stream);                         \
    }

QMM_ACT_ENTRY_POINTS(q8_0, A_Q8_0)
QMM_ACT_ENTRY_POINTS(q8_k, A_Q8_K)

qmm_status qmm_route(const void *logits, int dtype, const float *bias, int32_t *ids, float *weights, int64_t T,
                     int64_t E, int64_t logits_stride, int64_t top_k, int score, int64_t groups, int64_t groups_kept,
                     int64_t group_top, int renorm, float scale, void *stream) {
    if (!dtype_ok(dtype) || !pairs_ok(T, top_k, E) || top_k > E || T > kMaxTokens) return QMM_E_SHAPE;
    if (score != QMM_SCORE_SOFTMAX && score != QMM_SCORE_SIGMOID) return QMM_E_SHAPE;
    if (groups < 1 || groups > kWave || E % groups != 0 || groups_kept < 1 || groups_kept > groups) return QMM_E_SHAPE;
    if (top_k > E / groups * groups_kept || (group_top != 1 && group_top != 2) || !std::isfinite(scale)) return QMM_E_SHAPE;
    if (T > 1 && (logits_stride < 0 || logits_stride > kMaxBytes || (__int128)(T - 1) * logits_stride + E > kMaxBytes / 4))
        return QMM_E_SHAPE;
    QMM_TRY(check_index(logits, row_type_bytes(dtype)));
    QMM_TRY(check_index(ids, 4));
    QMM_TRY(check_index(weights, 4));
    if (bias != nullptr) QMM_TRY(check_index(bias, 4));
    QMM_TRY(check_device());
    const bool grouped = groups > 1 && groups_kept < groups;            // all groups kept: none are left out
    const RouteArgs a = {logits, bias, ids, weights, T, logits_stride, (int)E, (int)top_k, grouped ? (int)groups : 1,
                         (int)groups_kept, (int)group_top, score == QMM_SCORE_SOFTMAX, renorm != 0, scale, 0};
    return launched(launch_route(dtype, a, static_cast<hipStream_t>(stream)));
}

int64_t qmm_experts_plan_bytes(int64_t T, int64_t top_k, int64_t E) {
    return pairs_ok(T, top_k, E) ? plan_bytes(T * top_k, E) : 0;
}

qmm_status qmm_experts_plan(const int32_t *ids, void *plan, int64_t bytes, int64_t T, int64_t top_k, int64_t E,
                            void *stream) {
    if (!pairs_ok(T, top_k, E) || bytes < plan_bytes(T * top_k, E)) return QMM_E_SHAPE;
    QMM_TRY(check_index(ids, 4));
    QMM_TRY(check_ptrs({plan}));
    QMM_TRY(check_device());
    return launched(launch_experts_plan(ids, plan, (int)(T * top_k), (int)top_k, (int)E, static_cast<hipStream_t>(stream)));
}

#define QMM_EXPERTS_ENTRY_POINT(name, fmt, blk, wbytes)                                                             \
    qmm_status qmm_experts_matmul_##name(const void *w, int64_t expert_stride, const void *xq, int64_t x_rows,      \
                                         const int32_t *ids, const void *plan, int64_t plan_bytes, float *y,        \
                                         int64_t T, int64_t top_k, int64_t E, int64_t N, int64_t K, void *stream) { \
        return experts_matmul(fmt, launch_experts_few_##name, w, expert_stride, xq, x_rows, ids, plan, plan_bytes,  \
                              y, T, top_k, E, N, K, blk, wbytes, stream);                                           \
    }

QMM_EXPERTS_ENTRY_POINT(q4_0, F_Q4_0, 32, kQ40Bytes)
QMM_EXPERTS_ENTRY_POINT(q8_0, F_Q8_0, 32, kQ80Bytes)
QMM_EXPERTS_ENTRY_POINT(q4_1, F_Q4_1, 32, kQ41Bytes)
QMM_EXPERTS_ENTRY_POINT(q5_0, F_Q5_0, 32, kQ50Bytes)
QMM_EXPERTS_ENTRY_POINT(q5_1, F_Q5_1, 32, kQ51Bytes)
QMM_EXPERTS_ENTRY_POINT(q2_k, F_Q2_K, 256, kQ2KBytes)
QMM_EXPERTS_ENTRY_POINT(q4_k, F_Q4_K, 256, kQ4KBytes)
QMM_EXPERTS_ENTRY_POINT(q6_k, F_Q6_K, 256, kQ6KBytes)

qmm_status qmm_experts_combine(const float *y, const float *weights, const void *residual, void *out, int dtype,
                               int64_t T, int64_t top_k, int64_t N, int64_t residual_stride, int64_t out_stride,
                               void *stream) {
    if (!dtype_ok(dtype) || !pairs_ok(T, top_k, 1) || N < 1 || N > kMaxRows || T * top_k > kMaxOutputs / N)
        return QMM_E_SHAPE;
    if (N % 4 == 0) {
        if (residual != nullptr) QMM_TRY(check_in(residual, dtype, T, N, residual_stride));
        QMM_TRY(check_written(out, dtype, T, N, out_stride));
    } else {                                               // value by value: any stride will do
        if (T > 1) {
            for (const int64_t s : {residual != nullptr ? residual_stride : 0, out_stride})
                if (s < 0 || s > kMaxBytes / 4 / T) return QMM_E_SHAPE;
            if (out_stride < N) return QMM_E_SHAPE;
        }
        QMM_TRY(check_index(out, row_type_bytes(dtype)));
        if (residual != nullptr) QMM_TRY(check_index(residual, row_type_bytes(dtype)));
    }
    QMM_TRY(check_ptrs({y}));
    QMM_TRY(check_index(weights, 4));
    QMM_TRY(check_device());
    return launched(launch_experts_combine(dtype, y, weights, residual, out, T, (int)top_k, N, residual_stride,
                                           out_stride, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
