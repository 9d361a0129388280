// C ABI of the attention operators: argument checks, launch.  Declarations and
// contracts are in include/qmm.h.
#include <cmath>
#include <utility>

#include "api_check.h"
#include "kv_layout.h"

namespace qmm {
hipError_t launch_rope(int rt, Rope r, const void *x, void *y, const int32_t *positions, int64_t T, int H, int D,
                       Strides xs, Strides ys, hipStream_t st);
hipError_t launch_kv_write(int fmt, int nb, int rt, WriteArgs a, hipStream_t st);
hipError_t launch_kv_read(int fmt, int nb, int rt, ReadArgs a, hipStream_t st);
hipError_t launch_attn(int fmt, int nb, int rt, AttnArgs a, int64_t B, void *workspace, int64_t workspace_bytes,
                       hipStream_t st);
int64_t attn_workspace(int64_t B, int64_t Hq, int64_t heads, int64_t D, int64_t max_len, int64_t window);
}  // namespace qmm

namespace {

using namespace qmm;

constexpr int64_t kMaxHeads = 4096;
constexpr int64_t kMaxPage = 4096;
constexpr int64_t kMaxTokens = (int64_t(1) << 24) - 1;   // a workgroup of 256 each: a grid holds 2^32 threads

bool dtype_ok(int dt) { return dt == QMM_F32 || dt == QMM_F16 || dt == QMM_BF16; }

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Rows of T tokens and H heads of D values: what the strides may be.
qmm_status check_rows(const void *p, int dt, int64_t T, int64_t H, int64_t D, int64_t token, int64_t head) {
    if (token < 0 || head < 0 || token > kMaxBytes || head > kMaxBytes) return QMM_E_SHAPE;
    const __int128 last = (__int128)(T - 1) * token + (__int128)(H - 1) * head + D;
    if (last > kMaxBytes / row_type_bytes(dt)) return QMM_E_SHAPE;
    if (p == nullptr) return QMM_E_NULL;
    if (token % 4 != 0 || head % 4 != 0 || !aligned(p, 4 * row_type_bytes(dt))) return QMM_E_ALIGN;
    return QMM_OK;
}

// Rows that are written, of which no two may share an element: their offsets
// t * token + h * head lie D and more apart.
bool rows_apart(int64_t T, int64_t H, int64_t D, int64_t token, int64_t head) {
    if ((T > 1 && token < D) || (H > 1 && head < D)) return false;
    if (T == 1 || H == 1 || (H - 1) * head + D <= token || (T - 1) * token + D <= head) return true;
    if (T < H) std::swap(T, H), std::swap(token, head);
    for (int64_t h = 1; h < H; ++h) {                 // neither is inside a step of the other: the row before h steps, and after
        const int64_t t = h * head / token, before = h * head - t * token;
        if ((t < T && before < D) || (t + 1 < T && token - before < D)) return false;
    }
    return true;
}

qmm_status check_out(const void *p, int dt, int64_t T, int64_t H, int64_t D, int64_t token, int64_t head) {
    const qmm_status s = check_rows(p, dt, T, H, D, token, head);
    return s != QMM_OK ? s : rows_apart(T, H, D, token, head) ? QMM_OK : QMM_E_SHAPE;
}

bool head_dim_ok(int64_t d) { return d == 64 || d == 96 || d == 128 || d == 192 || d == 256; }

bool kv_sizes_ok(int64_t page, int64_t heads, int64_t dim) {
    return head_dim_ok(dim) && page >= kGroup && page <= kMaxPage && (page & (page - 1)) == 0 && heads >= 1 &&
           heads <= kMaxHeads;
}

int64_t page_bytes(int fmt, int64_t page, int64_t heads, int64_t dim) {
    return kv_sizes_ok(page, heads, dim) ? kv_page_bytes(fmt, page, heads, dim) : 0;
}

qmm_status check_cache(int fmt, const qmm_kv_cache *c, KvCache &out) {
    if (c == nullptr) return QMM_E_NULL;
    if (!kv_sizes_ok(c->page, c->heads, c->dim)) return QMM_E_SHAPE;
    if (c->n_pages < 1 || c->n_pages > kMaxDim || c->n_pages > kMaxBytes / page_bytes(fmt, c->page, c->heads, c->dim))
        return QMM_E_SHAPE;
    if (c->data == nullptr) return QMM_E_NULL;
    if (!aligned16(c->data)) return QMM_E_ALIGN;
    out = {static_cast<uint8_t *>(c->data), c->n_pages, __builtin_ctzll((unsigned long long)c->page), (int)c->heads};
    return QMM_OK;
}

qmm_status check_plan(const qmm_rope_plan *p, int64_t D, bool inverse, Rope &out) {
    if (p == nullptr) return QMM_E_NULL;
    if (p->rot < 2 || p->rot > D || p->rot % 2 != 0) return QMM_E_SHAPE;
    if (p->order != QMM_ROPE_HALF && p->order != QMM_ROPE_INTERLEAVED) return QMM_E_SHAPE;
    if (p->freqs == nullptr) return QMM_E_NULL;
    if (!aligned(p->freqs, 8)) return QMM_E_ALIGN;
    out = {p->freqs, (int)p->rot, p->order, inverse, p->mscale};
    return QMM_OK;
}

qmm_status check_index(const void *p, uintptr_t size) {
    if (p == nullptr) return QMM_E_NULL;
    return aligned(p, size) ? QMM_OK : QMM_E_ALIGN;
}

#define QMM_TRY(expr)                          \
    do {                                       \
        const qmm_status s_ = (expr);          \
        if (s_ != QMM_OK) return s_;           \
    } while (0)

qmm_status kv_write(int fmt, const qmm_rope_plan *plan, const qmm_kv_cache *cache, const void *q, void *q_out,
                    const void *k, const void *v, int dtype, const int32_t *positions, const int64_t *slots,
                    int64_t T, int64_t Hq, Strides qs, Strides qos, Strides ks, Strides vs, void *stream) {
    if (!dtype_ok(dtype) || T < 1 || T > kMaxTokens) return QMM_E_SHAPE;
    WriteArgs a = {};
    QMM_TRY(check_cache(fmt, cache, a.c));
    const int64_t H = cache->heads, D = cache->dim;
    if (Hq > 0) {
        if (Hq > kMaxHeads) return QMM_E_SHAPE;
        QMM_TRY(check_plan(plan, D, false, a.r));
        QMM_TRY(check_rows(q, dtype, T, Hq, D, qs.token, qs.head));
        QMM_TRY(check_out(q_out, dtype, T, Hq, D, qos.token, qos.head));
        QMM_TRY(check_index(positions, 4));
    }
    QMM_TRY(check_rows(k, dtype, T, H, D, ks.token, ks.head));
    QMM_TRY(check_rows(v, dtype, T, H, D, vs.token, vs.head));
    QMM_TRY(check_index(slots, 8));
    QMM_TRY(check_device());
    a.q = q;
    a.qo = q_out;
    a.k = k;
    a.v = v;
    a.positions = positions;
    a.slots = slots;
    a.T = T;
    a.Hq = (int)Hq;
    a.qs = qs;
    a.qos = qos;
    a.ks = ks;
    a.vs = vs;
    return launched(launch_kv_write(fmt, (int)(D / 32), dtype, a, static_cast<hipStream_t>(stream)));
}

qmm_status kv_read(int fmt, const qmm_kv_cache *cache, const int64_t *slots, void *k, void *v, int dtype, int64_t T,
                   Strides ks, Strides vs, void *stream) {
    if (!dtype_ok(dtype) || T < 1 || T > kMaxTokens) return QMM_E_SHAPE;
    ReadArgs a = {};
    QMM_TRY(check_cache(fmt, cache, a.c));
    if (k == nullptr && v == nullptr) return QMM_E_NULL;
    if (k != nullptr) QMM_TRY(check_out(k, dtype, T, cache->heads, cache->dim, ks.token, ks.head));
    if (v != nullptr) QMM_TRY(check_out(v, dtype, T, cache->heads, cache->dim, vs.token, vs.head));
    QMM_TRY(check_index(slots, 8));
    QMM_TRY(check_device());
    a.slots = slots;
    a.k = k;
    a.v = v;
    a.T = T;
    a.ks = ks;
    a.vs = vs;
    return launched(launch_kv_read(fmt, (int)(cache->dim / 32), dtype, a, static_cast<hipStream_t>(stream)));
}

// Bytes of the workspace; 0 for sizes outside the limits.
int64_t workspace_bytes(int64_t B, int64_t Hq, int64_t heads, int64_t dim, int64_t max_len, int64_t window) {
    if (B < 1 || B > 65535 || Hq < 1 || Hq > kMaxHeads || heads < 1 || heads > Hq || Hq % heads != 0) return 0;
    if (!head_dim_ok(dim) || max_len < 1 || max_len > kMaxDim - 8192 || window < 0 || window > kMaxDim) return 0;
    return attn_workspace(B, Hq, heads, dim, max_len, window);
}

qmm_status attn_decode(int fmt, const qmm_kv_cache *cache, const void *q, void *out, int dtype, const int32_t *pages,
                       int64_t pages_stride, const int32_t *lens, int64_t B, int64_t Hq, int64_t max_len, float scale,
                       float softcap, int64_t window, const float *mask, int64_t mask_stride, float *lse, Strides qs,
                       Strides os, void *workspace, int64_t ws_bytes, void *stream) {
    if (!dtype_ok(dtype)) return QMM_E_SHAPE;
    AttnArgs a = {};
    QMM_TRY(check_cache(fmt, cache, a.c));
    const int64_t need = workspace_bytes(B, Hq, cache->heads, cache->dim, max_len, window);
    if (need == 0 || need > kMaxBytes || ws_bytes < need) return QMM_E_SHAPE;
    if (pages_stride < 1 || pages_stride > kMaxDim || max_len > pages_stride * cache->page) return QMM_E_SHAPE;
    if (!(softcap >= 0.0f) || std::isinf(softcap) || std::isnan(scale)) return QMM_E_SHAPE;
    if (mask != nullptr && (mask_stride < max_len || mask_stride > kMaxBytes / 4 / B)) return QMM_E_SHAPE;
    QMM_TRY(check_rows(q, dtype, B, Hq, cache->dim, qs.token, qs.head));
    QMM_TRY(check_out(out, dtype, B, Hq, cache->dim, os.token, os.head));
    QMM_TRY(check_index(pages, 4));
    QMM_TRY(check_index(lens, 4));
    if (mask != nullptr) QMM_TRY(check_index(mask, 4));
    if (lse != nullptr) QMM_TRY(check_index(lse, 4));
    QMM_TRY(check_ptrs({workspace}));
    QMM_TRY(check_device());
    a.q = q;
    a.out = out;
    a.pages = pages;
    a.lens = lens;
    a.pages_stride = pages_stride;
    a.mask = mask;
    a.mask_stride = mask_stride;
    a.lse = lse;
    a.Hq = (int)Hq;
    a.max_len = (int)max_len;
    a.window = (int)(window < max_len ? window : 0);          // a window of the whole length is none
    a.scale = scale;
    a.softcap = softcap;
    a.qs = qs;
    a.os = os;
    return launched(launch_attn(fmt, (int)(cache->dim / 32), dtype, a, B, workspace, ws_bytes,
                                static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

qmm_status qmm_rope_freqs(double *freqs, float *mscale, int64_t rot, double base, int scaling, double factor,
                          double trained_len, double low, double high) {
    if (rot < 2 || rot > kMaxHeadDim || rot % 2 != 0 || !(base > 1.0) || std::isinf(base)) return QMM_E_SHAPE;
    if (scaling < QMM_ROPE_PLAIN || scaling > QMM_ROPE_BANDS) return QMM_E_SHAPE;
    if (scaling != QMM_ROPE_PLAIN && (!(factor >= 1.0) || std::isinf(factor))) return QMM_E_SHAPE;
    if (scaling >= QMM_ROPE_YARN && (!(low > 0.0) || !(high > low) || std::isinf(high) || !(trained_len > 0.0) ||
                                     std::isinf(trained_len)))
        return QMM_E_SHAPE;
    if (scaling == QMM_ROPE_NTK && rot == 2) return QMM_E_SHAPE;
    if (freqs == nullptr) return QMM_E_NULL;
    const double two_pi = 6.283185307179586477;
    if (scaling == QMM_ROPE_NTK) base *= std::pow(factor, (double)rot / (double)(rot - 2));
    // YARN: the pair (as a real number) that turns n times in trained_len positions
    double first = 0.0, last = 0.0;
    if (scaling == QMM_ROPE_YARN) {
        const double per = (double)rot / (2.0 * std::log(base));
        first = std::floor(per * std::log(trained_len / (high * two_pi)));
        last = std::ceil(per * std::log(trained_len / (low * two_pi)));
        first = first > 0.0 ? first : 0.0;
        last = last < (double)(rot - 1) ? last : (double)(rot - 1);
        if (!(last > first)) last = first + 0.001;
    }
    for (int64_t i = 0; i < rot / 2; ++i) {
        double f = std::pow(base, -2.0 * (double)i / (double)rot);
        if (scaling == QMM_ROPE_LINEAR) f /= factor;
        if (scaling == QMM_ROPE_YARN) {
            double s = ((double)i - first) / (last - first);
            s = s < 0.0 ? 0.0 : s > 1.0 ? 1.0 : s;
            f = f / factor * s + f * (1.0 - s);
        }
        if (scaling == QMM_ROPE_BANDS) {
            const double turns = trained_len * f / two_pi;
            if (turns < low)
                f /= factor;
            else if (turns <= high) {
                const double s = (turns - low) / (high - low);
                f = f * ((1.0 - s) / factor + s);
            }
        }
        freqs[i] = f;
    }
    if (mscale != nullptr) *mscale = scaling == QMM_ROPE_YARN ? (float)(1.0 + 0.1 * std::log(factor)) : 1.0f;
    return QMM_OK;
}

qmm_status qmm_rope(const qmm_rope_plan *plan, const void *x, void *y, int dtype, const int32_t *positions,
                    int inverse, int64_t T, int64_t H, int64_t D, int64_t x_token_stride, int64_t x_head_stride,
                    int64_t y_token_stride, int64_t y_head_stride, void *stream) {
    if (!dtype_ok(dtype) || T < 1 || T > kMaxTokens || H < 1 || H > kMaxHeads) return QMM_E_SHAPE;
    if (D < 4 || D > kMaxHeadDim || D % 4 != 0) return QMM_E_SHAPE;
    Rope r;
    QMM_TRY(check_plan(plan, D, inverse != 0, r));
    QMM_TRY(check_rows(x, dtype, T, H, D, x_token_stride, x_head_stride));
    QMM_TRY(check_out(y, dtype, T, H, D, y_token_stride, y_head_stride));
    QMM_TRY(check_index(positions, 4));
    QMM_TRY(check_device());
    return launched(launch_rope(dtype, r, x, y, positions, T, (int)H, (int)D, {x_token_stride, x_head_stride},
                                {y_token_stride, y_head_stride}, static_cast<hipStream_t>(stream)));
}

#define QMM_KV_ENTRY_POINTS(name, fmt)                                                                              \
    int64_t qmm_kv_page_bytes_##name(int64_t page, int64_t heads, int64_t dim) {                                    \
        return page_bytes(fmt, page, heads, dim);                                                                   \
    }                                                                                                               \
    qmm_status qmm_kv_write_##name(const qmm_kv_cache *cache, const void *k, const void *v, int dtype,              \
                                   const int64_t *slots, int64_t T, int64_t k_token_stride, int64_t k_head_stride,  \
                                   int64_t v_token_stride, int64_t v_head_stride, void *stream) {                   \
        return kv_write(fmt, nullptr, cache, nullptr, nullptr, k, v, dtype, nullptr, slots, T, 0, {0, 0}, {0, 0},   \
                        {k_token_stride, k_head_stride}, {v_token_stride, v_head_stride}, stream);                  \
    }                                                                                                               \
    qmm_status qmm_rope_kv_write_##name(                                                                            \
        const qmm_rope_plan *plan, const qmm_kv_cache *cache, const void *q, void *q_out, const void *k,            \
        const void *v, int dtype, const int32_t *positions, const int64_t *slots, int64_t T, int64_t Hq,            \
        int64_t q_token_stride, int64_t q_head_stride, int64_t q_out_token_stride, int64_t q_out_head_stride,       \
        int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,               \
        void *stream) {                                                                                             \
        if (Hq < 1) return QMM_E_SHAPE;                                                                             \
        return kv_write(fmt, plan, cache, q, q_out, k, v, dtype, positions, slots, T, Hq,                           \
                        {q_token_stride, q_head_stride}, {q_out_token_stride, q_out_head_stride},                   \
                        {k_token_stride, k_head_stride}, {v_token_stride, v_head_stride}, stream);                  \
    }                                                                                                               \
    qmm_status qmm_kv_read_##name(const qmm_kv_cache *cache, const int64_t *slots, void *k, void *v, int dtype,     \
                                  int64_t T, int64_t k_token_stride, int64_t k_head_stride,                         \
                                  int64_t v_token_stride, int64_t v_head_stride, void *stream) {                    \
        return kv_read(fmt, cache, slots, k, v, dtype, T, {k_token_stride, k_head_stride},                          \
                       {v_token_stride, v_head_stride}, stream);                                                    \
    }                                                                                                               \
    qmm_status qmm_attn_decode_##name(                                                                              \
        const qmm_kv_cache *cache, const void *q, void *out, int dtype, const int32_t *pages, int64_t pages_stride, \
        const int32_t *lens, int64_t B, int64_t Hq, int64_t max_len, float scale, float softcap, int64_t window,    \
        const float *mask, int64_t mask_stride, float *lse, int64_t q_token_stride, int64_t q_head_stride,          \
        int64_t out_token_stride, int64_t out_head_stride, void *workspace, int64_t workspace_bytes,                \
        void *stream) {                                                                                             \
        return attn_decode(fmt, cache, q, out, dtype, pages, pages_stride, lens, B, Hq, max_len, scale, softcap,    \
                           window, mask, mask_stride, lse, {q_token_stride, q_head_stride},                         \
                           {out_token_stride, out_head_stride}, workspace, workspace_bytes, stream);                \
    }

QMM_KV_ENTRY_POINTS(f16, KV_F16)
QMM_KV_ENTRY_POINTS(q8_0, KV_Q8_0)
QMM_KV_ENTRY_POINTS(q4_0, KV_Q4_0)

int64_t qmm_attn_decode_workspace(int64_t B, int64_t Hq, int64_t heads, int64_t dim, int64_t max_len,
                                  int64_t window) {
    return workspace_bytes(B, Hq, heads, dim, max_len, window);
}

}  // extern "C"
