"""CPU checks of the attention operators: refusals (before any device call),
frequency tables, the cache layout's arithmetic as the kernels compile it, and
the binding's checks."""
import ctypes
import math
import os
import shutil
import subprocess

import numpy as np
import pytest

from attention_ref import code_places, side_bytes
from conftest import ROOT

A = 1 << 20          # a 16-byte aligned fake device address (never dereferenced)
FORMATS = ("f16", "q8_0", "q4_0")


@pytest.fixture(scope="module")
def q():
    import matmul_quantize_q8_amd as q
    q.lib()
    return q


class Plan(ctypes.Structure):
    _fields_ = [("freqs", ctypes.c_void_p), ("rot", ctypes.c_int64), ("order", ctypes.c_int32),
                ("mscale", ctypes.c_float)]


class Cache(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("page", ctypes.c_int64),
                ("heads", ctypes.c_int64), ("dim", ctypes.c_int64)]


def _p(s):
    return ctypes.addressof(s) if s is not None else None


GOOD_PLAN = dict(freqs=A, rot=64, order=0, mscale=1.0)
GOOD_CACHE = dict(data=A, n_pages=4, page=32, heads=2, dim=64)


def rope(L, plan=GOOD_PLAN, x=A, y=A + 4096, dt=0, pos=A, T=3, H=2, D=64, xs=(128, 64), ys=(128, 64)):
    p = Plan(**plan) if plan else None
    return L.qmm_rope(_p(p), x, y, dt, pos, 0, T, H, D, *xs, *ys, None)


@pytest.mark.parametrize("change,code", [
    (dict(plan=None), 2), (dict(plan=dict(GOOD_PLAN, freqs=None)), 2), (dict(plan=dict(GOOD_PLAN, freqs=A + 4)), 3),
    (dict(plan=dict(GOOD_PLAN, rot=0)), 1), (dict(plan=dict(GOOD_PLAN, rot=63)), 1),
    (dict(plan=dict(GOOD_PLAN, rot=66)), 1), (dict(plan=dict(GOOD_PLAN, order=2)), 1),
    (dict(x=None), 2), (dict(y=None), 2), (dict(pos=None), 2), (dict(pos=A + 2), 3), (dict(x=A + 8), 3),
    (dict(x=A + 4, dt=1), 3), (dict(dt=3), 1), (dict(dt=-1), 1), (dict(T=0), 1), (dict(T=1 << 31), 1), (dict(T=1 << 24), 1),
    (dict(H=0), 1), (dict(H=4097), 1), (dict(D=66), 1), (dict(D=260), 1), (dict(xs=(126, 64)), 3),
    (dict(ys=(128, 62)), 3), (dict(xs=(-128, 64)), 1), (dict(xs=(1 << 39, 64)), 1), (dict(xs=(1 << 62, 1 << 62)), 1),
])
def test_rope_refusals(q, change, code):
    assert rope(q.lib(), **change) == code


BAD_CACHES = [(dict(data=None), 2), (dict(data=A + 8), 3), (dict(n_pages=0), 1), (dict(n_pages=1 << 33), 1),
              (dict(page=8), 1), (dict(page=48), 1), (dict(page=8192), 1), (dict(heads=0), 1), (dict(heads=5000), 1),
              (dict(dim=80), 1), (dict(dim=32), 1), (dict(dim=320), 1)]


def write(L, fmt, cache=None, k=A, v=A, dt=0, slots=A, T=3, ks=(128, 64), vs=(128, 64), no_cache=False):
    c = Cache(**dict(GOOD_CACHE, **(cache or {})))
    return getattr(L, "qmm_kv_write_" + fmt)(None if no_cache else _p(c), k, v, dt, slots, T, *ks, *vs, None)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("change,code", [(dict(cache=c), s) for c, s in BAD_CACHES] + [
    (dict(no_cache=True), 2), (dict(k=None), 2), (dict(v=None), 2), (dict(k=A + 8), 3), (dict(v=A + 4, dt=2), 3),
    (dict(slots=None), 2), (dict(slots=A + 4), 3), (dict(T=0), 1), (dict(dt=7), 1), (dict(ks=(130, 64)), 3),
    (dict(vs=(128, -4)), 1)])
def test_kv_write_refusals(q, fmt, change, code):
    assert write(q.lib(), fmt, **change) == code


def rope_write(L, fmt, plan=GOOD_PLAN, cache=None, qq=A, qo=A, pos=A, Hq=4, qs=(256, 64)):
    c, p = Cache(**dict(GOOD_CACHE, **(cache or {}))), Plan(**plan) if plan else None
    return getattr(L, "qmm_rope_kv_write_" + fmt)(_p(p), _p(c), qq, qo, A, A, 0, pos, A, 3, Hq, *qs, 256, 64, 128,
                                                  64, 128, 64, None)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("change,code", [
    (dict(plan=None), 2), (dict(plan=dict(GOOD_PLAN, rot=65)), 1), (dict(qq=None), 2), (dict(qo=None), 2),
    (dict(qo=A + 8), 3), (dict(pos=None), 2), (dict(pos=A + 1), 3), (dict(Hq=0), 1), (dict(Hq=-1), 1),
    (dict(Hq=5000), 1), (dict(qs=(255, 64)), 3), (dict(cache=dict(dim=100)), 1)])
def test_rope_kv_write_refusals(q, fmt, change, code):
    assert rope_write(q.lib(), fmt, **change) == code


def read(L, fmt, cache=None, slots=A, k=A, v=A, dt=0, T=3, ks=(128, 64)):
    c = Cache(**dict(GOOD_CACHE, **(cache or {})))
    return getattr(L, "qmm_kv_read_" + fmt)(_p(c), slots, k, v, dt, T, *ks, 128, 64, None)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("change,code", [(dict(cache=c), s) for c, s in BAD_CACHES] + [
    (dict(k=None, v=None), 2), (dict(k=A + 8), 3), (dict(k=None, v=A + 8), 3), (dict(slots=None), 2), (dict(T=0), 1),
    (dict(dt=3), 1), (dict(ks=(128, 63)), 3)])
def test_kv_read_refusals(q, fmt, change, code):
    assert read(q.lib(), fmt, **change) == code


def attn(L, fmt, cache=None, qq=A, out=A, dt=0, pages=A, n=8, lens=A, B=2, Hq=4, max_len=256, scale=0.125,
         softcap=0.0, window=0, mask=None, ms=0, lse=None, qs=(256, 64), ws=A, ws_bytes=1 << 39):
    c = Cache(**dict(GOOD_CACHE, **(cache or {})))
    return getattr(L, "qmm_attn_decode_" + fmt)(_p(c), qq, out, dt, pages, n, lens, B, Hq, max_len, scale, softcap,
                                                window, mask, ms, lse, *qs, 256, 64, ws, ws_bytes, None)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("change,code", [(dict(cache=c), s) for c, s in BAD_CACHES] + [
    (dict(qq=None), 2), (dict(out=None), 2), (dict(pages=None), 2), (dict(lens=None), 2), (dict(ws=None), 2),
    (dict(ws=A + 8), 3), (dict(qq=A + 8), 3), (dict(pages=A + 2), 3), (dict(lse=A + 2), 3),
    (dict(mask=A + 1, ms=256), 3), (dict(mask=A, ms=255), 1), (dict(B=0), 1), (dict(B=65536), 1), (dict(Hq=3), 1),
    (dict(Hq=0), 1), (dict(max_len=0), 1), (dict(max_len=257), 1), (dict(n=0), 1), (dict(dt=5), 1),
    (dict(window=-1), 1), (dict(softcap=-1.0), 1), (dict(softcap=math.nan), 1), (dict(softcap=math.inf), 1),
    (dict(scale=math.nan), 1), (dict(ws_bytes=0), 1), (dict(qs=(256, 62)), 3)])
def test_attn_decode_refusals(q, fmt, change, code):
    assert attn(q.lib(), fmt, **change) == code


def test_workspace_that_is_a_byte_short(q):
    need = q.qmm_attn_decode_workspace(2, 4, 2, 64, 256)
    assert need > 0
    assert attn(q.lib(), "q8_0", ws_bytes=need - 1) == 1


def test_workspace_grows_with_batch_and_length(q):
    """What suffices for a batch and a length suffices for smaller ones."""
    size = q.qmm_attn_decode_workspace
    for Hq, heads, dim in ((32, 8, 128), (32, 32, 64), (64, 1, 256), (20, 1, 96)):
        for n in (1, 255, 256, 257, 4096, 131072):
            of = [size(B, Hq, heads, dim, n) for B in range(1, 600, 7)]
            assert of == sorted(of)
        for B in (1, 3, 64, 511):
            of = [size(B, Hq, heads, dim, n) for n in range(1, 20000, 97)]
            assert of == sorted(of)
            assert size(B, Hq, heads, dim, 5000, 300) <= size(B, Hq, heads, dim, 5000)


@pytest.mark.parametrize("args", [(0, 4, 2, 64, 256), (2, 3, 2, 64, 256), (2, 4, 0, 64, 256), (2, 4, 2, 65, 256),
                                  (2, 4, 2, 64, 0), (2, 4, 2, 64, 1 << 31), (2, 4, 2, 64, 256, -1)])
def test_no_workspace_for_sizes_outside_the_limits(q, args):
    assert q.qmm_attn_decode_workspace(*args) == 0


def test_page_bytes(q):
    for fmt in FORMATS:
        for page, heads, dim in ((16, 1, 64), (64, 8, 128), (128, 3, 96)):
            assert q.kv_page_bytes(fmt, page, heads, dim) == 2 * heads * side_bytes(fmt, page, dim)
        assert q.kv_page_bytes(fmt, 24, 1, 64) == 0 and q.kv_page_bytes(fmt, 16, 1, 72) == 0


# ---------------------------------------------------------------------------
# Frequencies
# ---------------------------------------------------------------------------
def test_plain_linear_ntk_frequencies(q):
    f, ms = q.qmm_rope_freqs(128, 1e4)
    want = 1e4 ** (-np.arange(64) / 64)
    assert ms == 1.0 and np.allclose(f.numpy(), want, rtol=1e-14, atol=0)
    assert np.allclose(q.qmm_rope_freqs(128, 1e4, "linear", 8)[0].numpy(), want / 8, rtol=1e-14, atol=0)
    ntk = q.qmm_rope_freqs(128, 1e4, "ntk", 4)[0].numpy()
    assert ntk[0] == 1.0 and math.isclose(ntk[-1], want[-1] / 4, rel_tol=1e-12)     # fastest kept, slowest / factor
    assert np.all(np.diff(ntk) < 0)


def test_yarn_and_band_frequencies(q):
    plain = q.qmm_rope_freqs(128, 1e4)[0].numpy()
    f, ms = q.qmm_rope_freqs(128, 1e4, "yarn", 16, 4096, 1, 32)
    turns = 4096 * plain / (2 * math.pi)
    f = f.numpy()
    assert math.isclose(ms, 1 + 0.1 * math.log(16), rel_tol=1e-6)
    i = np.arange(64)
    first = math.floor(128 * math.log(4096 / (32 * 2 * math.pi)) / (2 * math.log(1e4)))
    last = math.ceil(128 * math.log(4096 / (2 * math.pi)) / (2 * math.log(1e4)))
    s = np.clip((i - first) / (last - first), 0, 1)
    assert np.allclose(f, plain * (1 - s) + plain / 16 * s, rtol=1e-13, atol=0)
    assert np.all(f[turns > 33] == plain[turns > 33])
    assert np.allclose(f[turns < 0.9], plain[turns < 0.9] / 16, rtol=1e-14)
    g, ms = q.qmm_rope_freqs(128, 5e5, "bands", 8, 8192, 1, 4)
    g, plain = g.numpy(), q.qmm_rope_freqs(128, 5e5)[0].numpy()
    turns = 8192 * plain / (2 * math.pi)
    mid = (turns >= 1) & (turns <= 4)
    s = (turns - 1) / 3
    assert ms == 1.0 and mid.any()
    assert np.all(g[turns > 4] == plain[turns > 4])
    assert np.allclose(g[turns < 1], plain[turns < 1] / 8, rtol=1e-14, atol=0)
    assert np.allclose(g[mid], plain[mid] * ((1 - s[mid]) / 8 + s[mid]), rtol=1e-13, atol=0)


@pytest.mark.parametrize("args", [(0, 1e4), (63, 1e4), (258, 1e4), (64, 1.0), (64, math.inf), (64, math.nan),
                                  (64, 1e4, "linear", 0.5), (64, 1e4, "linear", math.nan), (2, 1e4, "ntk", 2),
                                  (64, 1e4, "yarn", 2, 0, 1, 32), (64, 1e4, "yarn", 2, 4096, 4, 4),
                                  (64, 1e4, "bands", 2, 4096, 0, 4), (64, 1e4, "bands", 2, 4096, 1, math.inf)])
def test_frequency_refusals(q, args):
    with pytest.raises(q.QmmError) as e:
        q.qmm_rope_freqs(*args)
    assert e.value.code == "QMM_E_SHAPE"


def test_frequency_refusals_by_code(q):
    L = q.lib()
    assert L.qmm_rope_freqs(None, None, 64, 1e4, 0, 1.0, 0.0, 0.0, 0.0) == 2
    buf = (ctypes.c_double * 32)()
    assert L.qmm_rope_freqs(ctypes.addressof(buf), None, 64, 1e4, 5, 1.0, 0.0, 0.0, 0.0) == 1
    assert L.qmm_rope_freqs(ctypes.addressof(buf), None, 64, 1e4, 0, 1.0, 0.0, 0.0, 0.0) == 0 and buf[0] == 1.0


# ---------------------------------------------------------------------------
# The layout, as the kernels compile it, on the host
# ---------------------------------------------------------------------------
HIPCC = shutil.which("hipcc") or ("/opt/rocm/bin/hipcc" if os.path.exists("/opt/rocm/bin/hipcc") else None)

LAYOUT = r"""
#include <cstdio>
#include "kv_layout.h"
using namespace qmm;
template <int F, int NB> void dump(const char *name) {
    using K = Kv<F, NB>;
    static_assert(K::U % K::P == 0 || K::P % K::U == 0, "a value's pieces lie in one unit, or are whole units");
    static_assert(K::P <= K::U, "a value's piece lies in one unit");
    printf("%s %d side", name, 32 * NB);
    for (int page : {16, 32, 256}) printf(" %lld", (long long)K::side_bytes(page));
    printf("\n");
    for (int t = 0; t < 32; ++t) {
        printf("%s %d k %d", name, 32 * NB, t);
        for (int n = 0; n < 32 * NB; ++n) {
            const int j = K::byte_of(n / 32 * 8 + n % 8);
            printf(" %d", K::key_unit(t, n % 32 / 8, j / K::U) + j % K::U);
        }
        printf("\n%s %d v %d", name, 32 * NB, t);
        for (int n = 0; n < 32 * NB; ++n) printf(" %d", K::value_byte(t, n % 32 / 2, K::byte_of(n / 32 * 2 + n % 2)));
        printf("\n");
    }
}
template <int F> void all(const char *n) { dump<F, 2>(n); dump<F, 3>(n); dump<F, 4>(n); dump<F, 6>(n); dump<F, 8>(n); }
int main() {
    all<KV_F16>("f16"); all<KV_Q8_0>("q8_0"); all<KV_Q4_0>("q4_0");
    KvCache c = {nullptr, 5, 6, 3};
    long long bad[] = {-1, -(1LL << 40), 5, 1LL << 40, 0x7fffffffffffffffLL, (-1LL) >> 6, -64 >> 6};
    for (long long p : bad) printf("bad %d\n", (int)c.has_page(p));
    for (int p = 0; p < 5; ++p) printf("good %d\n", (int)c.has_page(p));
    KvCache far = {nullptr, 1 << 20, 6, 8};
    printf("far %lld\n", (long long)(far.page_at((1 << 20) - 1, 8704) - far.page_at(0, 8704)));
}
"""


@pytest.mark.skipif(HIPCC is None, reason="hipcc not found")
def test_layout_arithmetic_of_the_kernels(tmp_path, q):
    src, exe = tmp_path / "layout.hip", tmp_path / "layout"
    src.write_text(LAYOUT)
    cmd = [HIPCC, "--offload-arch=gfx950", "-O1", "-std=c++17", "-I",
           os.path.join(ROOT, "matmul_quantize_q8_amd", "csrc"), str(src), "-o", str(exe),
           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]
    out = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]
    lines = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60).stdout.splitlines()
    seen = 0
    for line in lines:
        w = line.split()
        if w[0] == "bad":
            assert w[1] == "0"
        elif w[0] == "good":
            assert w[1] == "1"
        elif w[0] == "far":
            assert int(w[1]) == ((1 << 20) - 1) * 8 * 2 * 8704
        elif w[2] == "side":
            assert [int(v) for v in w[3:]] == [side_bytes(w[0], p, int(w[1])) for p in (16, 32, 256)]
        else:
            seen += 1
            fmt, dim, values, t = w[0], int(w[1]), w[2] == "v", int(w[3])
            at, _ = code_places(fmt, dim, t, values)
            assert [int(v) for v in w[4:]] == at.tolist(), line[:60]
    assert seen == 3 * 5 * 64


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
def test_layout_uses_every_byte_once(fmt, dim):
    for values in (False, True):
        taken = []
        for t in range(32):
            at, high = code_places(fmt, dim, t, values)
            taken += (2 * at + high).tolist() if fmt == "q4_0" else at.tolist()
        step = 2 if fmt == "f16" else 1
        size = 32 * dim * step            # bytes, or a q4_0 row's halves
        assert sorted(taken) == list(range(0, size, step))


SPLIT = r"""
#include <cstdio>
#include "attn_decode.hip"
namespace qmm {
hipError_t launch_attn_f16(int, int, const AttnArgs &, int64_t, hipStream_t) { return hipSuccess; }
hipError_t launch_attn_q8_0(int, int, const AttnArgs &, int64_t, hipStream_t) { return hipSuccess; }
hipError_t launch_attn_q4_0(int, int, const AttnArgs &, int64_t, hipStream_t) { return hipSuccess; }
}
using namespace qmm;
int main() {
    long long cases = 0, bad = 0;
    const long long heads[][2] = {{1, 1}, {8, 1}, {32, 8}, {32, 32}, {14, 2}, {20, 1}, {64, 2}, {128, 16}, {17, 1}};
    const long long lens[] = {1, 2, 255, 256, 257, 300, 511, 512, 513, 700, 1000, 1025, 4096, 5000, 40000, 131072, 1000003,
                              (1LL << 31) - 8193};
    for (auto &h : heads)
        for (long long B = 1; B <= 1100; B += B < 80 ? 1 : 37)
            for (long long n : lens)
                for (long long w : {0LL, 1LL, 100LL, 500LL, 3000LL, n - 1, n, n + 5}) {
                    if (w < 0) continue;
                    const AttnSplit s = attn_split(B, h[0], h[1], n, w);
                    const long long span = attn_span(n, w);
                    ++cases;
                    // the chunks cover the span, none is empty for every sequence, none is cut inside a group,
                    // positions stay below 2^31, and the partial sums fit the workspace
                    bool ok = s.splits >= 1 && s.chunk % kGroup == 0 && (long long)s.chunk * s.splits >= span &&
                              (long long)s.chunk * (s.splits - 1) < span && (long long)s.chunk > 0 &&
                              n + 8192 <= (1LL << 31) - 1;
                    for (long long D : {64LL, 256LL})
                        ok = ok && part_bytes(B, h[0], s.splits, D) <= attn_workspace(B, h[0], h[1], D, n, w);
                    if (!ok && bad++ < 5) printf("bad %lld %lld %lld %lld %lld\n", h[0], h[1], B, n, w);
                }
    printf("cases %lld bad %lld\n", cases, bad);
}
"""


@pytest.mark.skipif(HIPCC is None, reason="hipcc not found")
def test_split_of_the_work_fits_the_workspace(tmp_path):
    src, exe = tmp_path / "split.hip", tmp_path / "split"
    src.write_text(SPLIT)
    cmd = [HIPCC, "--offload-arch=gfx950", "-O1", "-std=c++17", "-I",
           os.path.join(ROOT, "matmul_quantize_q8_amd", "csrc"), str(src), "-o", str(exe),
           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]
    out = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]
    text = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60).stdout
    assert text.strip().endswith("bad 0") and text.startswith("cases "), text


# ---------------------------------------------------------------------------
# The binding's checks
# ---------------------------------------------------------------------------
def test_binding_refuses_cpu_tensors_and_wrong_types(q):
    import torch
    with pytest.raises(ValueError):
        q.KVCache("q8_0", torch.zeros(q.kv_page_bytes("q8_0", 16, 1, 64), dtype=torch.uint8), 16, 1, 64)
    with pytest.raises(ValueError):
        q.KVCache("q5_0", torch.zeros(64, dtype=torch.uint8), 16, 1, 64)
    with pytest.raises(ValueError):
        q.KVCache("q8_0", torch.zeros(64, dtype=torch.uint8), 20, 1, 64)
    with pytest.raises(ValueError):
        q.RopePlan(torch.zeros(32, dtype=torch.float64))
    with pytest.raises(ValueError):
        q.RopePlan(torch.zeros(32, dtype=torch.float64), "other")
    with pytest.raises(ValueError):
        q.attn_workspace(1, 3, 2, 64, 16)
    with pytest.raises(ValueError):
        q.qmm_rope_freqs(64, scaling="other")
