"""The attention operators on an MI355X against plain 64-bit forms.

Rotation, cache writes and cache reads are compared bit for bit: every step is
a stated, correctly rounded operation.  Attention is compared within a bound
that is derived from the formula (see `bound`)."""
import math

import numpy as np
import pytest

import attention_ref as ref

pytestmark = pytest.mark.gpu

FORMATS = ("f16", "q8_0", "q4_0")
DIMS = (64, 96, 128, 192, 256)
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module")
def env():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import matmul_quantize_q8_amd as q
    import oracle
    q.lib()
    oracle.lib()
    return torch, q, oracle


def _say(*a):
    print("[case]", *a, flush=True)


def _t(torch, dtype):
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[dtype]


def _dev(torch, a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to("cuda")
    return t if dtype is None else t.to(_t(torch, dtype))


def _np(t):
    return t.detach().cpu().double().numpy()


def _round(torch, x, dtype):
    """f64 values of f32 values rounded to a row type, to nearest even (torch, CPU)."""
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(_t(torch, dtype)).double().numpy()


def _rows(torch, rng, shape, dtype, sigma=1.0):
    """A GPU tensor of rows and its values in f32."""
    x = torch.from_numpy((sigma * rng.standard_normal(shape)).astype(np.float32)).to(_t(torch, dtype))
    return x.to("cuda"), x.float().numpy()


def _freqs(rot):
    return 1e4 ** (-np.arange(rot // 2) * 2.0 / rot)


# ---------------------------------------------------------------------------
# Rotation: bit for bit
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("order", ["half", "interleaved"])
@pytest.mark.parametrize("T,H,D,rot", [(1, 1, 64, 64), (1, 40, 128, 128), (5, 3, 96, 96), (17, 2, 256, 256),
                                       (3, 5, 192, 64), (7, 9, 128, 2), (4, 3, 64, 62), (6, 33, 64, 22),
                                       (2, 3, 80, 80), (3, 2, 4, 4), (2, 7, 20, 6), (1030, 1, 64, 64)])
def test_rope(env, dtype, order, T, H, D, rot):
    torch, q, _ = env
    _say("rope", dtype, order, T, H, D, rot)
    rng = np.random.default_rng(T * 1000 + H + D + rot)
    x, xf = _rows(torch, rng, (T, H, D), dtype)
    pos = rng.integers(-1000, 1 << 20, T).astype(np.int32)
    pos[0] = 2 ** 31 - 1 if T > 1 else 1000003
    plan = q.RopePlan(_dev(torch, _freqs(rot)), order, 1.25)
    y = torch.full_like(x, float("nan"))
    q.qmm_rope(x, y, _dev(torch, pos), plan)
    want = ref.rotated(xf, pos, _freqs(rot), order, 1.25)
    assert np.array_equal(_np(y), _round(torch, want, dtype))
    q.qmm_rope(x, x, _dev(torch, pos), plan, inverse=True)          # in place, the other way
    want = ref.rotated(xf, pos, _freqs(rot), order, 1.25, inverse=True)
    assert np.array_equal(_np(x), _round(torch, want, dtype))


@pytest.mark.parametrize("order", ["half", "interleaved"])
def test_rope_gradient_and_differences(env, order):
    """The inverse takes dL/dy to dL/dx: against differences of L = sum(w y) in
    f64 (L is linear, so a difference is exact up to f64 rounding; each kernel
    value carries 3 f32 roundings of products below |a| + |b|)."""
    torch, q, _ = env
    _say("rope gradient", order)
    rng = np.random.default_rng(5)
    T, H, D, rot = 3, 2, 64, 48
    pos, f = np.array([3, 77777, 12], np.int32), _freqs(48)
    w, wf = _rows(torch, rng, (T, H, D), "f32")
    g = torch.empty_like(w)
    q.qmm_rope(w, g, _dev(torch, pos), q.RopePlan(_dev(torch, f), order), inverse=True)

    def turned64(x):
        ang = pos.astype(np.float64)[:, None] * f
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        i = np.arange(rot // 2)
        ia, ib = (i, i + rot // 2) if order == "half" else (2 * i, 2 * i + 1)
        y = x.copy()
        y[..., ia], y[..., ib] = x[..., ia] * c - x[..., ib] * s, x[..., ia] * s + x[..., ib] * c
        return y
    for t, h, d in [(0, 0, 0), (1, 1, 23), (1, 0, 24), (2, 1, 47), (2, 0, 48), (0, 1, 63), (1, 1, 1)]:
        x = rng.standard_normal((T, H, D))
        step = np.zeros_like(x)
        step[t, h, d] = 0.5
        diff = (np.sum(wf * turned64(x + step)) - np.sum(wf * turned64(x - step)))
        tol = 4 * 2.0 ** -24 * 2 * np.abs(wf[t, h]).max() + 1e-12 * np.abs(wf).sum()
        assert abs(float(g[t, h, d]) - diff) <= tol
    # forward then inverse is the identity within the roundings of both
    y, z = torch.empty_like(w), torch.empty_like(w)
    plan = q.RopePlan(_dev(torch, f), order)
    q.qmm_rope(w, y, _dev(torch, pos), plan)
    q.qmm_rope(y, z, _dev(torch, pos), plan, inverse=True)
    assert float((z - w).abs().max()) <= 16 * 2.0 ** -24 * np.abs(wf).max()


def test_rope_strides_and_rest(env):
    torch, q, _ = env
    _say("rope strides")
    rng = np.random.default_rng(8)
    T, H, D = 9, 6, 64
    qkv, f = _rows(torch, rng, (T, 2 * H + 1, D), "bf16")
    x, pos = qkv[:, 3:3 + H], np.arange(T, dtype=np.int32)
    out = torch.full((H, T, D + 8), 7.0, dtype=torch.bfloat16, device="cuda")      # heads outermost, padded rows
    y = out.permute(1, 0, 2)[..., :D]
    q.qmm_rope(x, y, _dev(torch, pos), q.RopePlan(_dev(torch, _freqs(32))))
    want = ref.rotated(f[:, 3:3 + H], pos, _freqs(32), "half")
    assert np.array_equal(_np(y), _round(torch, want, "bf16"))
    assert bool((out[..., D:] == 7.0).all())
    with pytest.raises(ValueError):
        q.qmm_rope(x, y.float(), _dev(torch, pos), q.RopePlan(_dev(torch, _freqs(32))))
    with pytest.raises(ValueError):
        q.qmm_rope(x, y, _dev(torch, pos.astype(np.int64)), q.RopePlan(_dev(torch, _freqs(32))))


# ---------------------------------------------------------------------------
# Cache: bit for bit
# ---------------------------------------------------------------------------
def _pool(torch, q, fmt, n_pages, page, heads, dim):
    """A cache whose every byte is 0xff: NaN as an f16 and as a scale."""
    data = torch.full((n_pages * q.kv_page_bytes(fmt, page, heads, dim),), 255, dtype=torch.uint8, device="cuda")
    return q.KVCache(fmt, data, page, heads, dim)


def _edge(x):
    """Zero blocks, ties of magnitude, tiny and large values, in rows [T][H][D]."""
    x[0, 0, :32] = 0.0
    x[0, 0, 33], x[0, 0, 40] = -3.5, 3.5
    x[0, -1, 32:64] = 0.01
    x[0, -1, 35], x[0, -1, 50] = 0.5, -0.5
    x[-1, 0, 32:64] *= 2.0 ** -20
    x[-1, -1, :32] *= 1000.0
    return x


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("T,heads,page,dtype", [(1, 1, 16, "f32"), (37, 3, 16, "bf16"), (21, 2, 64, "f16")])
def test_write_and_read(env, fmt, dim, T, heads, page, dtype):
    torch, q, orc = env
    _say("write", fmt, dim, T, heads, page, dtype)
    rng = np.random.default_rng(dim + T)
    n_pages = -(-T // page) + 2
    cache = _pool(torch, q, fmt, n_pages, page, heads, dim)
    kf, vf = (_edge(rng.standard_normal((T, heads, dim)).astype(np.float32)) for _ in range(2))
    k, v = (torch.from_numpy(x).to(_t(torch, dtype)) for x in (kf, vf))
    kf, vf = k.float().numpy(), v.float().numpy()
    slots = rng.permutation(n_pages * page)[:T].astype(np.int64)
    if T > 4:
        slots[1], slots[3] = -1, n_pages * page          # skipped
    q.KV_WRITE[fmt](k.to("cuda"), v.to("cuda"), cache, _dev(torch, slots))
    raw = cache.data.cpu().numpy()
    live = [i for i in range(T) if 0 <= slots[i] < n_pages * page]
    wk, wv = ref.through_cache(kf, fmt, orc), ref.through_cache(vf, fmt, orc)
    assert np.array_equal(ref.read_rows(raw, fmt, page, heads, dim, slots[live], False), wk[live])
    assert np.array_equal(ref.read_rows(raw, fmt, page, heads, dim, slots[live], True), wv[live])
    untouched = [s for s in range(n_pages * page) if s not in set(slots)]
    with np.errstate(invalid="ignore"):
        assert np.isnan(ref.read_rows(raw, fmt, page, heads, dim, untouched[:40], True)).all()
    for out in ("f32", "f16", "bf16"):                   # read back
        ko, vo = (torch.zeros(T, heads, dim, dtype=_t(torch, out), device="cuda") for _ in range(2))
        q.KV_READ[fmt](cache, _dev(torch, slots), ko, vo)
        for got, want in ((ko, wk), (vo, wv)):
            want = _round(torch, want, out)
            want[[i for i in range(T) if i not in live]] = np.nan
            assert np.array_equal(_np(got), want, equal_nan=True)
        only = torch.zeros_like(vo)
        q.KV_READ[fmt](cache, _dev(torch, slots), None, only)
        assert np.array_equal(_np(only), _np(vo), equal_nan=True)
        q.KV_READ[fmt](cache, _dev(torch, slots), only, None)
        assert np.array_equal(_np(only), _np(ko), equal_nan=True)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim,rot,order,dtype,T,Hq,heads", [
    (128, 128, "half", "f16", 16, 32, 8), (64, 64, "interleaved", "f32", 1, 14, 2), (96, 96, "half", "bf16", 33, 3, 3),
    (192, 62, "half", "f32", 5, 8, 1), (256, 128, "half", "bf16", 3, 5, 5), (128, 22, "interleaved", "f16", 200, 4, 4)])
def test_rope_and_write(env, fmt, dim, rot, order, dtype, T, Hq, heads):
    torch, q, orc = env
    _say("rope+write", fmt, dim, rot, order, dtype, T)
    rng = np.random.default_rng(dim + rot + T)
    page, n_pages = 32, -(-T // 32) + 1
    cache = _pool(torch, q, fmt, n_pages, page, heads, dim)
    qkv, f = _rows(torch, rng, (T, Hq + 2 * heads, dim), dtype)
    qq, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + heads], qkv[:, Hq + heads:]
    fq, fk, fv = f[:, :Hq], f[:, Hq:Hq + heads], f[:, Hq + heads:]
    pos = rng.integers(0, 1 << 20, T).astype(np.int32)
    slots = rng.permutation(n_pages * page)[:T].astype(np.int64)
    qo = torch.empty(T, Hq, dim, dtype=qkv.dtype, device="cuda")
    plan = q.RopePlan(_dev(torch, _freqs(rot)), order)
    q.ROPE_KV_WRITE[fmt](qq, qo, k, v, cache, _dev(torch, slots), _dev(torch, pos), plan)
    raw = cache.data.cpu().numpy()
    assert np.array_equal(_np(qo), _round(torch, ref.rotated(fq, pos, _freqs(rot), order), dtype))
    wk = ref.through_cache(ref.rotated(fk, pos, _freqs(rot), order), fmt, orc)
    assert np.array_equal(ref.read_rows(raw, fmt, page, heads, dim, slots, False), wk)
    assert np.array_equal(ref.read_rows(raw, fmt, page, heads, dim, slots, True), ref.through_cache(fv, fmt, orc))
    q.ROPE_KV_WRITE[fmt](qq, qq, k, v, cache, _dev(torch, slots), _dev(torch, pos), plan)      # queries in place
    assert torch.equal(qq, qo)
    assert np.array_equal(cache.data.cpu().numpy(), raw)


@pytest.mark.parametrize("fmt", FORMATS)
def test_many_tokens_written(env, fmt):
    """More tokens than workgroups in flight: neighbouring tokens share lines of
    the value codes and no write may lose another's bytes."""
    torch, q, orc = env
    T, heads, dim, page = 3001, 2, 128, 64
    _say("many tokens", fmt)
    rng = np.random.default_rng(3)
    cache = _pool(torch, q, fmt, 48, page, heads, dim)
    k, kf = _rows(torch, rng, (T, heads, dim), "f32")
    v, vf = _rows(torch, rng, (T, heads, dim), "f32")
    slots = np.arange(T, dtype=np.int64) + 7
    q.KV_WRITE[fmt](k, v, cache, _dev(torch, slots))
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    q.KV_READ[fmt](cache, _dev(torch, slots), ko, vo)
    assert np.array_equal(_np(ko), ref.through_cache(kf, fmt, orc))
    assert np.array_equal(_np(vo), ref.through_cache(vf, fmt, orc))


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------
def bound(reach, mag, out, n, dim, dtype, scale_max=0.0):
    """Per output: a score is off by at most es = reach * (2^-21 + dim * 2^-24)
    (queries split to 22 bits, products summed in f32) plus 8 roundings of the
    score itself; a weight relative by 2 es (numerator and maximum) plus 2^-20
    (exp, its argument's rounding at arguments up to about 16 above which the
    weight is below 1e-7, the split to 22 bits); the sums over n positions add
    n * 2^-24.  Numerator and denominator together double it.  The final
    rounding to the row type is half a step of the result."""
    es = reach * (2.0 ** -21 + dim * 2.0 ** -24) + (reach + scale_max) * 8 * 2.0 ** -24
    rel = 2 * (2 * es + 2.0 ** -20 + n * 2.0 ** -24)
    return rel[:, None] * mag + HALF_STEP[dtype] * np.abs(out) + 2.0 ** -25, 2 * es + 2.0 ** -20 + n * 2.0 ** -24


class Setup:
    """Sequences in a paged cache: written through the library, the pool poisoned
    elsewhere, pages in random order, page-table padding -1."""

    def __init__(self, env, fmt, lens, Hq, heads, dim, page, dtype, seed, sigma_q=1.5, max_len=None):
        torch, q, orc = env
        rng = np.random.default_rng(seed)
        self.env, self.fmt, self.lens, self.dtype, self.dim, self.heads = env, fmt, lens, dtype, dim, heads
        self.max_len = max(max(lens), 1) if max_len is None else max_len
        used = [-(-n // page) for n in lens]
        self.width = -(-self.max_len // page) + 1
        self.cache = _pool(torch, q, fmt, sum(used) + 2, page, heads, dim)
        order, at = rng.permutation(sum(used) + 2), 0
        self.table = np.full((len(lens), self.width), -1, np.int32)
        self.k, self.v = [], []
        for b, n in enumerate(lens):
            self.table[b, :used[b]] = order[at:at + used[b]]
            at += used[b]
            k = rng.standard_normal((n, heads, dim)).astype(np.float32)
            v = rng.standard_normal((n, heads, dim)).astype(np.float32)
            if n:
                i = np.arange(n)
                slots = self.table[b][i // page].astype(np.int64) * page + i % page
                q.KV_WRITE[fmt](_dev(torch, k), _dev(torch, v), self.cache, _dev(torch, slots))
            self.k.append(ref.through_cache(k, fmt, orc) if n else k.astype(np.float64))
            self.v.append(ref.through_cache(v, fmt, orc) if n else v.astype(np.float64))
        self.q, qf = _rows(torch, rng, (len(lens), Hq, dim), dtype, sigma_q)
        self.qf = qf.astype(np.float64)
        self.out = torch.full_like(self.q, float("nan"))
        self.lse = torch.full((len(lens), Hq), float("nan"), device="cuda")
        self.pages = _dev(torch, self.table)
        self.len = _dev(torch, np.array(lens, np.int32))
        self.ws = q.attn_workspace(len(lens), Hq, heads, dim, self.max_len)

    def run(self, **kw):
        _, q, _ = self.env
        q.ATTN_DECODE[self.fmt](self.q, self.out, self.cache, self.pages, self.len, self.max_len, self.ws,
                                lse=self.lse, **kw)

    def check(self, window=0, softcap=0.0, mask=None, scale=None, rows=None):
        scale = self.dim ** -0.5 if scale is None else scale
        got, lse = _np(self.out), _np(self.lse)
        for b, n in enumerate(self.lens) if rows is None else ((b, self.lens[b]) for b in rows):
            seen = np.arange(max(0, n - window) if window else 0, n)
            add = None
            if mask is not None:
                seen = seen[mask[b, seen] != -np.inf]
                add = mask[b, seen].astype(np.float64)
            o, l, reach, mag = ref.attention(self.qf[b], self.k[b][seen], self.v[b][seen], scale, softcap, add)
            if len(seen) == 0:
                assert np.all(got[b] == 0) and np.all(lse[b] == -np.inf), b
                continue
            top = 0.0 if add is None else float(np.abs(add[add > -1e30]).max(initial=0.0))
            tol, ltol = bound(reach, mag, o, len(seen), self.dim, self.dtype, top)
            err = np.abs(got[b] - o)
            assert np.all(err <= tol), (b, n, float((err / tol).max()), float(err.max()))
            if add is None or np.all(add > -1e30):
                assert np.all(np.abs(lse[b] - l) <= ltol + 2.0 ** -23 * np.abs(l)), (b, n)


LENS = [0, 1, 2, 15, 16, 17, 31, 33, 64, 100, 129, 255, 256, 257, 700]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("Hq,heads,page,dtype", [(14, 2, 16, "f32"), (4, 4, 64, "f16"), (20, 1, 32, "bf16")])
def test_attention(env, fmt, dim, Hq, heads, page, dtype):
    _say("attention", fmt, dim, Hq, heads, page, dtype)
    s = Setup(env, fmt, LENS, Hq, heads, dim, page, dtype, dim + Hq)
    s.run()
    s.check()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("Hq,heads", [(1, 1), (16, 1), (17, 1), (33, 1), (64, 2), (48, 16), (15, 5)])
def test_attention_head_groups(env, fmt, Hq, heads):
    _say("attention groups", fmt, Hq, heads)
    s = Setup(env, fmt, [130, 1, 48], Hq, heads, 64, 16, "f32", Hq)
    s.run()
    s.check()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("batch,n", [(1, 5000), (3, 2111), (1, 20000)])
def test_attention_long(env, fmt, batch, n):
    """Split over the length and joined."""
    _say("attention long", fmt, batch, n)
    s = Setup(env, fmt, [n] + [max(1, n // 3)] * (batch - 1), 8, 2, 128, 64, "f32", n)
    s.run()
    s.check()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("window", [1, 2, 16, 17, 100, 256, 699, 700, 5000])
def test_attention_window(env, fmt, window):
    torch, q, _ = env
    _say("attention window", fmt, window)
    s = Setup(env, fmt, LENS, 8, 2, 96, 32, "f32", window)
    s.ws = q.attn_workspace(len(LENS), 8, 2, 96, s.max_len, window)
    # what lies before the window is not looked at: neither its pages nor its rows
    table = s.table.copy()
    for b, n in enumerate(LENS):
        table[b, :max(0, n - window) // 32] = -7
    s.pages = _dev(torch, table)
    s.run(window=window)
    s.check(window=window)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("softcap", [0.5, 30.0])
def test_attention_softcap(env, fmt, softcap):
    _say("attention softcap", fmt, softcap)
    s = Setup(env, fmt, [200, 31], 4, 2, 128, 64, "f32", 77, sigma_q=6.0)
    s.run(softcap=softcap, scale=0.3)
    s.check(softcap=softcap, scale=0.3)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("extra", [0, 13])
def test_attention_mask(env, fmt, extra):
    """Additive masks: -inf here and there, whole rows of -inf, the type's lowest
    value under some and under all positions, rows behind -inf that hold NaN."""
    torch, q, _ = env
    _say("attention mask", fmt, extra)
    lens = [300, 300, 65, 90, 40, 513]
    s = Setup(env, fmt, lens, 6, 3, 64, 16, "f32", 5)
    rng = np.random.default_rng(1)
    low = np.finfo(np.float32).min
    mask = rng.standard_normal((len(lens), s.max_len + extra)).astype(np.float32)
    mask[0][rng.random(mask.shape[1]) < 0.3] = -np.inf
    mask[1] = -np.inf                                # nothing is seen
    mask[2] = low                                    # the lowest value everywhere: equal weights
    mask[3][::2] = low
    mask[4] = -np.inf
    mask[4][39] = low                                # one position, at the lowest value
    mask[5][:256] = -np.inf                          # the first chunk is empty
    # NaN behind -inf
    slot = int(s.table[0, 2]) * 16
    mask[0][32:48] = -np.inf
    side = ref.side_bytes(fmt, 16, 64)
    data = s.cache.data.view(-1, 2 * 3 * side)
    data[slot // 16] = 255
    s.run(mask=_dev(torch, mask))
    s.check(mask=mask)


@pytest.mark.parametrize("fmt", FORMATS)
def test_attention_mask_nan(env, fmt):
    """NaN in a mask reaches the rows that see its position and no others; past the
    length, and before the window, the mask is not looked at."""
    torch, q, _ = env
    _say("attention mask nan", fmt)
    s = Setup(env, fmt, [100, 100, 100, 70], 4, 2, 64, 16, "f32", 6)
    mask = np.zeros((4, 100), np.float32)
    mask[0, 99] = mask[1, 40] = np.nan
    mask[3, 70:] = np.nan
    s.run(mask=_dev(torch, mask))
    assert np.isnan(_np(s.out)[:2]).all() and np.isnan(_np(s.lse)[:2]).all()
    s.check(mask=np.nan_to_num(mask), rows=[2, 3])
    s.run(mask=_dev(torch, mask), window=50)
    assert np.isnan(_np(s.out)[0]).all()
    s.check(mask=np.nan_to_num(mask), rows=[1, 2, 3], window=50)


def test_attention_infinities(env):
    """Inf and NaN in rows that are seen make the result's columns (a key's: the
    whole row) infinite or NaN, and no others."""
    torch, q, orc = env
    _say("attention inf")
    s = Setup(env, "f16", [40, 40, 40], 2, 1, 64, 16, "f32", 9)
    for b, (values, x) in enumerate([(True, np.inf), (False, np.nan), (True, np.nan)]):
        k = torch.from_numpy(s.k[b][7:8].astype(np.float32)).cuda()
        v = torch.from_numpy(s.v[b][7:8].astype(np.float32)).cuda()
        (v if values else k)[0, 0, 5] = x
        q.KV_WRITE["f16"](k, v, s.cache, torch.tensor([int(s.table[b, 0]) * 16 + 7], device="cuda"))
    s.run()
    got = _np(s.out)
    assert not np.isfinite(got[0][:, 5]).any() and np.isfinite(np.delete(got[0], 5, 1)).all()
    assert np.isnan(got[1]).all()
    assert np.isnan(got[2][:, 5]).all() and np.isfinite(np.delete(got[2], 5, 1)).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("sigma", [1e-4, 300.0])
def test_attention_value_ranges(env, fmt, sigma):
    """Values and queries far from 1: small ones keep their precision, large ones do not overflow."""
    torch, q, orc = env
    _say("attention ranges", fmt, sigma)
    s = Setup(env, fmt, [150], 4, 2, 128, 16, "f32", 21)
    rng = np.random.default_rng(2)
    v = (sigma * rng.standard_normal((150, 2, 128))).astype(np.float32)
    if sigma > 1:
        v[100:] *= 40.0                              # beyond 254 * 127 in the later tiles
    i = np.arange(150)
    slots = s.table[0][i // 16].astype(np.int64) * 16 + i % 16
    k = torch.from_numpy(s.k[0].astype(np.float32)).cuda()
    q.KV_WRITE[fmt](k, _dev(torch, v), s.cache, _dev(torch, slots))
    s.k[0] = ref.through_cache(s.k[0].astype(np.float32), fmt, orc)
    s.v[0] = ref.through_cache(v, fmt, orc)
    assert np.isfinite(s.v[0]).all()
    for f in (1.0, 1e-6, 1e6):
        s.q, s.qf = (torch.from_numpy((s.qf * f).astype(np.float32)).cuda(), (s.qf * f).astype(np.float32).astype(float))
        s.run(scale=0.08 / f)
        o, _, reach, mag = ref.attention(s.qf[0], s.k[0], s.v[0], 0.08 / f)
        tol = bound(reach, mag, o, 150, 128, "f32")[0] - 2.0 ** -25 + 2.0 ** -25 * min(1.0, sigma)
        assert np.all(np.abs(_np(s.out)[0] - o) <= tol), f
        s.q, s.qf = torch.from_numpy((s.qf / f).astype(np.float32)).cuda(), (s.qf / f).astype(np.float32).astype(float)


@pytest.mark.parametrize("fmt", FORMATS)
def test_attention_bad_lengths_and_pages(env, fmt):
    torch, q, _ = env
    _say("attention bad lengths and pages", fmt)
    lens = [100, 50, 100, 60, 100]
    s = Setup(env, fmt, lens, 4, 2, 64, 16, "f32", 31)
    bad = np.array([100, -1, 101, 60, 100], np.int32)
    s.len = _dev(torch, bad)
    table = s.table.copy()
    table[3, 1] = s.cache.n_pages                    # under positions 16..31
    table[4, 6] = -5                                 # under positions 96..99
    s.pages = _dev(torch, table)
    s.run()
    got = _np(s.out)
    assert np.isnan(got[1:]).all()
    s.check(rows=[0])
    s.run(window=8)
    assert np.isnan(_np(s.out)[[1, 2, 4]]).all()
    s.check(rows=[0, 3], window=8)                   # the bad page is before the window


@pytest.mark.parametrize("fmt", FORMATS)
def test_attention_repeats_strides_streams(env, fmt):
    """Heads-outermost views with padding, a stream of its own, equal bits on repeats."""
    torch, q, _ = env
    _say("attention strides", fmt)
    s = Setup(env, fmt, [900, 33, 0, 4000], 8, 4, 128, 32, "bf16", 41)
    s.run()
    first, lse = s.out.clone(), s.lse.clone()
    for _ in range(3):
        s.out.fill_(float("nan"))
        s.run()
        assert torch.equal(s.out, first) and torch.equal(s.lse, lse)
    big = torch.zeros(8, 4, 160, dtype=torch.bfloat16, device="cuda")
    s.q = big.permute(1, 0, 2)[..., 16:144].copy_(s.q)
    out = torch.full((8, 4, 136), 3.0, dtype=torch.bfloat16, device="cuda")
    s.out = out.permute(1, 0, 2)[..., :128]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    s.run(stream=stream)
    torch.cuda.current_stream().wait_stream(stream)
    assert torch.equal(s.out.contiguous(), first)
    assert bool((out[..., 128:] == 3.0).all())


def test_workspace_serves_other_sizes(env):
    """One workspace, calls of different batches, lengths and splits in turn: each
    gives the bits it gives on a workspace of its own."""
    torch, q, _ = env
    _say("workspace reuse")
    setups = [Setup(env, "q8_0", lens, 8, 2, 64, 16, "f32", i) for i, lens in enumerate(
        [[900] * 3, [3000], [17, 2000] * 20, [5000, 100], [300] * 40, [1500] * 7])]
    own = []
    for s in setups:
        s.run()
        own.append((s.out.clone(), s.lse.clone()))
        s.check()
    shared = q.attn_workspace(40, 8, 2, 64, 5000)
    for _ in range(2):
        for s, (out, lse) in zip(setups, own):
            assert q.qmm_attn_decode_workspace(len(s.lens), 8, 2, 64, s.max_len) <= shared.numel()
            s.ws = shared
            s.out.fill_(float("nan"))
            s.run()
            assert torch.equal(s.out, out) and torch.equal(s.lse, lse)


@pytest.mark.parametrize("fmt", FORMATS)
def test_step_in_a_graph(env, fmt):
    """A decode step (rotate, write, attend) captured once, replayed at growing
    lengths with the program's own work between, against the eager result."""
    torch, q, orc = env
    _say("graph", fmt)
    Hq, heads, dim, page, most = 8, 2, 64, 16, 64
    cache = _pool(torch, q, fmt, 6, page, heads, dim)
    plan = q.RopePlan(_dev(torch, _freqs(dim)))
    qkv = torch.zeros(1, Hq + 2 * heads, dim, device="cuda")
    qo, out = torch.zeros(1, Hq, dim, device="cuda"), torch.zeros(1, Hq, dim, device="cuda")
    pages = torch.tensor([[4, 1, 5, 0]], dtype=torch.int32, device="cuda")
    slot, pos = torch.zeros(1, dtype=torch.int64, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = q.attn_workspace(1, Hq, heads, dim, most)

    def step():
        q.ROPE_KV_WRITE[fmt](qkv[:, :Hq], qo, qkv[:, Hq:Hq + heads], qkv[:, Hq + heads:], cache, slot, pos, plan)
        q.ATTN_DECODE[fmt](qo, out, cache, pages, lens, most, ws)

    def at(n):
        qkv.copy_(torch.from_numpy(np.random.default_rng(n).standard_normal(qkv.shape).astype(np.float32)))
        slot.fill_(int([4, 1, 5, 0][n // page]) * page + n % page)
        pos.fill_(n)
        lens.fill_(n + 1)
    eager = []
    for n in range(40):
        at(n)
        step()
        eager.append(out.clone())
    torch.cuda.synchronize()
    cache.data.fill_(255)
    at(0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in range(40):
        at(n)
        out.fill_(float("nan"))
        graph.replay()
        junk = torch.randn(1000, device="cuda").sum()
        torch.cuda.synchronize()
        assert torch.equal(out, eager[n]), n
        assert math.isfinite(float(junk))


def test_offsets_past_32_bits(env):
    """A cache of over 4 GiB: its last pages are written, read and attended to."""
    torch, q, orc = env
    _say("far pages")
    heads, dim, page = 32, 256, 256
    size = q.kv_page_bytes("f16", page, heads, dim)
    n_pages = (5 << 30) // size
    cache = q.KVCache.empty("f16", n_pages, page, heads, dim)
    n = 300
    rng = np.random.default_rng(4)
    k, kf = _rows(torch, rng, (n, heads, dim), "f32")
    v, vf = _rows(torch, rng, (n, heads, dim), "f32")
    table = np.array([[n_pages - 1, n_pages - 3]], np.int32)
    i = np.arange(n)
    slots = _dev(torch, table[0][i // page].astype(np.int64) * page + i % page)
    q.qmm_kv_write_f16(k, v, cache, slots)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    q.qmm_kv_read_f16(cache, slots, ko, vo)
    assert np.array_equal(_np(ko), ref.through_cache(kf, "f16", orc))
    assert np.array_equal(_np(vo), ref.through_cache(vf, "f16", orc))
    qq, qf = _rows(torch, rng, (1, heads, dim), "f32")
    out = torch.empty_like(qq)
    q.qmm_attn_decode_f16(qq, out, cache, _dev(torch, table), torch.tensor([n], dtype=torch.int32, device="cuda"), n,
                          q.attn_workspace(1, heads, heads, dim, n))
    o, _, reach, mag = ref.attention(qf[0].astype(float), ref.through_cache(kf, "f16", orc),
                                     ref.through_cache(vf, "f16", orc), dim ** -0.5)
    assert np.all(np.abs(_np(out)[0] - o) <= bound(reach, mag, o, n, dim, "f32")[0])


def test_binding_refusals(env):
    torch, q, _ = env
    _say("binding refusals")
    s = Setup(env, "q8_0", [40], 4, 2, 64, 16, "f32", 1)
    with pytest.raises(ValueError):
        q.qmm_attn_decode_q4_0(s.q, s.out, s.cache, s.pages, s.len, 40, s.ws)              # another format
    with pytest.raises(ValueError):
        q.qmm_attn_decode_q8_0(s.q, s.out.half(), s.cache, s.pages, s.len, 40, s.ws)       # another type
    with pytest.raises(ValueError):
        q.qmm_attn_decode_q8_0(s.q, s.out, s.cache, s.pages.long(), s.len, 40, s.ws)
    with pytest.raises(ValueError):
        q.qmm_attn_decode_q8_0(s.q, s.out, s.cache, s.pages, s.len.cpu(), 40, s.ws)
    with pytest.raises(q.QmmError) as e:
        q.qmm_attn_decode_q8_0(s.q, s.out, s.cache, s.pages, s.len, 40, s.ws[:64])
    assert e.value.code == "QMM_E_SHAPE"
    with pytest.raises(q.QmmError):
        q.qmm_attn_decode_q8_0(s.q, s.out, s.cache, s.pages, s.len, s.width * 16 + 1, s.ws)
    with pytest.raises(ValueError):
        q.qmm_kv_write_q8_0(s.q, s.q, s.cache, torch.zeros(1, dtype=torch.int64, device="cuda"))   # 4 heads, not 2
    with pytest.raises(ValueError):
        q.qmm_kv_read_q8_0(s.cache, torch.zeros(1, dtype=torch.int64, device="cuda"), None, None)


@pytest.mark.parametrize("cache", FORMATS)
@pytest.mark.parametrize("weights", ["q4_0", "q8_0", "q4_k"])
def test_attention_block_example(env, cache, weights, monkeypatch, capsys):
    """The example runs matvec, rotation, cache and attention together and checks itself."""
    import importlib.util
    import os
    import sys
    _say("example", cache, weights)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location("attention_decode", os.path.join(root, "examples",
                                                                                   "attention_decode.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    monkeypatch.setattr(sys, "argv", ["attention_decode", "--tokens", "9", "--prompt", "39", "--cache", cache,
                                      "--weights", weights])
    assert example.main() == 0
    assert "us a step" in capsys.readouterr().out
