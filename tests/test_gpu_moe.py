"""The mixture-of-experts operators on an MI355X against plain 64-bit forms."""
import math

import numpy as np
import pytest

import moe_ref as ref

pytestmark = pytest.mark.gpu

FORMATS = ("q4_0", "q8_0", "q4_1", "q5_0", "q5_1", "q2_k", "q4_k", "q6_k")
DTYPES = ("f32", "f16", "bf16")


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
    return t.detach().float().cpu().numpy()


def _round(torch, x, dtype):
    """f32 values of f32 values rounded to a row type."""
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(_t(torch, dtype)).float().numpy()


def _rows(torch, rng, shape, dtype, sigma=1.0, pad=0):
    """A GPU tensor of rows, `pad` values apart, and its values in f32."""
    x = torch.from_numpy((sigma * rng.standard_normal((shape[0], shape[1] + pad))).astype(np.float32))
    x = x.to(_t(torch, dtype)).to("cuda")[:, :shape[1]]
    return x, _np(x)


# ---------------------------------------------------------------------------
# Norm
# ---------------------------------------------------------------------------
def _norm_check(torch, q, orc, fmt, dtype, x, xf, r, rf, w, eps, offset, got_sum, got_y, xq):
    """s is one f32 sum rounded to the type; y is the exact value rounded once to f32 (f64 leaves 1e-12 at most), then
    to the type; the blocks are the quantizer's of f32 y."""
    s = xf if rf is None else _round(torch, xf + rf, dtype)
    if got_sum is not None:
        assert np.array_equal(_np(got_sum), s)
    want = ref.norm(s, None if w is None else w.cpu().numpy(), eps, offset)
    step = 2.0 ** -24 + (ref.STEP[dtype] if dtype != "f32" else 0)
    if got_y is not None:
        tiny = 2.0 ** -25 if dtype == "f16" else 2.0 ** -149
        assert np.all(np.abs(_np(got_y).astype(np.float64) - want) <= (step + 1e-12) * np.abs(want) + tiny)
    y32 = _np(got_y) if got_y is not None and dtype == "f32" else want.astype(np.float32)
    blocks = (orc.quantize_q8_0 if fmt == "q8_0" else orc.quantize_q8_k)(y32)
    assert np.array_equal(xq.cpu().numpy().reshape(-1), np.asarray(blocks).reshape(-1))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", ["q8_0", "q8_k"])
@pytest.mark.parametrize("T,blocks", [(1, 1), (1, 16), (3, 5), (7, 13), (130, 2), (5, 17), (2, 65), (3, 129), (1, 513)])
def test_norm(env, fmt, dtype, T, blocks):
    torch, q, orc = env
    K = blocks * ref.VALUES[fmt] if fmt == "q8_0" or blocks < 100 else 256 * (blocks // 8)
    _say("norm", fmt, dtype, T, K)
    rng = np.random.default_rng(T * 1000 + K)
    x, xf = _rows(torch, rng, (T, K), dtype, pad=4)
    r, rf = _rows(torch, rng, (T, K), dtype, sigma=3.0, pad=8)
    w = _dev(torch, (1 + 0.2 * rng.standard_normal(K)).astype(np.float32))
    xq = torch.full((T, q.row_bytes(fmt, K)), 255, dtype=torch.uint8, device="cuda")
    s, y = torch.empty(T, K + 4, dtype=x.dtype, device="cuda")[:, :K], torch.empty(T, K, dtype=x.dtype, device="cuda")
    q.RMS_NORM[fmt](x, w, xq, residual=r, sum=s, y=y, eps=1e-5)
    _norm_check(torch, q, orc, fmt, dtype, x, xf, r, rf, w, 1e-5, 0.0, s, y, xq)
    # alone; ones as the weight; an offset
    q.RMS_NORM[fmt](x, None, xq)
    _norm_check(torch, q, orc, fmt, dtype, x, xf, None, None, None, 1e-6, 0.0, None, None, xq)
    q.RMS_NORM[fmt](x, w, xq, residual=r, weight_offset=1.0)
    _norm_check(torch, q, orc, fmt, dtype, x, xf, r, rf, w, 1e-6, 1.0, None, None, xq)
    # in place: the stream is updated, the rows are normed
    q.RMS_NORM[fmt](x, w, xq, residual=r, sum=r, y=x)
    _norm_check(torch, q, orc, fmt, dtype, x, xf, r, rf, w, 1e-6, 0.0, r, x, xq)


@pytest.mark.parametrize("fmt", ["q8_0", "q8_k"])
def test_norm_of_any_size_of_value(env, fmt):
    """Squares far beyond f32, rows of zeros, and a NaN or an infinity, which shows in its own row alone."""
    torch, q, orc = env
    _say("norm sizes", fmt)
    rng, K = np.random.default_rng(3), 512
    base = rng.standard_normal((6, K)).astype(np.float32)
    base[0] *= 1e25
    base[1] *= 1e-25
    base[2] = 0
    base[3, 300] = math.nan
    base[4, 7] = math.inf
    x = _dev(torch, base)
    xq = torch.zeros(6, q.row_bytes(fmt, K), dtype=torch.uint8, device="cuda")
    y = torch.empty_like(x)
    q.RMS_NORM[fmt](x, None, xq, y=y, eps=0.0)
    want = ref.norm(base[[0, 1, 5]], None, 0.0)
    got = _np(y)
    assert np.all(np.abs(got[[0, 1, 5]] - want) <= (2.0 ** -24 + 1e-12) * np.abs(want))
    assert np.isnan(got[2]).all()                                      # 0 / 0 with eps 0
    q.RMS_NORM[fmt](x, None, xq, y=y, eps=1e-6)
    values, _ = ref.decoded(xq.cpu().numpy(), fmt)
    assert np.all(values[2] == 0) and np.isnan(values[3]).all()
    assert np.isfinite(values[[0, 1, 2, 5]]).all()
    assert np.isnan(values[4].reshape(-1, ref.VALUES[fmt])[0]).all()    # inf / inf; finite / inf = 0 in other blocks
    assert np.all(values[4].reshape(-1, ref.VALUES[fmt])[1:] == 0)


# ---------------------------------------------------------------------------
# Gated activation
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("fmt,rows,F", [("q8_0", 1, 32), ("q8_0", 3, 96), ("q8_0", 33, 800), ("q8_0", 257, 64),
                                        ("q8_k", 1, 256), ("q8_k", 5, 768), ("q8_k", 40, 1280)])
def test_glu(env, fmt, act, dtype, rows, F):
    """Values y = a u with a relative error of at most r: the activation's 16 f32 steps at most, times the
    amplification of its exponent's error (|z| < 64 + 32 for the inputs here), and one product.  A value q d of a
    block then lies within d/2 of y, plus the scale's own rounding (f16: 127 d 2^-11) and 127 d (2 r)."""
    torch, q, orc = env
    _say("glu", fmt, act, dtype, rows, F)
    rng = np.random.default_rng(rows * 7 + F)
    both, bf = _rows(torch, rng, (rows, 2 * F), dtype, sigma=2.0)
    gate, up = both[:, :F], both[:, F:]
    xq = torch.full((rows, q.row_bytes(fmt, F)), 255, dtype=torch.uint8, device="cuda")
    q.GLU[fmt](gate, up, xq, act=act)
    want = ref.activation(bf[:, :F], act) * bf[:, F:].astype(np.float64)
    values, d = ref.decoded(xq.cpu().numpy(), fmt)
    r = 16 * 96 * 2.0 ** -24
    amax = np.abs(want.reshape(rows, -1, ref.VALUES[fmt])).max(-1)
    step = 2.0 ** -11 if fmt == "q8_0" else 2.0 ** -23
    assert np.all(np.abs(d - amax / 127) <= (step + 2 * r) * amax / 127 + 2.0 ** -25)
    off = np.abs(values - want).reshape(rows, -1, ref.VALUES[fmt])
    assert np.all(off <= (amax / 127)[..., None] * (0.5 + 127 * (step + 2 * r)) + 127 * 2.0 ** -25 * (fmt == "q8_0"))
    if fmt == "q8_k":                                                  # the groups' sums are those of the codes
        b = xq.cpu().numpy().reshape(-1, 292)
        codes = np.ascontiguousarray(b[:, 4:260]).view(np.int8).astype(np.int32).reshape(-1, 16, 16).sum(-1)
        assert np.array_equal(np.ascontiguousarray(b[:, 260:]).view(np.int16), codes)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_glu_limits(env, act):
    """Far gates: the activation is 0 or the gate itself, not a NaN; NaN and infinity show in their block."""
    torch, q, orc = env
    _say("glu limits", act)
    g = np.ones((1, 160), np.float32)
    g[0, :32] = [-1e30, 1e30] * 16
    g[0, 32:64] = [-200, -30] * 16
    g[0, 70] = math.nan
    g[0, 100] = math.inf
    gate, up = _dev(torch, g), torch.ones(1, 160, device="cuda")
    up[0, :32] = 1e-30
    xq = torch.zeros(1, q.row_bytes("q8_0", 160), dtype=torch.uint8, device="cuda")
    q.GLU["q8_0"](gate, up, xq, act=act)
    v = ref.decoded(xq.cpu().numpy(), "q8_0")[0].reshape(5, 32)
    assert np.all(v[0, ::2] == 0) and np.all(np.abs(v[0, 1::2] - 1) <= 0.01)
    assert np.all(np.abs(v[1]) <= 1e-6)
    assert np.isnan(v[2]).all() and np.isnan(v[3]).all() and np.isfinite(v[4]).all()


# ---------------------------------------------------------------------------
# Routing
# ---------------------------------------------------------------------------
def _routed(env, logits, top, **kw):
    torch, q, _ = env
    T = logits.shape[0]
    ids = torch.full((T, top), 77, dtype=torch.int32, device="cuda")
    w = torch.full((T, top), math.nan, device="cuda")
    bias = kw.pop("bias", None)
    kept = kw.pop("kept", 1)
    q.qmm_route(logits, ids, w, bias=None if bias is None else _dev(torch, bias), groups_kept=kept, **kw)
    return ids.cpu().numpy(), w.double().cpu().numpy()


def _route_check(env, logits, lf, top, **kw):
    """ids are those of the definition; weights its f64 values (within 1e-9) rounded once."""
    ids, w = _routed(env, logits, top, **dict(kw))
    want, ww = ref.route(lf, top, **kw)
    assert np.array_equal(ids, want)
    assert np.array_equal(np.isnan(w), np.isnan(ww))
    ok = ~np.isnan(ww)
    assert np.all(np.abs(w - ww)[ok] <= ((2.0 ** -24 + 1e-9) * np.abs(ww) + 2.0 ** -149)[ok])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,top", [(1, 1, 1), (1, 8, 2), (5, 60, 4), (3, 64, 64), (9, 65, 6), (6, 128, 8), (2, 200, 16),
                                     (3, 257, 8), (2, 512, 20)])
def test_route(env, dtype, score, T, E, top):
    torch, q, _ = env
    _say("route", dtype, score, T, E, top)
    rng = np.random.default_rng(T * 100 + E)
    logits, lf = _rows(torch, rng, (T, E), dtype, sigma=2.0, pad=3)
    for renorm in (True, False):
        _route_check(env, logits, lf, top, score=score, renorm=renorm)
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32)
    _route_check(env, logits, lf, top, score=score, bias=bias, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("E,groups,kept,top", [(8, 2, 1, 2), (8, 8, 3, 3), (96, 6, 2, 8), (256, 8, 4, 8), (512, 64, 9, 16),
                                               (15, 3, 3, 4), (130, 2, 1, 7)])
def test_route_groups(env, score, group_top, E, groups, kept, top):
    torch, q, _ = env
    _say("route groups", score, group_top, E, groups, kept, top)
    rng = np.random.default_rng(E + groups)
    logits, lf = _rows(torch, rng, (7, E), "f32", sigma=2.0)
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32)
    for b in (None, bias):
        _route_check(env, logits, lf, top, score=score, bias=b, groups=groups, kept=kept, group_top=group_top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_hidden_experts(env, score):
    """Logits of -inf: few experts left, none left, whole groups hidden; masks of the type's lowest value are numbers."""
    torch, q, _ = env
    _say("route hidden", score)
    rng = np.random.default_rng(8)
    lf = rng.standard_normal((6, 32)).astype(np.float32)
    lf[0, 3:] = -math.inf
    lf[1] = -math.inf
    lf[2, 8:24] = -math.inf
    lf[3, 5:] = np.finfo(np.float32).min
    lf[4, 1:] = -math.inf
    logits = _dev(torch, lf)
    for kw in (dict(), dict(renorm=False), dict(groups=4, kept=2, group_top=2),
               dict(bias=np.linspace(0, 0.2, 32).astype(np.float32))):
        _route_check(env, logits, lf, 6, score=score, **kw)
    bias = np.zeros(32, np.float32)
    bias[::2] = -math.inf
    _route_check(env, logits, lf, 6, score=score, bias=bias)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_ties_and_far_logits(env, score):
    torch, q, _ = env
    _say("route ties", score)
    lf = np.zeros((5, 100), np.float32)
    lf[0, 40:] = -0.0
    lf[1, [70, 3, 66]] = 1.0
    lf[2] = np.linspace(-5000, -4000, 100)            # sigmoids that all round to 0
    lf[3] = np.linspace(-1e30, 1e30, 100)
    lf[4, 1::2] = 2.0 ** -24                          # apart by less than f32 scores are
    logits = _dev(torch, lf)
    _route_check(env, logits, lf, 8, score=score)
    _route_check(env, logits[:2], lf[:2], 8, score=score, groups=4, kept=2, group_top=2)
    _route_check(env, logits[:2], lf[:2], 8, score=score, bias=np.zeros(100, np.float32))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_nan_shows(env, score):
    torch, q, _ = env
    _say("route nan", score)
    lf = np.random.default_rng(2).standard_normal((2, 64)).astype(np.float32)
    lf[0, 50] = math.nan
    ids, w = _routed(env, _dev(torch, lf), 4, score=score)
    assert ids[0, 0] == 50 and np.isnan(w[0]).all()
    assert np.all((ids >= 0) & (ids < 64)) and np.isfinite(w[1]).all()


# ---------------------------------------------------------------------------
# Experts' products
# ---------------------------------------------------------------------------
def _matrices(torch, orc, q, fmt, E, N, K, rng, pad=None):
    """E matrices on the GPU [E][N][row bytes], `pad` rows apart (by default up to eight rows: whole 16 bytes), and
    their bytes."""
    pad = -N % 8 if pad is None else pad
    rb = q.row_bytes(fmt, K)
    packed = [np.asarray(orc.quantize_w(fmt, (rng.standard_normal((N, K)) * K ** -0.5).astype(np.float32))).reshape(N, rb)
              for _ in range(E)]
    room = np.full((E, N + pad, rb), 255, np.uint8)
    room[:, :N] = np.stack(packed)
    return _dev(torch, room)[:, :N], packed


def _ids(rng, T, top, E, skew=False):
    like = rng.standard_normal((T, E)) + (2.0 * rng.standard_normal(E) if skew else 0)
    return np.argsort(-like, 1)[:, :top].astype(np.int32)


def _product(env, fmt, T, top, E, N, K, per_pair, ids, pad=None, seed=0):
    torch, q, orc = env
    rng = np.random.default_rng(seed + T + N + K)
    w, packed = _matrices(torch, orc, q, fmt, E, N, K, rng, pad)
    act = q.ACT_FORMAT[fmt]
    rows = T * top if per_pair else T
    xq = np.asarray(orc.quantize_x(fmt, rng.standard_normal((rows, K)).astype(np.float32))).reshape(rows, -1)
    y = torch.full((T, top, N), math.nan, device="cuda")
    plan = q.experts_plan(T, top, E)
    ids_d = _dev(torch, ids)
    q.qmm_experts_plan(ids_d, E, plan)
    q.EXPERTS_MATMUL[fmt](w, _dev(torch, xq), ids_d, plan, y)
    want, mag = ref.experts(orc, fmt, packed, xq, ids, N, K, per_pair)
    # integer block sums are exact; two terms a block, each of three f32 steps, and the sum over the blocks
    steps = 2 * (K // q.BLOCK_VALUES[act]) + 8
    bound = steps * 2.0 ** -24 * mag + 2.0 ** -149
    got = y.double().cpu().numpy()
    assert not np.isnan(got).any()
    assert np.all(np.abs(got - want) <= bound), float(np.max(np.abs(got - want) / bound))
    return y


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,top,E,N,blocks,per_pair", [
    (1, 1, 1, 8, 2, False), (1, 4, 8, 40, 4, False), (1, 8, 16, 100, 3, True), (3, 2, 4, 64, 24, False),
    (8, 8, 8, 72, 8, True), (16, 2, 4, 136, 7, False), (5, 3, 64, 24, 33, True), (2, 2, 4, 16, 130, False)])
def test_experts_few(env, fmt, T, top, E, N, blocks, per_pair):
    """Up to 64 pairs: no plan."""
    torch, q, orc = env
    K = blocks * q.BLOCK_VALUES[fmt] if fmt not in ("q2_k", "q4_k", "q6_k") else 256 * max(1, blocks // 3)
    _say("experts few", fmt, T, top, E, N, K, per_pair)
    _product(env, fmt, T, top, E, N, K, per_pair, _ids(np.random.default_rng(T), T, top, E))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,top,E,N,blocks,per_pair", [
    (33, 2, 16, 40, 4, False), (20, 6, 40, 136, 5, True), (65, 1, 12, 8, 1, False),      # a few rows each
    (40, 4, 8, 130, 6, False), (200, 2, 8, 264, 3, True), (101, 3, 5, 12, 9, False),      # tiles of 32
    (300, 4, 8, 136, 4, False), (257, 1, 3, 300, 5, True), (1030, 2, 2, 20, 2, False)])   # tiles of 128
def test_experts_planned(env, fmt, T, top, E, N, blocks, per_pair):
    torch, q, orc = env
    K = blocks * q.BLOCK_VALUES[fmt] if fmt not in ("q2_k", "q4_k", "q6_k") else 256 * max(1, blocks // 2)
    _say("experts planned", fmt, T, top, E, N, K, per_pair)
    _product(env, fmt, T, top, E, N, K, per_pair, _ids(np.random.default_rng(T), T, top, E, skew=True))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,top,E,N,K,per_pair", [
    (40, 2, 64, 768, 512, False), (200, 2, 16, 1800, 256, True),         # many workgroups: 16 and 32 rows a tile
    (20, 4, 16, 896, 1280, False), (100, 2, 8, 1400, 768, True),         # a few hundred
    (2100, 2, 8, 136, 512, False), (1030, 4, 5, 300, 256, True)])        # 128 rows a tile
def test_experts_large(env, fmt, T, top, E, N, K, per_pair):
    torch, q, orc = env
    _say("experts large", fmt, T, top, E, N, K, per_pair)
    _product(env, fmt, T, top, E, N, K, per_pair, _ids(np.random.default_rng(T), T, top, E, skew=T < 1000))


@pytest.mark.parametrize("fmt", ["q4_0", "q8_0", "q4_1", "q5_0", "q5_1"])
def test_experts_128_rows_of_odd_blocks(env, fmt):
    _say("experts odd blocks", fmt)
    _product(env, fmt, 2100, 2, 8, 24, 288, False, _ids(np.random.default_rng(3), 2100, 2, 8))


@pytest.mark.parametrize("fmt", ["q4_0", "q8_0", "q4_1", "q5_0", "q5_1"])
@pytest.mark.parametrize("T,top,E,N,per_pair", [
    (40, 2, 64, 776, False), (20, 4, 16, 904, True), (33, 2, 16, 40, False),              # tiles of 16 rows, by workgroups
    (200, 2, 16, 1800, True), (100, 2, 8, 1400, False), (300, 4, 16, 56, True), (5, 3, 6, 72, False),       # of 32
    (300, 3, 20, 40, True), (90, 1, 2, 200, False)])                                      # of 32, few workgroups
@pytest.mark.parametrize("blocks", [9, 10, 12, 15, 19, 31])
def test_experts_part_of_a_stage(env, fmt, T, top, E, N, per_pair, blocks):
    """Rows that are no whole number of 256 values: of an odd number of blocks, of an even one."""
    _say("experts part", fmt, T, top, E, N, blocks, per_pair)
    _product(env, fmt, T, top, E, N, 32 * blocks, per_pair, _ids(np.random.default_rng(T + blocks), T, top, E, skew=True))


@pytest.mark.parametrize("fmt", ["q2_k", "q4_k", "q6_k"])
@pytest.mark.parametrize("T", [30, 700, 1700])
def test_experts_of_one_superblock(env, fmt, T):
    _say("experts of one super-block", fmt, T)
    _product(env, fmt, T, 3, 9, 136, 256, T == 700, _ids(np.random.default_rng(T), T, 3, 9, skew=True))


@pytest.mark.parametrize("fmt", FORMATS)
def test_experts_one_block(env, fmt):
    """K of one block, with a plan."""
    _say("experts of one block", fmt)
    _product(env, fmt, 260, 2, 5, 70, 256 if fmt.endswith("_k") else 32, True, _ids(np.random.default_rng(8), 260, 2, 5))


@pytest.mark.parametrize("fmt", ["q4_0", "q8_0", "q4_1", "q5_0", "q5_1"])
@pytest.mark.parametrize("blocks", [9, 13, 14])
def test_experts_128_rows_of_part_stages(env, fmt, blocks):
    _say("experts part of a stage, 128 rows", fmt, blocks)
    _product(env, fmt, 2090, 2, 7, 136, 32 * blocks, blocks == 13, _ids(np.random.default_rng(3), 2090, 2, 7, skew=True))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,top,E,N,K,per_pair", [(2200, 2, 7, 72, 768, False), (2300, 2, 5, 300, 512, True),
                                                  (4200, 1, 1, 1400, 256, False), (2500, 2, 4, 2600, 256, True)])
def test_experts_tiles_of_128_in_parts(env, fmt, T, top, E, N, K, per_pair):
    """Few columns, and more, at many rows an expert."""
    torch, q, orc = env
    _say("experts parts", fmt, T, top, E, N, K, per_pair)
    _product(env, fmt, T, top, E, N, K, per_pair, _ids(np.random.default_rng(T), T, top, E, skew=True))


@pytest.mark.parametrize("T", [9, 40, 300, 1500, 2500])
@pytest.mark.parametrize("fmt", ["q4_0", "q4_k"])
def test_experts_unusual_ids(env, fmt, T):
    """Ids outside the experts give zeros; one expert for all; the same expert twice for a token; experts unused."""
    torch, q, orc = env
    E, top, N, K = 6, 2, 40, 256
    _say("experts ids", fmt, T)
    rng = np.random.default_rng(T)
    ids = _ids(rng, T, top, E)
    ids[::3, 1] = -1
    ids[1::4, 0] = E
    ids[-1] = np.iinfo(np.int32).max, np.iinfo(np.int32).min
    y = _product(env, fmt, T, top, E, N, K, False, ids)
    out = (ids < 0) | (ids >= E)
    assert np.all(y.cpu().numpy()[out] == 0)
    _product(env, fmt, T, top, E, N, K, True, np.full((T, top), 4, np.int32))
    _product(env, fmt, T, top, E, N, K, False, np.full((T, top), -1, np.int32))


@pytest.mark.parametrize("fmt", ["q4_0", "q5_1", "q6_k"])
def test_experts_stride_and_odd_rows(env, fmt):
    """Matrices of an odd row count, padded to whole 16 bytes, with bytes between them that nothing reads as weights."""
    torch, q, orc = env
    _say("experts stride", fmt)
    for T in (3, 70, 600):
        _product(env, fmt, T, 2, 4, 23, 256, False, _ids(np.random.default_rng(1), T, 2, 4), pad=9 if fmt != "q5_1" else 1)


@pytest.mark.parametrize("T", [4, 60, 700])
def test_experts_rows_are_independent(env, T):
    """A row's bits do not depend on the other rows' contents, and repeat."""
    torch, q, orc = env
    _say("experts independent", T)
    E, top, N, K = 4, 2, 64, 512
    rng = np.random.default_rng(T)
    ids = _ids(rng, T, top, E)
    a = _product(env, "q4_0", T, top, E, N, K, False, ids, seed=5)
    b = _product(env, "q4_0", T, top, E, N, K, False, ids, seed=5)
    assert torch.equal(a, b)


# ---------------------------------------------------------------------------
# Weighted sum
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,top,N", [(1, 1, 4), (1, 8, 2048), (3, 2, 7), (5, 3, 1), (17, 4, 100), (130, 8, 36), (2, 64, 12)])
def test_combine(env, dtype, T, top, N):
    """f32: a product and a sum a slot (one fused step each), the residual's sum, one rounding to the type."""
    torch, q, _ = env
    _say("combine", dtype, T, top, N)
    rng = np.random.default_rng(T + N)
    y = rng.standard_normal((T, top, N)).astype(np.float32)
    w = rng.random((T, top)).astype(np.float32)
    r, rf = _rows(torch, rng, (T, N), dtype, pad=4)
    for res in (None, r):
        out = torch.full((T, N + 8), math.nan, dtype=r.dtype, device="cuda")[:, :N]
        q.qmm_experts_combine(_dev(torch, y), _dev(torch, w), out, residual=res)
        terms = w.astype(np.float64)[..., None] * y
        want = terms.sum(1) + (0 if res is None else rf)
        mag = np.abs(terms).sum(1) + (0 if res is None else np.abs(rf))
        bound = (top + 1) * 2.0 ** -24 * mag + (0 if dtype == "f32" else ref.STEP[dtype] * np.abs(want) * 1.01 + 2.0 ** -25)
        assert np.all(np.abs(_np(out) - want) <= bound)
    q.qmm_experts_combine(_dev(torch, y).view(T * top, N), _dev(torch, w), r, residual=r)          # onto the stream
    assert np.array_equal(_np(r), _np(out))


# ---------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------
def _block(torch, q, fmt, T, dim=512, F=256, E=8, top=2, seed=0, orc=None):
    """A feed-forward block's buffers and one pass through it."""
    rng = np.random.default_rng(seed)
    act = q.ACT_FORMAT[fmt]
    gate_up, gu = _matrices(torch, orc, q, fmt, E, 2 * F, dim, rng)
    down, dn = _matrices(torch, orc, q, fmt, E, dim, F, rng)
    b = dict(x=torch.zeros(T, dim, device="cuda"), stream=torch.zeros(T, dim, device="cuda"),
             norm=_dev(torch, (1 + 0.1 * rng.standard_normal(dim)).astype(np.float32)),
             router=_dev(torch, (rng.standard_normal((dim, E)) * dim ** -0.5).astype(np.float32)),
             y=torch.empty(T, dim, device="cuda"), logits=torch.empty(T, E, device="cuda"),
             xq=torch.empty(T, q.row_bytes(act, dim), dtype=torch.uint8, device="cuda"),
             ids=torch.empty(T, top, dtype=torch.int32, device="cuda"), w=torch.empty(T, top, device="cuda"),
             plan=q.experts_plan(T, top, E), h=torch.empty(T, top, 2 * F, device="cuda"),
             hq=torch.empty(T * top, q.row_bytes(act, F), dtype=torch.uint8, device="cuda"),
             z=torch.empty(T, top, dim, device="cuda"), out=torch.empty(T, dim, device="cuda"))

    def step():
        q.RMS_NORM[act](b["x"], b["norm"], b["xq"], residual=b["stream"], sum=b["stream"], y=b["y"])
        torch.mm(b["y"], b["router"], out=b["logits"])
        q.qmm_route(b["logits"], b["ids"], b["w"])
        q.qmm_experts_plan(b["ids"], E, b["plan"])
        q.EXPERTS_MATMUL[fmt](gate_up, b["xq"], b["ids"], b["plan"], b["h"])
        h = b["h"].view(T * top, 2 * F)
        q.GLU[act](h[:, :F], h[:, F:], b["hq"])
        q.EXPERTS_MATMUL[fmt](down, b["hq"], b["ids"], b["plan"], b["z"])
        q.qmm_experts_combine(b["z"], b["w"], b["out"], residual=b["stream"])
    return b, step, gu, dn


@pytest.mark.parametrize("fmt", ["q4_0", "q4_k"])
@pytest.mark.parametrize("T", [1, 30, 300])
def test_block(env, fmt, T):
    """All of them in a row, each against its definition on what the one before left."""
    torch, q, orc = env
    _say("block", fmt, T)
    dim, F, E, top = 512, 256, 8, 2
    b, step, gu, dn = _block(torch, q, fmt, T, dim, F, E, top, orc=orc)
    rng = np.random.default_rng(T)
    x, s0 = rng.standard_normal((T, dim)).astype(np.float32), rng.standard_normal((T, dim)).astype(np.float32)
    b["x"].copy_(torch.from_numpy(x))
    b["stream"].copy_(torch.from_numpy(s0))
    step()
    torch.cuda.synchronize()
    s = x + s0
    assert np.array_equal(_np(b["stream"]), s)
    ids, w = ref.route(_np(b["logits"]), top)
    assert np.array_equal(b["ids"].cpu().numpy(), ids)
    nb = {"q4_0": 32, "q4_k": 256}[fmt]
    h, hm = ref.experts(orc, fmt, gu, b["xq"].cpu().numpy(), ids, 2 * F, dim, False)
    assert np.all(np.abs(_np(b["h"]) - h) <= (2 * dim // nb + 8) * 2.0 ** -24 * hm)
    z, zm = ref.experts(orc, fmt, dn, b["hq"].cpu().numpy(), ids, dim, F, True)
    assert np.all(np.abs(_np(b["z"]) - z) <= (2 * F // nb + 8) * 2.0 ** -24 * zm)
    terms = _np(b["w"]).astype(np.float64)[..., None] * _np(b["z"])
    mag = np.abs(terms).sum(1) + np.abs(s)
    assert np.all(np.abs(_np(b["out"]) - (terms.sum(1) + s)) <= (top + 1) * 2.0 ** -24 * mag)


@pytest.mark.parametrize("T", [1, 30, 300])
def test_block_in_a_graph(env, T):
    """Captured once on its own stream, replayed with other work between, against the eager results."""
    torch, q, orc = env
    _say("graph", T)
    b, step, _, _ = _block(torch, q, "q4_0", T, orc=orc)

    def at(n):
        rng = np.random.default_rng(n)
        b["x"].copy_(torch.from_numpy(rng.standard_normal(b["x"].shape).astype(np.float32)))
        b["stream"].copy_(torch.from_numpy(rng.standard_normal(b["x"].shape).astype(np.float32)))
    eager = []
    for n in range(6):
        at(n)
        step()
        eager.append([b[k].clone() for k in ("out", "ids", "xq", "hq")])
    graph = torch.cuda.CUDAGraph()
    at(0)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for n in range(6):
        at(n)
        for k in ("out", "h", "z"):
            b[k].fill_(math.nan)
        b["plan"].fill_(85)
        graph.replay()
        junk = torch.randn(1000, device="cuda").sum()
        torch.cuda.synchronize()
        for k, v in zip(("out", "ids", "xq", "hq"), eager[n]):
            assert torch.equal(b[k], v), (n, k)
        assert math.isfinite(float(junk))


def test_on_another_stream(env):
    torch, q, orc = env
    _say("stream")
    b, step, _, _ = _block(torch, q, "q8_0", 20, orc=orc)
    b["x"].normal_()
    b["stream"].normal_()
    keep = b["stream"].clone()
    step()
    want = b["out"].clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b["stream"].copy_(keep)
        b["out"].fill_(math.nan)
        step()
    side.synchronize()
    assert torch.equal(b["out"], want)


# ---------------------------------------------------------------------------
# Further calls that the contracts allow
# ---------------------------------------------------------------------------
def _counted(torch, q, T, top, E, N=8, K=64):
    """Matrices whose codes are all 1 with scale e + 1 and activations of whole numbers with scale 1: every product is
    exact, (e + 1) times the sum of the row's codes, below 2^24."""
    w = np.zeros((E, N, K // 32, 34), np.uint8)
    w[..., :2] = (np.arange(E) + 1).astype(np.float16).view(np.uint8).reshape(E, 1, 1, 2)
    w[..., 2:] = 1
    codes = np.random.default_rng(T + E).integers(-127, 128, (T, K // 32, 32)).astype(np.int8)
    x = np.zeros((T, K // 32, 34), np.uint8)
    x[..., :2] = np.ones(1, np.float16).view(np.uint8)
    x[..., 2:] = codes.view(np.uint8)
    return (_dev(torch, w.reshape(E, N, -1)), _dev(torch, x.reshape(T, -1)), codes.astype(np.int64).sum((1, 2)))


@pytest.mark.parametrize("skew", ["even", "one", "few", "none"])
@pytest.mark.parametrize("E,top", [(512, 4), (65, 1), (1, 1), (3, 2)])
@pytest.mark.parametrize("T", [600, 2100, 2600, 70001])
def test_plan_of_many_pairs(env, T, E, top, skew):
    """One segment, several, 256 of them; experts of every count, and all pairs with one or without any."""
    torch, q, _ = env
    _say("plan", T, E, top, skew)
    rng = np.random.default_rng(T + E)
    ids = rng.integers(0, E, (T, top)).astype(np.int32)
    if skew == "one":
        ids[:] = E - 1
    elif skew == "few":
        ids = np.minimum(ids, rng.integers(-1, 3, (T, top))).astype(np.int32)
    elif skew == "none":
        ids[rng.random((T, top)) < 0.9] = -7
    w, x, sums = _counted(torch, q, T, top, E)
    plan = q.experts_plan(T, top, E)
    plan.fill_(0x55)
    y = torch.full((T, top, 8), math.nan, device="cuda")
    ids_d = _dev(torch, ids)
    q.qmm_experts_plan(ids_d, E, plan)
    q.qmm_experts_matmul_q8_0(w, x, ids_d, plan, y)
    want = np.where((ids >= 0) & (ids < E), (ids + 1) * sums[:, None], 0)
    assert np.array_equal(y.cpu().numpy(), np.repeat(want[..., None], 8, 2).astype(np.float32))


def test_products_of_more_tiles_than_a_launch(env):
    """K of one block and over 32768 tiles: several launches."""
    torch, q, _ = env
    T, E = 4_250_000, 2
    _say("many tiles", T)
    ids = np.random.default_rng(5).integers(-1, E, (T, 1)).astype(np.int32)
    w, x, sums = _counted(torch, q, T, 1, E, K=32)
    plan = q.experts_plan(T, 1, E)
    y = torch.full((T, 1, 8), math.nan, device="cuda")
    ids_d = _dev(torch, ids)
    q.qmm_experts_plan(ids_d, E, plan)
    q.qmm_experts_matmul_q8_0(w, x, ids_d, plan, y)
    want = ((ids[:, 0] + 1) * sums).astype(np.float32)          # -1: zero
    assert np.array_equal(y[:, 0].cpu().numpy(), np.repeat(want[:, None], 8, 1))


@pytest.mark.parametrize("fmt,K", [("q4_0", 512), ("q8_0", 288), ("q5_1", 320), ("q4_1", 96), ("q2_k", 512), ("q6_k", 768)])
@pytest.mark.parametrize("T", [1, 9, 60, 130, 700, 2300])
def test_experts_other_rows_do_not_matter(env, fmt, K, T):
    """A NaN row, and other contents, leave the bits of the rest."""
    torch, q, orc = env
    _say("other rows", fmt, T, K)
    E, top, N = 5, 2, 40
    rng = np.random.default_rng(T)
    w, _ = _matrices(torch, orc, q, fmt, E, N, K, rng)
    act = q.ACT_FORMAT[fmt]
    xq = np.asarray(orc.quantize_x(fmt, rng.standard_normal((T, K)).astype(np.float32))).reshape(T, -1)
    ids = _dev(torch, _ids(rng, T, top, E))
    plan = q.experts_plan(T, top, E)
    q.qmm_experts_plan(ids, E, plan)
    out = []
    for other in (False, True):
        x = xq.copy()
        if other:
            x[::3] = x[::3][::-1]
            x[1::7, :4] = 0xff                       # f16 and f32 NaN scales
        y = torch.full((T, top, N), 7.0, device="cuda")
        q.EXPERTS_MATMUL[fmt](w, _dev(torch, x), ids, plan, y)
        out.append(y.cpu().numpy())
    same = np.ones(T, bool)
    same[::3] = same[1::7] = False
    assert act in ("q8_0", "q8_k") and np.array_equal(out[0][same].view(np.uint32), out[1][same].view(np.uint32))
    assert np.all(np.isnan(out[1][1::7]))
    assert not np.isnan(out[0]).any()


@pytest.mark.parametrize("fmt,K", [("q4_0", 512), ("q8_0", 288), ("q5_0", 64), ("q4_1", 32), ("q4_k", 512), ("q6_k", 768)])
@pytest.mark.parametrize("T", [40, 130, 700, 2300])
def test_experts_of_another_plan(env, fmt, K, T):
    """The rows of a plan's bytes that are not of these ids stay inside y (the kernels keep them there)."""
    torch, q, orc = env
    _say("another plan", fmt, T, K)
    E, top, N = 5, 2, 40
    rng = np.random.default_rng(T)
    w, _ = _matrices(torch, orc, q, fmt, E, N, K, rng)
    xq = _dev(torch, np.asarray(orc.quantize_x(fmt, rng.standard_normal((T, K)).astype(np.float32))).reshape(T, -1))
    ids = _dev(torch, _ids(rng, T, top, E))
    plan = q.experts_plan(T, top, E)
    room = torch.full((T * top + 512, N), 7.0, device="cuda")
    y = room[256:-256]
    for fill in (0x00, 0x01, 0x7f, 0x80, 0xff):
        plan.fill_(fill)
        q.EXPERTS_MATMUL[fmt](w, xq, ids, plan, y)
        torch.cuda.synchronize()
        assert torch.all(room[:256] == 7.0) and torch.all(room[-256:] == 7.0), fill
    q.qmm_experts_plan(ids, E, plan)
    q.EXPERTS_MATMUL[fmt](w, xq, ids, plan, y)
    assert torch.isfinite(y).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("K", [96, 4096, 16416, 33024])
def test_norm_in_place(env, dtype, K):
    """sum over x, sum over the residual, y over x, y over the residual, against separate outputs; rows of stride 0."""
    torch, q, _ = env
    _say("norm in place", dtype, K)
    T = 5
    x = torch.randn(T, K, device="cuda").to(_t(torch, dtype))
    r = torch.randn(T, K, device="cuda").to(_t(torch, dtype))
    xq, s, y = (torch.empty(T, q.row_bytes("q8_0", K), dtype=torch.uint8, device="cuda"), torch.empty_like(x),
                torch.empty_like(x))
    q.qmm_rms_norm_q8_0(x, None, xq, residual=r, sum=s, y=y)
    for names in (dict(sum="x"), dict(sum="r"), dict(y="x"), dict(y="r"), dict(sum="x", y="r"), dict(sum="r", y="x")):
        b = dict(x=x.clone(), r=r.clone())
        again = torch.empty_like(xq)
        q.qmm_rms_norm_q8_0(b["x"], None, again, residual=b["r"], **{k: b[v] for k, v in names.items()})
        assert torch.equal(again, xq), names
        for k, v in names.items():
            assert torch.equal(b[v], dict(sum=s, y=y)[k]), names
    wide = torch.empty(T, xq.shape[1], dtype=torch.uint8, device="cuda")
    q.qmm_rms_norm_q8_0(x[:1].expand(T, K), None, wide, residual=r[:1].expand(T, K))
    assert torch.equal(wide, xq[:1].expand(T, -1))


def test_two_streams_at_once(env):
    """The same matrices on two streams, a plan each."""
    torch, q, orc = env
    _say("two streams")
    E, top, N, K, T = 8, 2, 136, 512, 400
    rng = np.random.default_rng(0)
    w, _ = _matrices(torch, orc, q, "q4_0", E, N, K, rng)
    sides = []
    for n in range(2):
        xq = _dev(torch, np.asarray(orc.quantize_x("q4_0", rng.standard_normal((T, K)).astype(np.float32))).reshape(T, -1))
        sides.append(dict(ids=_dev(torch, _ids(rng, T, top, E)), xq=xq, plan=q.experts_plan(T, top, E),
                          y=torch.empty(T, top, N, device="cuda"), stream=torch.cuda.Stream()))

    def run(s, stream):
        q.qmm_experts_plan(s["ids"], E, s["plan"], stream=stream)
        q.qmm_experts_matmul_q4_0(w, s["xq"], s["ids"], s["plan"], s["y"], stream=stream)
    want = []
    for s in sides:
        run(s, None)
        want.append(s["y"].clone())
    torch.cuda.synchronize()
    for _ in range(5):
        for s in sides:
            with torch.cuda.stream(s["stream"]):
                s["y"].fill_(math.nan)
            run(s, s["stream"])
        torch.cuda.synchronize()
        assert all(torch.equal(s["y"], v) for s, v in zip(sides, want))


def test_two_graphs_by_turns(env):
    """Two captured passes of different sizes, replayed by turns: nothing of one is left in the other."""
    torch, q, orc = env
    _say("two graphs")
    made = []
    for T in (20, 260):
        b, step, _, _ = _block(torch, q, "q4_k", T, seed=T, orc=orc)
        b["x"].normal_()
        keep = b["stream"].normal_().clone()
        step()
        want = b["out"].clone()
        b["stream"].copy_(keep)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        made.append((b, keep, want, graph, step))        # the pass holds the matrices
    for _ in range(3):
        for b, keep, want, graph, _ in made:
            b["stream"].copy_(keep)
            b["out"].fill_(math.nan)
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(b["out"], want) for b, _, want, _, _ in made)
