"""The mixture-of-experts entry points' refusals (no GPU: the addresses are not
memory, so every call is one that is refused, where the rest is fine for an array
that is missing)."""
import math

import pytest

A = 1 << 20
OK_UP_TO_NULL, SHAPE, NULL, ALIGN = 2, 1, 2, 3
FORMATS = ("q4_0", "q8_0", "q4_1", "q5_0", "q5_1", "q2_k", "q4_k", "q6_k")


@pytest.fixture(scope="module")
def q():
    import matmul_quantize_q8_amd as q
    q.lib()
    return q


def norm(q, fmt="q8_0", **kw):
    a = dict(x=A, residual=A, sum=A, weight=A, xq=None, y=A, dtype=0, T=4, K=512, xs=512, rs=512, ss=512, ys=512, eps=1e-6,
             offset=0.0)
    a.update(kw)
    return getattr(q.lib(), "qmm_rms_norm_" + fmt)(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(), NULL), (dict(T=0), SHAPE), (dict(T=-1), SHAPE), (dict(K=0), SHAPE), (dict(K=40), SHAPE), (dict(dtype=3), SHAPE),
    (dict(dtype=-1), SHAPE), (dict(eps=-1.0), SHAPE), (dict(eps=math.nan), SHAPE), (dict(eps=math.inf), SHAPE),
    (dict(offset=math.nan), SHAPE), (dict(x=None), NULL), (dict(x=A + 4), ALIGN), (dict(xs=-4), SHAPE), (dict(xs=513), ALIGN),
    (dict(residual=A + 8), ALIGN), (dict(residual=None, rs=-1), NULL), (dict(ss=508), SHAPE), (dict(ys=256), SHAPE),
    (dict(sum=None, ss=-1), NULL), (dict(y=None, ys=0), NULL), (dict(xs=0), NULL), (dict(xq=A + 2), ALIGN),
    (dict(xq=A, weight=A + 4), ALIGN), (dict(T=1, xs=3, rs=-7, ss=1, ys=2), NULL), (dict(T=1 << 31), SHAPE),
    (dict(T=1 << 30, K=1 << 20, xs=0), SHAPE), (dict(xs=1 << 50), SHAPE)])
def test_norm(q, kw, code):
    for fmt in ("q8_0", "q8_k"):
        assert norm(q, fmt, **kw) == code


def test_block_lengths(q):
    assert norm(q, "q8_0", K=544, xs=544, rs=544, ss=544, ys=544) == NULL
    assert norm(q, "q8_k", K=544, xs=544, rs=544, ss=544, ys=544) == SHAPE


def glu(q, fmt="q8_0", **kw):
    a = dict(gate=A, up=A, xq=None, dtype=1, act=0, rows=4, F=512, gs=1024, us=1024)
    a.update(kw)
    return getattr(q.lib(), "qmm_glu_" + fmt)(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(), NULL), (dict(rows=0), SHAPE), (dict(F=100), SHAPE), (dict(act=3), SHAPE), (dict(act=-1), SHAPE),
    (dict(dtype=5), SHAPE), (dict(gate=None), NULL), (dict(up=A + 4), ALIGN), (dict(us=1022), ALIGN), (dict(gs=-4), SHAPE),
    (dict(gs=0, us=0), NULL), (dict(xq=A + 8), ALIGN)])
def test_glu(q, kw, code):
    for fmt in ("q8_0", "q8_k"):
        assert glu(q, fmt, **kw) == code


def route(q, **kw):
    a = dict(logits=A, dtype=0, bias=A, ids=A, weights=None, T=4, E=64, stride=64, top=8, score=0, groups=1, kept=1,
             group_top=1, renorm=1, scale=1.0)
    a.update(kw)
    return q.lib().qmm_route(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(), NULL), (dict(T=0), SHAPE), (dict(T=1 << 24), SHAPE), (dict(E=0), SHAPE), (dict(E=513), SHAPE),
    (dict(E=512, top=64), NULL), (dict(E=512, top=65), SHAPE), (dict(top=0), SHAPE), (dict(E=8, top=9), SHAPE),
    (dict(score=2), SHAPE), (dict(groups=0), SHAPE), (dict(groups=7), SHAPE), (dict(groups=128, E=128), SHAPE),
    (dict(groups=8, kept=9), SHAPE), (dict(groups=8, kept=0), SHAPE), (dict(groups=8, kept=1), NULL),
    (dict(groups=16, kept=1), SHAPE), (dict(group_top=3), SHAPE), (dict(group_top=0), SHAPE), (dict(scale=math.nan), SHAPE), (dict(scale=math.inf), SHAPE), (dict(scale=-math.inf), SHAPE),
    (dict(stride=-1), SHAPE), (dict(stride=0), NULL), (dict(logits=None), NULL), (dict(logits=A + 2), ALIGN),
    (dict(logits=A + 2, dtype=2), NULL), (dict(ids=None), NULL), (dict(ids=A + 1), ALIGN), (dict(bias=A + 2, weights=A), ALIGN),
    (dict(bias=None), NULL), (dict(dtype=3), SHAPE)])
def test_route(q, kw, code):
    assert route(q, **kw) == code


def test_plan_bytes(q):
    size = q.qmm_experts_plan_bytes
    for bad in ((0, 1, 1), (1, 0, 1), (1, 1, 0), (1, 65, 128), (1, 1, 513), ((1 << 26) + 1, 1, 8), (1 << 23, 9, 8)):
        assert size(*bad) == 0, bad
    # room for every pair, its token, and the most tiles: T top_k pairs may all lie in one expert or be spread
    for T, top, E in ((1, 1, 1), (64, 8, 128), (4096, 8, 64), (1 << 20, 8, 512), (65, 1, 512)):
        assert size(T, top, E) >= 8 * T * top + 32
    assert size(1 << 26, 1, 8) > 0 and size(1 << 20, 64, 512) > 0


@pytest.mark.parametrize("top,E", [(1, 1), (1, 8), (1, 512), (2, 8), (4, 512), (8, 128), (64, 64)])
def test_plan_bytes_suffice_for_fewer_tokens(q, top, E):
    """A buffer made for the largest batch serves every smaller one: around each change of the rows of a tile and of
    the pairs of a segment, and between."""
    size = q.qmm_experts_plan_bytes
    edges = {n // top + d for n in (1, 64, 2048, 4096, 16 * E, 20 * E, 32 * E, 64 * E, 128 * E, 1 << 18, 1 << 26) for d in
             range(-70, 71)}
    between = {int(1.003 ** k) for k in range(6100)} | {(1 << 18) * k // (16 * top) for k in range(1, 64)}
    sizes = [size(T, top, E) for T in sorted(edges | between) if 1 <= T <= (1 << 26) // top]
    assert len(sizes) > 2000 and sizes == sorted(sizes) and sizes[0] > 0
    # the calls take it
    assert plan(q, T=(1 << 18) // top, top=top, E=E, bytes=size((1 << 18) // top + 1, top, E)) == NULL


def plan(q, **kw):
    a = dict(ids=A, plan=None, bytes=1 << 20, T=100, top=2, E=8)
    a.update(kw)
    return q.lib().qmm_experts_plan(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(), NULL), (dict(T=0), SHAPE), (dict(bytes=100), SHAPE), (dict(E=513), SHAPE), (dict(ids=None), NULL),
    (dict(ids=A + 2), ALIGN), (dict(plan=A + 8), ALIGN)])
def test_plan(q, kw, code):
    assert plan(q, **kw) == code


def product(q, fmt, **kw):
    rb = q.row_bytes(fmt, 512)
    a = dict(w=A, stride=64 * rb, xq=A, x_rows=100, ids=A, plan=None, bytes=1 << 20, y=A, T=100, top=2, E=8, N=64, K=512)
    a.update(kw)
    return getattr(q.lib(), "qmm_experts_matmul_" + fmt)(*a.values(), None)


@pytest.mark.parametrize("fmt", FORMATS)
def test_product(q, fmt):
    rb = q.row_bytes(fmt, 512)
    for kw, code in [
            (dict(), NULL), (dict(x_rows=200), NULL), (dict(x_rows=101), SHAPE), (dict(x_rows=0), SHAPE), (dict(N=0), SHAPE),
            (dict(N=(1 << 20) + 1, stride=1 << 35), SHAPE), (dict(K=500), SHAPE), (dict(K=0), SHAPE), (dict(T=0), SHAPE),
            (dict(stride=64 * rb - 16), SHAPE), (dict(stride=64 * rb + 16), NULL), (dict(stride=64 * rb + 8), ALIGN),
            (dict(stride=1 << 60), SHAPE), (dict(bytes=64), SHAPE), (dict(w=None), NULL), (dict(w=A + 8), ALIGN),
            (dict(xq=A + 2), ALIGN), (dict(y=A + 4), ALIGN), (dict(y=None), NULL), (dict(ids=None), NULL),
            (dict(ids=A + 2), ALIGN), (dict(plan=A + 4), ALIGN), (dict(E=513), SHAPE),
            (dict(T=1 << 25, x_rows=1 << 25), SHAPE)]:                     # activations of 4 GiB and more
        assert product(q, fmt, **kw) == code, kw


def test_product_block_lengths(q):
    assert product(q, "q4_0", K=32, stride=64 * 18) == NULL
    assert product(q, "q4_k", K=32, stride=64 * 144) == SHAPE


def combine(q, **kw):
    a = dict(y=A, weights=None, residual=A, out=A, dtype=2, T=4, top=2, N=64, rs=64, os=64)
    a.update(kw)
    return q.lib().qmm_experts_combine(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(), NULL), (dict(T=0), SHAPE), (dict(N=0), SHAPE), (dict(N=(1 << 20) + 4), SHAPE), (dict(os=60), SHAPE),
    (dict(os=66), ALIGN), (dict(rs=0), NULL), (dict(rs=-4), SHAPE), (dict(out=A + 4), ALIGN), (dict(out=None), NULL),
    (dict(residual=None, rs=-1), NULL), (dict(y=A + 4), ALIGN), (dict(y=None), NULL), (dict(N=63, os=63, rs=63), NULL),
    (dict(N=63, os=62), SHAPE), (dict(N=63, out=A + 1), ALIGN), (dict(N=63, out=A + 2, residual=A + 6), NULL),
    (dict(dtype=3), SHAPE), (dict(top=65), SHAPE), (dict(T=1 << 20, top=64, N=1 << 12, os=1 << 12), SHAPE)])
def test_combine(q, kw, code):
    assert combine(q, **kw) == code


@pytest.mark.parametrize("kw", [dict(os=-3), dict(os=1), dict(rs=-1), dict(rs=1 << 62, os=1 << 62), dict(os=1 << 50)])
def test_combine_of_one_row_reads_no_stride(q, kw):
    """Rows of N values, a multiple of four or not; two rows are refused."""
    for N in (63, 64):
        a = dict(dict(N=N, rs=N, os=N, T=1), **kw)
        assert combine(q, **a) == NULL, N
        assert combine(q, **dict(a, T=2)) != NULL, N


@pytest.mark.parametrize("stride", [-1, 1, 1 << 62])
def test_route_of_one_row_reads_no_stride(q, stride):
    assert route(q, T=1, stride=stride) == NULL
    assert route(q, T=2, stride=stride) == (NULL if stride == 1 else SHAPE)


def test_binding_refuses_other_tensors(q):
    """Shapes, types and devices are checked before the library is called."""
    import torch
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="not on the GPU"):
        q.qmm_rms_norm_q8_0(x, None, torch.zeros(4, 68, dtype=torch.uint8))
    with pytest.raises(ValueError, match="not on the GPU"):
        q.qmm_route(x, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2))
    with pytest.raises(ValueError, match="not on the GPU"):
        q.qmm_experts_plan(torch.zeros(4, 2, dtype=torch.int32), 8, torch.zeros(64, dtype=torch.uint8))
    with pytest.raises(ValueError, match="no plan"):
        q.experts_plan(0, 1, 1)
