"""What decode attention's two-part f16 products keep, against 64 bits.

The limit is on the error's norm over a head's output: with f32 rows every weight
carries four roundings of 2^-22 (the query's split, the score's sum, the
exponential, the weight's split), each of which moves the output by that much of
itself; twice their sum is 2^-19.  A plain f32 computation may be worse (its sums
grow with the length, its scores with their size); then twice its error counts.
The CPU tests show that this limit tells a dropped low part, or a reference that
does not look at the block scales, from the kernel's rule."""
import os
import re

import numpy as np
import pytest

import attention_ref as ref
from conftest import ROOT
from test_gpu_attention import _dev, _np, _pool, env  # noqa: F401

LIMIT = 2.0 ** -19


def off(got, want):
    """Largest relative error of a head's output, in norm."""
    return float((np.linalg.norm(got - want, axis=-1) / np.linalg.norm(want, axis=-1)).max())


def plain_f32(q, k, v, scale):
    """Attention of f32 rows, every step in f32: q [Hq][D], k, v [n][H][D]."""
    q, k, v = (x.astype(np.float32) for x in (q, k, v))
    out, lse, group = np.empty_like(q), np.empty(len(q)), len(q) // k.shape[1]
    for h in range(len(q)):
        s = k[:, h // group] @ q[h] * np.float32(scale)
        p = np.exp(s - s.max())
        out[h], lse[h] = p @ v[:, h // group] / p.sum(dtype=np.float32), s.max() + np.log(p.sum(dtype=np.float32))
    return out.astype(np.float64), lse


def rows(case, n, Hq, heads, dim, seed):
    """q, k, v of a case, f32: the values' magnitude, one position whose score lies
    `sink` above the others' largest and whose values are zero, and one block of 32
    whose values are 2^-`low` of the others'."""
    sigma, sink, low = case
    rng = np.random.default_rng(seed)
    q, k, v = (rng.standard_normal(s).astype(np.float32) for s in ((Hq, dim), (n, heads, dim), (n, heads, dim)))
    q *= 1.5
    v *= np.float32(sigma)
    if sink:
        q[:, 0], k[:, :, 0], at = 4.0, 0.0, n // 3
        top = max(float((k[:, h] @ q[h * (Hq // heads):(h + 1) * (Hq // heads)].T).max()) for h in range(heads))
        k[at], v[at] = 0.0, 0.0
        k[at, :, 0] = top / 4 + sink * dim ** 0.5 / 4
    if low:
        v[..., 32:64] *= np.float32(2.0 ** -low)
    return q, k, v


# ---------------------------------------------------------------------------
# The products' split, on the CPU
# ---------------------------------------------------------------------------
def _f16(x):
    return x.astype(np.float16).astype(np.float64)


def _constants():
    text = open(os.path.join(ROOT, "matmul_quantize_q8_amd", "csrc", "attn_chunk.h")).read()
    c = {n: float(re.search(rf"\b{n} = (-?[0-9.]+)f?[,;]", text).group(1)) for n in (
        "kWeightBits", "kSlackBits", "kMostBits", "kSetBits", "kLeastBits", "kReachBits", "kNoScale", "kMostLift")}
    return c, {"q8_0": int(re.search(r"kFirstLift = F == KV_Q8_0 \? (\d+) : 0", text).group(1)), "q4_0": 0}


def _coded(v, fmt):
    """Codes [n][blocks][32] and f16 scales [n][blocks] of rows [n][dim]."""
    b = v.astype(np.float64).reshape(len(v), -1, 32)
    if fmt == "q8_0":
        d = np.abs(b).max(-1) / 127
    else:
        d = np.take_along_axis(b, np.abs(b).argmax(-1)[..., None], -1)[..., 0] / -8
    low, high = (-128, 127) if fmt == "q8_0" else (-8, 7)
    code = np.clip(np.rint(b / np.where(d, d, 1.0)[..., None]), low, high)
    return code * (d != 0)[..., None], _f16(d)


def split_attention(s, code, d, fmt, weights=2, blind=False):
    """One head by the kernel's rule, everything else exact: s [n] log2 scores; four
    waves take tiles of 64 in turn, four column groups of 16 each with references of
    its own.  `weights` f16 parts a product; blind: every tile is a common one, its
    scales as they are."""
    c, first = _constants()
    parts = []
    for wave in range(4):
        lift, gained = 0 if blind else first[fmt], False
        r, rp, l, o = [-np.inf] * 4, [-np.inf] * 4, [0.0] * 4, [np.zeros(code.shape[1:]) for _ in range(4)]
        for t in range(64 * wave, len(s), 256):
            cols = [x for x in range(4) if t + 16 * x < len(s)]
            at = [slice(t + 16 * x, min(t + 16 * x + 16, len(s))) for x in cols]
            scales = np.abs(d[t:t + 64]) * 2.0 ** lift
            tops = [s[i].max() for i in at]
            uncommon = not blind and (gained or scales.min() < 2.0 ** -7 or scales.max() >= 2.0)
            by, was = 1.0, lift
            if uncommon:
                largest = np.abs(d[t:t + 64]).max()
                if largest > 0 and abs(np.log2(largest) + lift + 2.5) > 3.5:
                    lift = int(min(max(-2 - np.floor(np.log2(largest)), 0), c["kMostLift"]))
                by, gained, scales = 2.0 ** (lift - was), False, np.abs(d[t:t + 64]) * 2.0 ** lift
                least = c["kLeastBits"] if scales.min() < 2.0 ** -7 or scales.max() >= 2.0 else 0.0
            for x in range(4):
                o[x] = o[x] * by
            for x, i in zip(cols, at):
                dt = d[i] * 2.0 ** lift
                nxt = r[x]
                if tops[x] - r[x] > c["kWeightBits"] + c["kSlackBits"]:
                    nxt = np.floor(tops[x] - c["kWeightBits"])
                    l[x] *= 2.0 ** (r[x] - nxt)
                to = nxt
                if uncommon:
                    e = np.abs(dt).max(-1)
                    most = (s[i] + np.where(e > 0, np.log2(np.where(e > 0, e, 1.0)), c["kNoScale"] + lift)).max()
                    if not least <= most - nxt <= c["kMostBits"]:
                        b = most - rp[x]
                        move = b > c["kMostBits"] or (b < c["kLeastBits"] and most > nxt - c["kReachBits"])
                        to = max(np.floor(most - c["kSetBits"]), nxt - c["kReachBits"]) if move else rp[x]
                    gained = gained or to != nxt
                o[x] = o[x] * 2.0 ** (rp[x] - to)
                r[x], rp[x] = nxt, to
                p = 2.0 ** (s[i] - nxt)
                w = (p * 2.0 ** (nxt - to))[:, None] * dt
                hi = _f16(w)
                assert np.all(np.isfinite(hi))
                w = hi + _f16(w - hi) if weights == 2 else hi
                l[x], o[x] = l[x] + p.sum(), o[x] + (w[..., None] * code[i]).sum(0)
        parts += [(r[x], l[x], o[x] * 2.0 ** (rp[x] - r[x] - lift)) for x in range(4) if r[x] > -np.inf]
    top = max(p[0] for p in parts)
    l, o = (sum(p[i] * 2.0 ** (p[0] - top) for p in parts) for i in (1, 2))
    return (o / l).ravel()


CASES = [(1.0, 0, 0), (1e-2, 0, 0), (1e-3, 0, 0), (1e-4, 0, 0), (1e-5, 0, 0), (0.3, 8, 0), (0.3, 12, 0), (0.3, 16, 0),
         (0.3, 30, 0), (1.0, 0, 6), (1.0, 0, 10), (300.0, 0, 0)]


def _model(case, fmt, n):
    q, k, v = rows(case, n, 1, 1, 128, n)
    s = (k[:, 0].astype(np.float64) @ q[0]) * 128 ** -0.5 * np.log2(np.e)
    code, d = _coded(v[:, 0], fmt)
    p = 2.0 ** (s - s.max())
    return s, code, d, ((p[:, None] * d)[..., None] * code).sum(0).reshape(-1, 32) / p.sum()


@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
@pytest.mark.parametrize("n", [40, 700, 4096])
@pytest.mark.parametrize("case", CASES)
def test_split_keeps_22_bits(case, fmt, n):
    s, code, d, want = _model(case, fmt, n)
    assert off(split_attention(s, code, d, fmt).reshape(-1, 32), want) < LIMIT          # a block at a time


@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
def test_limit_tells_weights_of_one_part(fmt):
    for case in CASES:
        s, code, d, want = _model(case, fmt, 700)
        assert off(split_attention(s, code, d, fmt, weights=1).reshape(-1, 32), want) > 20 * LIMIT


@pytest.mark.parametrize("case", [(1e-3, 0, 0), (1e-4, 0, 0), (1e-5, 0, 0), (0.3, 8, 0), (0.3, 12, 0), (0.3, 16, 0)])
def test_limit_tells_a_reference_without_scales(case):
    s, code, d, want = _model(case, "q8_0", 700)
    assert off(split_attention(s, code, d, "q8_0", blind=True).reshape(-1, 32), want) > 2 * LIMIT


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_limit_tells_queries_of_one_part(dim):
    q, k, v = (x.astype(np.float64) for x in rows((1.0, 0, 0), 700, 4, 2, dim, dim))
    up = 2.0 ** (7 - np.floor(np.log2(np.abs(q).max(-1, keepdims=True))))
    hi = _f16(q * up)
    two, one = (hi + _f16(q * up - hi)) / up, hi / up
    want = ref.attention(q, k, v, dim ** -0.5)[0]
    assert off(ref.attention(two, k, v, dim ** -0.5)[0], want) < LIMIT
    assert off(ref.attention(one, k, v, dim ** -0.5)[0], want) > 20 * LIMIT


# ---------------------------------------------------------------------------
# The kernels
# ---------------------------------------------------------------------------
def attend(env, fmt, q, k, v, page=64, **kw):
    """One sequence through the library, f32 rows: out, lse, and the decoded k and v."""
    torch, lib, orc = env
    n, heads, dim = k.shape
    cache = _pool(torch, lib, fmt, -(-n // page) + 1, page, heads, dim)
    table = np.random.default_rng(n).permutation(cache.n_pages)[None, :-(-n // page)].astype(np.int32)
    i = np.arange(n)
    slots = table[0][i // page].astype(np.int64) * page + i % page
    lib.KV_WRITE[fmt](_dev(torch, k), _dev(torch, v), cache, _dev(torch, slots))
    qd = _dev(torch, q[None])
    out = torch.full_like(qd, float("nan"))
    lse = torch.full((1, len(q)), float("nan"), device="cuda")
    lib.ATTN_DECODE[fmt](qd, out, cache, _dev(torch, table), torch.tensor([n], dtype=torch.int32, device="cuda"), n,
                         lib.attn_workspace(1, len(q), heads, dim, n), lse=lse, **kw)
    return _np(out)[0], _np(lse)[0], ref.through_cache(k, fmt, orc), ref.through_cache(v, fmt, orc)


def check(env, fmt, q, k, v, page=64, block=False):
    print("[case] accuracy", fmt, q.shape, k.shape, page, flush=True)
    dim = q.shape[1]
    got, lse, k, v = attend(env, fmt, q, k, v, page)
    want, l = ref.attention(q.astype(np.float64), k, v, dim ** -0.5)[:2]
    plain, pl = plain_f32(q, k, v, dim ** -0.5)
    if block:
        got, want, plain = (x.reshape(-1, 32) for x in (got, want, plain))
    at, limit = off(got, want), max(LIMIT, 2 * off(plain, want))
    assert at <= limit, (at, limit)
    assert np.all(np.abs(lse - l) <= LIMIT * (1 + np.abs(l)) + 2 * np.abs(pl - l).max())


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["f16", "q8_0", "q4_0"])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("Hq,heads", [(6, 2), (8, 1), (20, 1)])
def test_attention_keeps_22_bits(env, fmt, dim, Hq, heads):  # noqa: F811
    check(env, fmt, *rows((1.0, 0, 0), 300, Hq, heads, dim, dim + Hq), page=32)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["f16", "q8_0", "q4_0"])
@pytest.mark.parametrize("Hq,heads", [(8, 2), (8, 1), (16, 1)])
def test_long_attention_keeps_22_bits(env, fmt, Hq, heads):  # noqa: F811
    check(env, fmt, *rows((1.0, 0, 0), 6000, Hq, heads, 128, Hq))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
@pytest.mark.parametrize("dim,Hq,heads", [(64, 4, 2), (96, 5, 1), (96, 16, 1), (128, 8, 2), (192, 16, 1), (256, 4, 1)])
@pytest.mark.parametrize("n", [40, 700])
@pytest.mark.parametrize("case", CASES[1:])
def test_attention_keeps_22_bits_at_any_scale(env, fmt, dim, Hq, heads, n, case):  # noqa: F811
    """Small values, large ones, positions of zero values with the largest score,
    blocks far below the others (each block's error over its own norm)."""
    check(env, fmt, *rows(case, n, Hq, heads, dim, n + dim), block=case[2] > 0)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
def test_one_large_value_costs_the_others_nothing(env, fmt):  # noqa: F811
    q, k, v = rows((0.1, 0, 0), 3000, 8, 2, 128, 3)
    v[5, :, 40] = 300.0
    check(env, fmt, q, k, v, block=True)


@pytest.mark.gpu
@pytest.mark.parametrize("sink", [8, 16])
def test_f16_cache_beside_a_zero_row(env, sink):  # noqa: F811
    """f16 caches have no scales: beside the largest weight of its tile of at most
    64 positions, a product is off by up to 2^-29 of that weight; other tiles keep
    22 bits of their own."""
    q, k, v = rows((0.3, sink, 0), 700, 4, 2, 128, sink)
    got, _, k, v = attend(env, "f16", q, k, v)
    want = ref.attention(q.astype(np.float64), k, v, 128 ** -0.5)[0]
    plain = plain_f32(q, k, v, 128 ** -0.5)[0]
    size = np.linalg.norm(want, axis=-1)
    tile = 64 * 2.0 ** -29 * np.linalg.norm(v, axis=-1).max()       # the sink's weight is nearly all of the sum
    err = np.linalg.norm(got - want, axis=-1)
    assert np.all(err <= max(LIMIT, 2 * off(plain, want)) * size + tile)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["f16", "q8_0", "q4_0"])
@pytest.mark.parametrize("scale", [1.0, 300.0])
@pytest.mark.parametrize("low", [-1e4, -3e7, -6e7, -1e8, -1.3e8, -1.8e8, -1e9, -1e20])
def test_equal_masks_of_any_size(env, fmt, scale, low):  # noqa: F811
    """Scores that are all equal, at magnitudes whose f32 step is up to more than the
    reference's distance: the output is the mean, the log-sum-exp the mask's value."""
    torch, lib, _ = env
    print("[case] equal masks", fmt, scale, low, flush=True)
    q, k, v = rows((scale, 0, 0), 300, 4, 2, 64, 5)
    mask = torch.full((1, 300), low, device="cuda")
    got, lse, _, v = attend(env, fmt, 0 * q, k, v, page=16, mask=mask)
    want = v.mean(0).repeat(2, 0)
    assert off(got, want) < LIMIT
    exact = float(mask[0, 0]) + np.log(300)
    assert np.all(np.abs(lse - exact) <= 2.0 ** -22 * abs(exact))
