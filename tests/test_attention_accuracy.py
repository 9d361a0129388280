"""Decode attention at the edges of its f16 products' range, against 64 bits.

The limit is on the error's norm over a head's output: with f32 rows every weight
carries four roundings of 2^-22 (the query's split, the score's sum, the
exponential, the weight's split), each of which moves the output by that much of
itself; twice their sum is 2^-19."""
import numpy as np
import pytest

import attention_ref as ref
from test_gpu_attention import _dev, _np, _pool, env  # noqa: F401

LIMIT = 2.0 ** -19


def off(got, want):
    """Largest relative error of a head's output, in norm."""
    return float((np.linalg.norm(got - want, axis=-1) / np.linalg.norm(want, axis=-1)).max())


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
