"""Decode attention on an MI355X where lengths, pages and masks meet."""
import numpy as np
import pytest

from test_gpu_attention import FORMATS, Setup, _dev, _np, env  # noqa: F401


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("Hq,heads,dim", [(4, 2, 64), (16, 1, 128), (8, 1, 256)])
def test_bad_page_behind_a_mask(env, fmt, Hq, heads, dim):  # noqa: F811
    """A page number outside the cache under positions that length and window leave gives
    NaN whatever the mask hides: all of the page, all of its tile of up to 64 positions, or
    half of the page.  Before the window the page is not looked at."""
    torch, _, _ = env
    print("[case] bad page behind a mask", fmt, Hq, heads, dim, flush=True)
    lens = [400, 400, 400, 400, 400, 30]
    s = Setup(env, fmt, lens, Hq, heads, dim, 16, "f32", 11)
    table = s.table.copy()
    table[:3, 9] = [-1, s.cache.n_pages, -(1 << 31)]         # under positions 144 .. 159
    table[5, 1] = 1 << 30                                    # under the last 14 of 30
    s.pages = _dev(torch, table)
    mask = np.zeros((len(lens), s.max_len), np.float32)
    mask[0, 144:160] = -np.inf
    mask[1, 64:256] = -np.inf
    mask[2, 144:152] = -np.inf
    mask[3, 144:160] = -np.inf                               # the same mask over good pages
    mask[5, 16:30] = -np.inf
    s.run(mask=_dev(torch, mask))
    bad = [0, 1, 2, 5]
    assert np.isnan(_np(s.out)[bad]).all() and np.isnan(_np(s.lse)[bad]).all()
    s.check(mask=mask, rows=[3, 4])
    s.run(mask=_dev(torch, mask), window=200)                # from position 200 on
    assert np.isnan(_np(s.out)[5]).all()
    s.check(mask=mask, rows=[0, 1, 2, 3, 4], window=200)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n", [1, 50, 5000])
def test_lse_of_the_lowest_mask(env, fmt, n):  # noqa: F811
    """Where every position that is seen has the mask's lowest value, the log-sum-exp is
    that value (ln n and the scores are far below half a step of it), the output their
    mean; beside any other position they do not count."""
    torch, _, _ = env
    print("[case] lowest mask", fmt, n, flush=True)
    low = np.finfo(np.float32).min
    s = Setup(env, fmt, [n, n, n], 4, 2, 64, 16, "f32", n)
    mask = np.full((3, n), low, np.float32)
    mask[1, ::2] = -np.inf
    mask[2, n // 2] = -5.0
    if n == 1:
        mask[1] = low
    s.run(mask=_dev(torch, mask))
    lse = _np(s.lse)
    assert np.all(lse[:2] == low) and np.all(np.abs(lse[2]) < 100)
    s.check(mask=mask)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("window", [200, 241, 242, 255, 256, 257, 2985, 2986, 2999])
def test_windows_on_a_workspace_for_all(env, fmt, window):  # noqa: F811
    """Windows up to a position less than the length, on a workspace made without one."""
    print("[case] window", fmt, window, flush=True)
    s = Setup(env, fmt, [257, 256, 3] if window < 300 else [3000, 2990, 40], 8, 2, 64, 16, "f32", window)
    s.run(window=window)
    s.check(window=window)
