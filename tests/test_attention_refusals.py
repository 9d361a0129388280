"""Refusals of the attention entry points that need no GPU: output rows that
share memory, tensors of another device, and the workspace of windows.  The
addresses are not memory, so every call here is one that is refused: where the
rows are fine, for an index array that is missing."""
import itertools

import pytest

from test_attention_host import (FORMATS, GOOD_CACHE, GOOD_PLAN, A, Cache, Plan, _p, attn, q, read,  # noqa: F401
                                 rope)

SHAPE, NULL = 1, 2


def overlap(T, H, D, token, head):
    """Whether two of the rows share an element, from their offsets."""
    at = sorted(t * token + h * head for t in range(T) for h in range(H))
    return any(b - a < D for a, b in zip(at, at[1:]))


def test_output_rows_that_overlap_are_refused(q):  # noqa: F811
    """Every pair of strides up to a few rows, against the offsets themselves."""
    D, seen = 8, set()
    for T, H in itertools.product((1, 2, 3, 5), (1, 2, 3, 4)):
        for token, head in itertools.product(range(0, 49, 4), range(0, 49, 4)):
            bad = overlap(T, H, D, token, head)
            seen.add(bad)
            code = rope(q.lib(), plan=dict(freqs=A, rot=8, order=0, mscale=1.0), T=T, H=H, D=D, xs=(32, 8),
                        ys=(token, head), pos=None)
            assert code == (SHAPE if bad else NULL), (T, H, token, head)
    assert seen == {False, True}


def test_many_heads_between_tokens(q):  # noqa: F811
    """Strides that interleave 4096 heads: token rows between the heads' and not nested in them."""
    def code(T, H, token, head):
        return rope(q.lib(), T=T, H=H, D=64, xs=(0, 0), ys=(token, head), pos=None)
    assert code(2, 4096, 64, 128) == NULL
    assert code(3, 4096, 64, 128) == SHAPE                   # token 2 lies on the next head's token 0
    assert code(1 << 20, 4096, 64, 64 << 20) == NULL
    assert code((1 << 20) + 1, 4096, 64, 64 << 20) == SHAPE
    assert code(1 << 20, 2, 128, 64) == NULL
    assert code(1 << 20, 3, 128, 64) == SHAPE


def test_input_rows_may_overlap(q):  # noqa: F811
    assert rope(q.lib(), xs=(0, 0), pos=None) == NULL
    assert attn(q.lib(), "q8_0", qs=(0, 0), lens=None) == NULL


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("strides", [(0, 64), (128, 0), (0, 0), (64, 64), (96, 64)])
def test_every_output_is_checked(q, fmt, strides):  # noqa: F811
    L = q.lib()
    cache, plan = Cache(**GOOD_CACHE), Plan(**GOOD_PLAN)
    assert read(L, fmt, ks=strides, slots=None) == SHAPE
    assert read(L, fmt, ks=(128, 64), slots=None) == NULL
    f = getattr(L, "qmm_kv_read_" + fmt)
    assert f(_p(cache), None, A, A, 0, 3, 128, 64, *strides, None) == SHAPE
    assert f(_p(cache), None, None, A, 0, 3, 0, 0, *strides, None) == SHAPE
    f = getattr(L, "qmm_rope_kv_write_" + fmt)
    assert f(_p(plan), _p(cache), A, A, A, A, 0, A, None, 3, 4, 256, 64, *strides, 128, 64, 128, 64, None) == SHAPE
    assert f(_p(plan), _p(cache), A, A, A, A, 0, A, None, 3, 4, 256, 64, 256, 64, 128, 64, 128, 64, None) == NULL
    f = getattr(L, "qmm_attn_decode_" + fmt)
    assert f(_p(cache), A, A, 0, A, 8, None, 2, 4, 256, 0.125, 0.0, 0, None, 0, None, 256, 64, *strides, A, 1 << 39,
             None) == SHAPE
