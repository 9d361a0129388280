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


# ---------------------------------------------------------------------------
# Devices: a second one is a stand-in, as no tensor of the calls is read
# ---------------------------------------------------------------------------
class OnDevice:
    """A tensor of a shape and type that says which GPU it is on."""

    def __init__(self, shape, dtype, device=0):
        self.shape, self.dtype, self.index, self.device = tuple(shape), dtype, device, f"cuda:{device}"
        self.is_cuda = device >= 0

    def get_device(self):
        return self.index

    def stride(self):
        s, n = [], 1
        for x in reversed(self.shape):
            s.insert(0, n)
            n *= x
        return tuple(s)

    def numel(self):
        return self.stride()[0] * self.shape[0]

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return A


def _calls(q, fmt):  # noqa: F811
    """(function of named stand-ins, the stand-ins' shapes and types) of every entry point."""
    import torch
    f, i4, i8, u1 = torch.float32, torch.int32, torch.int64, torch.uint8
    size = q.kv_page_bytes(fmt, 16, 2, 64)

    def plan(t):
        return q.RopePlan(t["freqs"])

    def cache(t):
        return q.KVCache(fmt, t["data"], 16, 2, 64)
    rows, plans, caches = {"k": ((3, 2, 64), f), "v": ((3, 2, 64), f)}, {"freqs": ((32,), torch.float64)}, {
        "data": ((4 * size,), u1)}
    slots, positions = {"slots": ((3,), i8)}, {"positions": ((3,), i4)}
    qs = {"q": ((3, 4, 64), f), "out": ((3, 4, 64), f)}
    return {
        "rope": (lambda t: q.qmm_rope(t["k"], t["v"], t["positions"], plan(t)), {**rows, **positions, **plans}),
        "write": (lambda t: q.KV_WRITE[fmt](t["k"], t["v"], cache(t), t["slots"]), {**rows, **slots, **caches}),
        "rope_write": (lambda t: q.ROPE_KV_WRITE[fmt](t["q"], t["out"], t["k"], t["v"], cache(t), t["slots"],
                                                      t["positions"], plan(t)),
                       {**rows, **qs, **slots, **positions, **plans, **caches}),
        "read": (lambda t: q.KV_READ[fmt](cache(t), t["slots"], t["k"], t["v"]), {**rows, **slots, **caches}),
        "read_values": (lambda t: q.KV_READ[fmt](cache(t), t["slots"], None, t["v"]),
                        {"v": rows["v"], **slots, **caches}),
        "attn": (lambda t: q.ATTN_DECODE[fmt](t["q"], t["out"], cache(t), t["pages"], t["lens"], 32, t["workspace"],
                                              mask=t["mask"], lse=t["lse"]),
                 {**qs, **caches, "pages": ((3, 2), i4), "lens": ((3,), i4), "workspace": ((4096,), u1),
                  "mask": ((3, 32), f), "lse": ((3, 4), f)})}


@pytest.mark.parametrize("entry", ["rope", "write", "rope_write", "read", "read_values", "attn"])
def test_tensors_of_another_device_are_refused(q, entry, monkeypatch):  # noqa: F811
    called = []
    monkeypatch.setattr(q.attention, "_call", lambda *a: called.append(a))
    monkeypatch.setattr(q.attention, "_stream", lambda *a: 0)
    monkeypatch.setattr(q.attention, "_current", lambda: 0, raising=False)
    f, tensors = _calls(q, "q8_0")[entry]

    def run(device):
        f({name: OnDevice(*of, device.get(name, device.get("", 0))) for name, of in tensors.items()})
    run({})
    assert len(called) == 1
    for other in (1, -1):
        for name in tensors:
            with pytest.raises(ValueError):
                run({name: other})
    with pytest.raises(ValueError, match="current"):         # all on the device that is not the current one
        run({"": 1})
    monkeypatch.setattr(q.attention, "_current", lambda: 1)
    assert len(called) == 1
    run({"": 1})
    assert len(called) == 2


def test_workspace_of_windows(q):  # noqa: F811
    """A workspace made without a window serves calls with any: a window sees no more than all."""
    size = q.qmm_attn_decode_workspace
    for Hq, heads, dim in ((32, 8, 128), (14, 2, 64), (64, 1, 256)):
        for n in (1, 255, 256, 257, 512, 1000, 4096, 131072):
            whole = {B: size(B, Hq, heads, dim, n) for B in (1, 3, 64, 700)}
            for w in (1, 16, n // 2, n - 241, n - 16, n - 15, n - 2, n - 1, n, n + 1, 2 * n):
                for B in whole:
                    if w > 0:
                        assert 0 < size(B, Hq, heads, dim, n, w) <= whole[B], (Hq, n, w, B)
