"""Binding of the attention operators: rotary positions, the paged key-value
cache and the attention of one new token over it (include/qmm.h).

Rows are torch tensors [tokens][heads][dim] of float32, float16 or bfloat16 on
the GPU, the values of a row contiguous, any token and head strides (so slices
of a fused QKV product go in as they are).  Shapes, types and devices (every
tensor of a call is on the current one) are checked here (ValueError); sizes,
strides and alignment by the library (QmmError).  Nothing is copied and nothing
is allocated by a call, except by the helpers that say so.
"""
from __future__ import annotations

import ctypes
import math

KV_FORMATS = ("f16", "q8_0", "q4_0")
ROPE_ORDERS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"plain": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}

EXPORTS = tuple(["qmm_rope", "qmm_rope_freqs", "qmm_attn_decode_workspace"] +
                [p + f for p in ("qmm_kv_page_bytes_", "qmm_kv_write_", "qmm_rope_kv_write_", "qmm_kv_read_",
                                 "qmm_attn_decode_") for f in KV_FORMATS])


class _Plan(ctypes.Structure):
    _fields_ = [("freqs", ctypes.c_void_p), ("rot", ctypes.c_int64), ("order", ctypes.c_int32),
                ("mscale", ctypes.c_float)]


class _Cache(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("page", ctypes.c_int64),
                ("heads", ctypes.c_int64), ("dim", ctypes.c_int64)]


def declare(L) -> None:
    """Argument types of the attention entry points of libqmm.so."""
    P, I64, I32, F, D = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_double
    sig = {"qmm_rope_freqs": [P, P, I64, D, I32, D, D, D, D],
           "qmm_rope": [P, P, P, I32, P, I32] + 7 * [I64] + [P]}
    for f in KV_FORMATS:
        sig["qmm_kv_write_" + f] = [P, P, P, I32, P] + 5 * [I64] + [P]
        sig["qmm_rope_kv_write_" + f] = [P, P, P, P, P, P, I32, P, P] + 10 * [I64] + [P]
        sig["qmm_kv_read_" + f] = [P, P, P, P, I32] + 5 * [I64] + [P]
        sig["qmm_attn_decode_" + f] = [P, P, P, I32, P, I64, P, I64, I64, I64, F, F, I64, P, I64, P, I64, I64, I64,
                                       I64, P, I64, P]
    for name, args in sig.items():
        getattr(L, name).argtypes = args
        getattr(L, name).restype = ctypes.c_int
    for f in KV_FORMATS:
        getattr(L, "qmm_kv_page_bytes_" + f).argtypes = [I64, I64, I64]
        getattr(L, "qmm_kv_page_bytes_" + f).restype = I64
    L.qmm_attn_decode_workspace.argtypes = [I64] * 6
    L.qmm_attn_decode_workspace.restype = I64


# Set by the package: its call, the stream of a call on a device, its library
# access and the current device.
_call = _stream = _lib = _current = None


def bind(call, stream, lib, current) -> None:
    global _call, _stream, _lib, _current
    _call, _stream, _lib, _current = call, stream, lib, current


# torch, imported at the first use of it, and the row types' codes.
_torch = None
_CODES = {}


def _t():
    global _torch
    if _torch is None:
        import torch
        _CODES.update({torch.float32: 0, torch.float16: 1, torch.bfloat16: 2})
        _torch = torch
    return _torch


def _device(name, t) -> int:
    """The index of a call's first tensor's device, which has to be the current one."""
    device = t.get_device()
    if device < 0:
        raise _elsewhere(name, device, None)
    if device != _current():
        raise ValueError(f"{name}: on cuda:{device}, and the current device is cuda:{_current()}")
    return device


def _elsewhere(name, got, device):
    return ValueError(f"{name}: not on the GPU" if got < 0 else f"{name}: on cuda:{got}, the call is on cuda:{device}")


def _rows(name, t, shape, dtype, device):
    """(address, token stride, head stride) of rows of that shape and type."""
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name}: want {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    token, head, one = t.stride()
    if one != 1:
        raise ValueError(f"{name}: the values of a row have to be contiguous")
    if t.get_device() != device:
        raise _elsewhere(name, t.get_device(), device)
    return t.data_ptr(), token, head


def _code(dtype) -> int:
    c = _CODES.get(dtype)
    if c is None:
        raise ValueError(f"rows are float32, float16 or bfloat16, not {dtype}")
    return c


def _three(name, t):
    """The shape of rows."""
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name}: want rows [tokens][heads][dim], got {tuple(shape)}")
    return shape


def _array(name, t, dtype, shape, device=None):
    """Address of a contiguous array on the GPU, on the call's device if there is a call."""
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: want a contiguous {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    on = t.get_device()
    if on < 0 or (on != device and device is not None):
        raise _elsewhere(name, on, device)
    return t.data_ptr()


# -- rotation -------------------------------------------------------------------
def qmm_rope_freqs(rot: int, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0,
                   trained_len: float = 0.0, low: float = 0.0, high: float = 0.0):
    """(frequencies, mscale) of a rotation of `rot` values: a float64 CPU tensor [rot/2] and a float."""
    torch = _t()
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling is one of {', '.join(ROPE_SCALINGS)}, not {scaling!r}")
    out, ms = torch.empty(max(int(rot) // 2, 1), dtype=torch.float64), ctypes.c_float()
    _call("qmm_rope_freqs", out.data_ptr(), ctypes.addressof(ms), rot, base, ROPE_SCALINGS[scaling], factor,
          trained_len, low, high)
    return out, ms.value


class RopePlan:
    """A model's rotation: frequencies (float64 [rot/2] on the GPU), the order of
    the pairs ("half" or "interleaved") and the factor on cosine and sine."""

    def __init__(self, freqs, order: str = "half", mscale: float = 1.0):
        torch = _t()
        if order not in ROPE_ORDERS:
            raise ValueError(f"order is one of {', '.join(ROPE_ORDERS)}, not {order!r}")
        self.freqs = freqs
        self._c = _Plan(_array("freqs", freqs, torch.float64, (freqs.numel(),)), 2 * freqs.numel(),
                        ROPE_ORDERS[order], mscale)
        self._p, self._device = ctypes.addressof(self._c), freqs.get_device()

    def on(self, device):
        """The C structure's address, for a call on that device."""
        if device != self._device:
            raise _elsewhere("plan", self._device, device)
        return self._p


def qmm_rope(x, y, positions, plan: RopePlan, inverse: bool = False, stream=None) -> None:
    """y = x [T][H][D] with the first rot values of every row rotated to its
    token's position (int32 [T]); inverse: by the negative angle, which takes
    the gradient of y to that of x.  y may be x."""
    torch, shape, dtype, device = _t(), _three("x", x), x.dtype, _device("x", x)
    xa, xt, xh = _rows("x", x, shape, dtype, device)
    ya, yt, yh = _rows("y", y, shape, dtype, device)
    _call("qmm_rope", plan.on(device), xa, ya, _code(dtype),
          _array("positions", positions, torch.int32, shape[:1], device), 1 if inverse else 0, shape[0], shape[1],
          shape[2], xt, xh, yt, yh, _stream(stream, device))


# -- cache ----------------------------------------------------------------------
def kv_page_bytes(fmt: str, page: int, heads: int, dim: int) -> int:
    """Bytes of one page of a cache in `fmt` (0 for sizes outside the limits)."""
    return getattr(_lib(), "qmm_kv_page_bytes_" + fmt)(page, heads, dim)


def _page_bytes(fmt):
    def page_bytes(page: int, heads: int, dim: int) -> int:
        return kv_page_bytes(fmt, page, heads, dim)
    page_bytes.__name__ = "qmm_kv_page_bytes_" + fmt
    page_bytes.__doc__ = f"Bytes of one page of a {fmt} cache (0 for sizes outside the limits)."
    return page_bytes


class KVCache:
    """One layer's paged key-value cache over `data`, a contiguous uint8 tensor
    on the GPU of a whole number of pages (KVCache.empty makes one)."""

    def __init__(self, fmt: str, data, page: int, heads: int, dim: int):
        torch = _t()
        if fmt not in KV_FORMATS:
            raise ValueError(f"the cache's format is one of {', '.join(KV_FORMATS)}, not {fmt!r}")
        size = kv_page_bytes(fmt, page, heads, dim)
        if size == 0:
            raise ValueError(f"no cache of pages of {page} positions, {heads} heads of {dim}")
        _array("data", data, torch.uint8, (data.numel(),))
        if data.numel() == 0 or data.numel() % size:
            raise ValueError(f"data: {data.numel()} bytes are no whole number of pages of {size}")
        self.fmt, self.data, self.page, self.heads, self.dim = fmt, data, page, heads, dim
        self.n_pages = data.numel() // size
        self._c = _Cache(data.data_ptr(), self.n_pages, page, heads, dim)
        self._p, self._device = ctypes.addressof(self._c), data.get_device()

    @classmethod
    def empty(cls, fmt: str, n_pages: int, page: int, heads: int, dim: int, device="cuda"):
        """A new cache; its rows hold nothing until they are written."""
        return cls(fmt, _t().empty(n_pages * kv_page_bytes(fmt, page, heads, dim), dtype=_torch.uint8, device=device),
                   page, heads, dim)


def _of(cache, fmt, device):
    if cache.fmt != fmt:
        raise ValueError(f"the cache holds {cache.fmt}, not {fmt}")
    if cache._device != device:
        raise _elsewhere("cache", cache._device, device)
    return cache._p


def _kv_write(fmt):
    name = "qmm_kv_write_" + fmt

    def kv_write(k, v, cache: KVCache, slots, stream=None) -> None:
        torch, dtype, T, device = _t(), k.dtype, k.shape[0], _device("k", k)
        shape = (T, cache.heads, cache.dim)
        ka, kt, kh = _rows("k", k, shape, dtype, device)
        va, vt, vh = _rows("v", v, shape, dtype, device)
        _call(name, _of(cache, fmt, device), ka, va, _code(dtype), _array("slots", slots, torch.int64, (T,), device), T,
              kt, kh, vt, vh, _stream(stream, device))
    kv_write.__name__ = name
    kv_write.__doc__ = f"Write keys and values [T][H][D] into the slots (int64 [T]) of a {fmt} cache."
    return kv_write


def _rope_kv_write(fmt):
    name = "qmm_rope_kv_write_" + fmt

    def rope_kv_write(q, q_out, k, v, cache: KVCache, slots, positions, plan: RopePlan, stream=None) -> None:
        torch, dtype, T, device = _t(), k.dtype, k.shape[0], _device("k", k)
        shape, qshape = (T, cache.heads, cache.dim), (T, _three("q", q)[1], cache.dim)
        qa, qt, qh = _rows("q", q, qshape, dtype, device)
        oa, ot, oh = _rows("q_out", q_out, qshape, dtype, device)
        ka, kt, kh = _rows("k", k, shape, dtype, device)
        va, vt, vh = _rows("v", v, shape, dtype, device)
        _call(name, plan.on(device), _of(cache, fmt, device), qa, oa, ka, va, _code(dtype),
              _array("positions", positions, torch.int32, (T,), device),
              _array("slots", slots, torch.int64, (T,), device), T, qshape[1], qt, qh, ot, oh, kt, kh, vt, vh,
              _stream(stream, device))
    rope_kv_write.__name__ = name
    rope_kv_write.__doc__ = (f"Rotate queries into q_out and write the rotated keys and the values into the slots "
                             f"of a {fmt} cache, in one launch.")
    return rope_kv_write


def _kv_read(fmt):
    name = "qmm_kv_read_" + fmt

    def kv_read(cache: KVCache, slots, k, v, stream=None) -> None:
        torch = _t()
        some = k if k is not None else v
        if some is None:
            raise ValueError("neither k nor v is wanted")
        dtype, T, device = some.dtype, slots.shape[0], _device("k" if some is k else "v", some)
        shape = (T, cache.heads, cache.dim)
        ka, kt, kh = _rows("k", k, shape, dtype, device) if k is not None else (None, 0, 0)
        va, vt, vh = _rows("v", v, shape, dtype, device) if v is not None else (None, 0, 0)
        _call(name, _of(cache, fmt, device), _array("slots", slots, torch.int64, (T,), device), ka, va, _code(dtype), T,
              kt, kh, vt, vh, _stream(stream, device))
    kv_read.__name__ = name
    kv_read.__doc__ = (f"Read the slots (int64 [T]) of a {fmt} cache back into k and v [T][H][D] (either may be None; "
                       "NaN rows for slots outside the cache).")
    return kv_read


# -- attention ------------------------------------------------------------------
def qmm_attn_decode_workspace(B: int, Hq: int, heads: int, dim: int, max_len: int, window: int = 0) -> int:
    """Bytes of the workspace of qmm_attn_decode_* (0 for sizes outside the limits)."""
    return _lib().qmm_attn_decode_workspace(B, Hq, heads, dim, max_len, window)


def attn_workspace(B: int, Hq: int, heads: int, dim: int, max_len: int, window: int = 0, device="cuda"):
    """A new workspace for qmm_attn_decode_*, enough for smaller batches, lengths and windows too."""
    size = qmm_attn_decode_workspace(B, Hq, heads, dim, max_len, window)
    if size == 0:
        raise ValueError(f"no attention of batch {B}, {Hq} on {heads} heads of {dim}, length {max_len}")
    return _t().empty(size, dtype=_torch.uint8, device=device)


def _attn_decode(fmt):
    name = "qmm_attn_decode_" + fmt

    def attn_decode(q, out, cache: KVCache, pages, lens, max_len: int, workspace, scale=None, softcap: float = 0.0,
                    window: int = 0, mask=None, lse=None, stream=None) -> None:
        torch, dtype, device = _t(), q.dtype, _device("q", q)
        B, Hq, _ = _three("q", q)
        shape = (B, Hq, cache.dim)
        qa, qt, qh = _rows("q", q, shape, dtype, device)
        oa, ot, oh = _rows("out", out, shape, dtype, device)
        width = pages.shape[-1]
        ma, ms = None, 0
        if mask is not None:
            ms = mask.shape[-1]
            ma = _array("mask", mask, torch.float32, (B, ms), device)
        size = workspace.numel()
        _call(name, _of(cache, fmt, device), qa, oa, _code(dtype),
              _array("pages", pages, torch.int32, (B, width), device), width,
              _array("lens", lens, torch.int32, (B,), device), B, Hq, max_len,
              1.0 / math.sqrt(cache.dim) if scale is None else scale, softcap, window, ma, ms,
              None if lse is None else _array("lse", lse, torch.float32, (B, Hq), device), qt, qh, ot, oh,
              _array("workspace", workspace, torch.uint8, (size,), device), size, _stream(stream, device))
    attn_decode.__name__ = name
    attn_decode.__doc__ = (
        f"Attention of one new token of each sequence over a {fmt} cache: q, out [B][Hq][D]; pages int32 "
        "[B][n] page numbers; lens int32 [B] positions seen, each at most max_len; scale defaults to "
        "1/sqrt(dim); softcap and window 0 = none; mask float32 [B][>= max_len] is added to the scores; lse "
        "float32 [B][Hq] receives the log-sum-exp.")
    return attn_decode


for _f in KV_FORMATS:
    globals().update({"qmm_kv_page_bytes_" + _f: _page_bytes(_f), "qmm_kv_write_" + _f: _kv_write(_f),
                      "qmm_rope_kv_write_" + _f: _rope_kv_write(_f), "qmm_kv_read_" + _f: _kv_read(_f),
                      "qmm_attn_decode_" + _f: _attn_decode(_f)})
KV_WRITE = {f: globals()["qmm_kv_write_" + f] for f in KV_FORMATS}
ROPE_KV_WRITE = {f: globals()["qmm_rope_kv_write_" + f] for f in KV_FORMATS}
KV_READ = {f: globals()["qmm_kv_read_" + f] for f in KV_FORMATS}
ATTN_DECODE = {f: globals()["qmm_attn_decode_" + f] for f in KV_FORMATS}
