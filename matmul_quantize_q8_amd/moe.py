"""Binding of the mixture-of-experts operators: residual + norm and gated
activation with quantized output, routing, the experts' products and their
weighted sum (include/qmm.h).

Arguments are torch tensors on the current device.  Rows are [tokens][values] of
float32, float16 or bfloat16, the values of a row contiguous, any row stride;
quantized rows are uint8 [rows][row_bytes(format, K)], contiguous.  Shapes, types
and devices are checked here (ValueError); sizes, strides and alignment by the
library (QmmError).  Nothing is copied and nothing is allocated by a call, except
by the helpers that say so.
"""
from __future__ import annotations

import ctypes

from . import attention as _a
from .attention import _array, _code, _device, _elsewhere, _t

ACT_FORMATS = ("q8_0", "q8_k")
_VALUES = {"q8_0": 32, "q8_k": 256}
_BYTES = {"q8_0": 34, "q8_k": 292}
# (values, bytes) of a weight block and the activations it takes.
_WEIGHTS = {"q4_0": (32, 18, "q8_0"), "q8_0": (32, 34, "q8_0"), "q4_1": (32, 20, "q8_0"), "q5_0": (32, 22, "q8_0"),
            "q5_1": (32, 24, "q8_0"), "q2_k": (256, 84, "q8_k"), "q4_k": (256, 144, "q8_k"), "q6_k": (256, 210, "q8_k")}
GLU_ACTS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}
ROUTE_SCORES = {"softmax": 0, "sigmoid": 1}

EXPORTS = tuple(["qmm_route", "qmm_experts_plan_bytes", "qmm_experts_plan", "qmm_experts_combine"] +
                [p + f for p in ("qmm_rms_norm_", "qmm_glu_") for f in ACT_FORMATS] +
                ["qmm_experts_matmul_" + f for f in _WEIGHTS])


def declare(L) -> None:
    """Argument types of the mixture-of-experts entry points of libqmm.so."""
    P, I64, I32, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    sig = {"qmm_route": [P, I32, P, P, P, I64, I64, I64, I64, I32, I64, I64, I64, I32, F, P],
           "qmm_experts_plan": [P, P, I64, I64, I64, I64, P],
           "qmm_experts_combine": [P, P, P, P, I32] + 5 * [I64] + [P]}
    for f in ACT_FORMATS:
        sig["qmm_rms_norm_" + f] = [P, P, P, P, P, P, I32] + 6 * [I64] + [F, F, P]
        sig["qmm_glu_" + f] = [P, P, P, I32, I32] + 4 * [I64] + [P]
    for f in _WEIGHTS:
        sig["qmm_experts_matmul_" + f] = [P, I64, P, I64, P, P, I64, P] + 5 * [I64] + [P]
    for name, args in sig.items():
        getattr(L, name).argtypes = args
        getattr(L, name).restype = ctypes.c_int
    L.qmm_experts_plan_bytes.argtypes = [I64] * 3
    L.qmm_experts_plan_bytes.restype = I64


# Set by the package: its call, the stream of a call on a device and its library access.
_call = _stream = _lib = None


def bind(call, stream, lib) -> None:
    global _call, _stream, _lib
    _call, _stream, _lib = call, stream, lib


def _two(name, t):
    """The shape of rows."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name}: want rows [tokens][values], got {tuple(shape)}")
    return shape


def _rows(name, t, shape, dtype, device):
    """(address, stride) of rows of that shape and type."""
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name}: want {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    stride, one = t.stride()
    if one != 1 and shape[1] > 1:
        raise ValueError(f"{name}: the values of a row have to be contiguous")
    if t.get_device() != device:
        raise _elsewhere(name, t.get_device(), device)
    return t.data_ptr(), stride


def _blocks(fmt, K):
    """Bytes of a row of K values (K that are no whole blocks are the library's to refuse)."""
    return K // _VALUES[fmt] * _BYTES[fmt]


# -- norm and gated activation -----------------------------------------------------
def _rms_norm(fmt):
    name = "qmm_rms_norm_" + fmt

    def rms_norm(x, weight, xq, residual=None, sum=None, y=None, eps: float = 1e-6, weight_offset: float = 0.0,
                 stream=None) -> None:
        torch, dtype, device = _t(), x.dtype, _device("x", x)
        shape = _two("x", x)
        xa, xs = _rows("x", x, shape, dtype, device)
        ra, rs = (None, 0) if residual is None else _rows("residual", residual, shape, dtype, device)
        sa, ss = (None, 0) if sum is None else _rows("sum", sum, shape, dtype, device)
        ya, ys = (None, 0) if y is None else _rows("y", y, shape, dtype, device)
        T, K = shape
        _call(name, xa, ra, sa, None if weight is None else _array("weight", weight, torch.float32, (K,), device),
              _array("xq", xq, torch.uint8, (T, _blocks(fmt, K)), device), ya, _code(dtype), T, K, xs, rs, ss, ys, eps,
              weight_offset, _stream(stream, device))
    rms_norm.__name__ = name
    rms_norm.__doc__ = (
        f"xq = {fmt.upper()} blocks of y = s (weight_offset + weight) / sqrt(mean(s^2) + eps), s = x + residual, of rows "
        "[T][K]; sum and y, where given, receive s and y.  weight: float32 [K], or None for ones.")
    return rms_norm


def _glu(fmt):
    name = "qmm_glu_" + fmt

    def glu(gate, up, xq, act: str = "silu", stream=None) -> None:
        torch, dtype, device = _t(), gate.dtype, _device("gate", gate)
        shape = _two("gate", gate)
        code = GLU_ACTS.get(act)
        if code is None:
            raise ValueError(f"act is one of {', '.join(GLU_ACTS)}, not {act!r}")
        ga, gs = _rows("gate", gate, shape, dtype, device)
        ua, us = _rows("up", up, shape, dtype, device)
        rows, F = shape
        _call(name, ga, ua, _array("xq", xq, torch.uint8, (rows, _blocks(fmt, F)), device), _code(dtype), code, rows, F,
              gs, us, _stream(stream, device))
    glu.__name__ = name
    glu.__doc__ = (f"xq = {fmt.upper()} blocks of act(gate) * up, rows [rows][F]; act is silu, gelu or gelu_tanh.")
    return glu


# -- routing -------------------------------------------------------------------------
def qmm_route(logits, ids, weights, score: str = "softmax", bias=None, groups: int = 1, groups_kept: int = 1,
              group_top: int = 1, renorm: bool = True, scale: float = 1.0, stream=None) -> None:
    """The top experts of each token: ids int32 [T][top_k] and weights float32
    [T][top_k] from logits [T][E], scored by "softmax" or "sigmoid", chosen with
    the bias (float32 [E]) added, among the groups_kept best of `groups` groups."""
    torch, dtype, device = _t(), logits.dtype, _device("logits", logits)
    T, E = _two("logits", logits)
    code = ROUTE_SCORES.get(score)
    if code is None:
        raise ValueError(f"score is one of {', '.join(ROUTE_SCORES)}, not {score!r}")
    la, ls = _rows("logits", logits, (T, E), dtype, device)
    shape = (T, _two("ids", ids)[1])
    _call("qmm_route", la, _code(dtype), None if bias is None else _array("bias", bias, torch.float32, (E,), device),
          _array("ids", ids, torch.int32, shape, device), _array("weights", weights, torch.float32, shape, device), T, E,
          ls, shape[1], code, groups, groups_kept, group_top, 1 if renorm else 0, scale, _stream(stream, device))


# -- experts ---------------------------------------------------------------------------
def qmm_experts_plan_bytes(T: int, top_k: int, E: int) -> int:
    """Bytes of the plan of up to T tokens with top_k of E experts (0 for sizes outside the limits)."""
    return _lib().qmm_experts_plan_bytes(T, top_k, E)


def experts_plan(T: int, top_k: int, E: int, device="cuda"):
    """A new buffer for qmm_experts_plan, for up to T tokens."""
    size = qmm_experts_plan_bytes(T, top_k, E)
    if size == 0:
        raise ValueError(f"no plan of {T} tokens with {top_k} of {E} experts")
    return _t().empty(size, dtype=_a._torch.uint8, device=device)


def qmm_experts_plan(ids, E: int, plan, stream=None) -> None:
    """Sort the pairs of ids (int32 [T][top_k]) by expert into the plan (uint8)."""
    torch, device = _t(), _device("ids", ids)
    T, top = _two("ids", ids)
    size = plan.numel()
    _call("qmm_experts_plan", _array("ids", ids, torch.int32, (T, top), device),
          _array("plan", plan, torch.uint8, (size,), device), size, T, top, E, _stream(stream, device))


def _experts_matmul(fmt):
    name = "qmm_experts_matmul_" + fmt
    values, size, act = _WEIGHTS[fmt]

    def experts_matmul(w, xq, ids, plan, y, stream=None) -> None:
        torch, device = _t(), _device("w", w)
        if len(w.shape) != 3 or w.dtype != torch.uint8:
            raise ValueError(f"w: want uint8 [experts][rows][row bytes], got {w.dtype} {tuple(w.shape)}")
        E, N, rb = w.shape
        K = rb // size * values
        expert, row, one = w.stride()
        if rb % size or one != 1 or (row != rb and N > 1):
            raise ValueError(f"w: the rows of an expert have to be contiguous blocks of {size} bytes")
        T, top = _two("ids", ids)
        rows = xq.shape[0]
        shape = (T, top, N) if len(y.shape) == 3 else (T * top, N)
        bytes_ = plan.numel()
        _call(name, w.data_ptr(), expert if E > 1 else (N * rb + 15) // 16 * 16,       # one expert: any stride
              _array("xq", xq, torch.uint8, (rows, _blocks(act, K)), device), rows,
              _array("ids", ids, torch.int32, (T, top), device), _array("plan", plan, torch.uint8, (bytes_,), device),
              bytes_, _array("y", y, torch.float32, shape, device), T, top, E, N, K, _stream(stream, device))
    experts_matmul.__name__ = name
    experts_matmul.__doc__ = (
        f"y [T][top_k][N] (or [T top_k][N], float32): the row of xq of each token (T rows) or pair (T top_k rows) times its "
        f"expert's matrix.  w: uint8 [E][N][row_bytes({fmt!r}, K)], matrices at any stride of whole 16 bytes; ids int32 "
        "[T][top_k] and the plan made of them; pairs without an expert get zeros.")
    return experts_matmul


def qmm_experts_combine(y, weights, out, residual=None, stream=None) -> None:
    """out [T][N] = residual + the sum over a token's experts of weights [T][top_k] times y [T][top_k][N]."""
    torch, dtype, device = _t(), out.dtype, _device("out", out)
    shape = _two("out", out)
    T, N = shape
    top = _two("weights", weights)[1]
    oa, os = _rows("out", out, shape, dtype, device)
    ra, rs = (None, 0) if residual is None else _rows("residual", residual, shape, dtype, device)
    _call("qmm_experts_combine", _array("y", y, torch.float32, (T, top, N) if len(y.shape) == 3 else (T * top, N), device),
          _array("weights", weights, torch.float32, (T, top), device), ra, oa, _code(dtype), T, top, N, rs, os,
          _stream(stream, device))


for _f in ACT_FORMATS:
    globals().update({"qmm_rms_norm_" + _f: _rms_norm(_f), "qmm_glu_" + _f: _glu(_f)})
for _f in _WEIGHTS:
    globals()["qmm_experts_matmul_" + _f] = _experts_matmul(_f)
RMS_NORM = {f: globals()["qmm_rms_norm_" + f] for f in ACT_FORMATS}
GLU = {f: globals()["qmm_glu_" + f] for f in ACT_FORMATS}
EXPERTS_MATMUL = {f: globals()["qmm_experts_matmul_" + f] for f in _WEIGHTS}
