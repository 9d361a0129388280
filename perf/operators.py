"""Workloads of the attention-side operators: rotary positions, the paged
key-value cache (written quantized, read back) and the attention of one new
token over it.

Each case is one pass through one operator, as a decode or prompt step calls
it.  `run` computes it in plain torch operations, or, where `own` is true, with
the framework's entry points; both take the same state, whose cache is in the
byte layout that the framework documents (include/qmm.h, "key-value cache").
"""
import math

import torch

own = False

DEVICE = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
CODE_BITS = {"f16": 16, "q8_0": 8, "q4_0": 4}


# ---------------------------------------------------------------------------
# The cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # One token of one sequence, deep in a long context: queries and keys of
        # 32 + 8 heads rotated in one call.  Nothing but latency.
        dict(name="rope_one_token", op="rope", tokens=1, heads=40, dim=128, rot=128, order="half", dtype="f16",
             inverse=False, start=100000),
        # A prompt of 4096 tokens, 32 query heads of 128: the ordinary rotation.
        dict(name="rope_prompt", op="rope", tokens=4096, heads=32, dim=128, rot=128, order="half", dtype="bf16",
             inverse=False, start=0),
        # The gradient of a partial, interleaved rotation (32 of 64 values) in
        # f32, at an odd token count.
        dict(name="rope_gradient", op="rope", tokens=2047, heads=14, dim=64, rot=32, order="interleaved", dtype="f32",
             inverse=True, start=5),
        # The decode step of 16 sequences: rotate q and k, quantize k and v into
        # the cache, and read the new rows back.
        dict(name="write_step_q8_0", op="write", fmt="q8_0", tokens=16, q_heads=32, heads=8, dim=128, page=64,
             rope=True, rot=128, order="half", dtype="f16"),
        # A prompt of 4096 tokens written with its rotation, then read back for
        # the prompt's own attention.
        dict(name="write_prompt_q8_0", op="write", fmt="q8_0", tokens=4096, q_heads=32, heads=8, dim=128, page=64,
             rope=True, rot=128, order="half", dtype="bf16"),
        # Keys without rotary positions into a 4-bit cache; two heads of 64, an
        # odd token count, small pages.
        dict(name="write_plain_q4_0", op="write", fmt="q4_0", tokens=777, q_heads=0, heads=2, dim=64, page=16,
             rope=False, rot=0, order="half", dtype="f32"),
        # A cached prefix of 8192 tokens read back as bf16.
        dict(name="read_prefix_q8_0", op="read", fmt="q8_0", tokens=8192, heads=8, dim=128, page=64, dtype="bf16"),
        # 32 heads of 96 from a 4-bit cache, as f32, with padding slots.
        dict(name="read_q4_0", op="read", fmt="q4_0", tokens=1001, heads=32, dim=96, page=32, dtype="f32"),
        # One short sequence, 14 query heads on 2 key heads of 64: latency.
        dict(name="attn_short_q8_0", op="attn", fmt="q8_0", batch=1, length=203, q_heads=14, heads=2, dim=64, page=16,
             dtype="f16", window=0, softcap=0.0, mask=False),
        # An ordinary serving batch: 16 ragged sequences of up to 4096 tokens.
        dict(name="attn_batch_q8_0", op="attn", fmt="q8_0", batch=16, length=4096, q_heads=32, heads=8, dim=128,
             page=64, dtype="bf16", window=0, softcap=0.0, mask=False),
        # One sequence of 131072 tokens in a 4-bit cache: all of the work lies
        # along the length.
        dict(name="attn_long_q4_0", op="attn", fmt="q4_0", batch=1, length=131072, q_heads=32, heads=8, dim=128,
             page=128, dtype="f16", window=0, softcap=0.0, mask=False),
        # The largest: one key head for each query head, unquantized cache, f32
        # activations, with the log-sum-exp that joins partial attentions.
        dict(name="attn_wide_f16", op="attn", fmt="f16", batch=32, length=4096, q_heads=32, heads=32, dim=128, page=64,
             dtype="f32", window=0, softcap=0.0, mask=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "attn", "attn", "attn"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op == "rope":
        dim = rng.choice([64, 96, 128, 192, 256])
        rot = rng.choice([dim, dim, dim // 2, dim // 4, 2 * rng.randint(1, dim // 2)])
        heads = _log_int(rng, 1, 64)
        return dict(op=op, tokens=_log_int(rng, 1, max(1, 2 ** 25 // (heads * dim))), heads=heads, dim=dim, rot=rot,
                    order=rng.choice(["half", "interleaved"]), dtype=dtype, inverse=rng.random() < 0.3,
                    start=_log_int(rng, 1, 1000000))
    fmt = rng.choice(["q8_0", "q8_0", "q4_0", "f16"])
    dim = rng.choice([64, 96, 128, 128, 192, 256])
    page = rng.choice([16, 32, 64, 128])
    heads = rng.choice([1, 2, 4, 8, 8, 16, 32])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16, 20])
    while group * heads > 128:
        group = max(1, group // 2)
    if op == "write":
        rope = rng.random() < 0.7
        most = max(1, 2 ** 24 // ((group + 2) * heads * dim))
        return dict(op=op, fmt=fmt, tokens=_log_int(rng, 1, most), q_heads=group * heads if rope else 0, heads=heads,
                    dim=dim, page=page, rope=rope, rot=rng.choice([dim, dim, dim // 2, 2 * rng.randint(1, dim // 2)])
                    if rope else 0, order=rng.choice(["half", "interleaved"]), dtype=dtype)
    if op == "read":
        return dict(op=op, fmt=fmt, tokens=_log_int(rng, 1, 2 ** 24 // (2 * heads * dim)), heads=heads, dim=dim,
                    page=page, dtype=dtype)
    batch = _log_int(rng, 1, 64)
    most = min(131072, 2 ** 28 // (batch * heads * dim), 2 ** 26 // (batch * group))
    return dict(op=op, fmt=fmt, batch=batch, length=_log_int(rng, 1, most), q_heads=group * heads, heads=heads,
                dim=dim, page=page, dtype=dtype, window=rng.choice([0, 0, 0, _log_int(rng, 1, 4096)]),
                softcap=rng.choice([0.0, 0.0, 30.0]), mask=rng.random() < 0.25)


def lengths(case):
    """Cache lengths of the sequences: the first has the whole length, the others
    are spread over the upper part of it (a batch in steady state)."""
    n = case["length"]
    return [n if b == 0 else 1 + int((n - 1) * math.sqrt((b * 0.6180339887498949) % 1.0))
            for b in range(case["batch"])]


# ---------------------------------------------------------------------------
# The cache's bytes: for each (page, head) the keys of all positions, then the
# values.  Sixteen positions at a time their codes lie as a 64-lane wave loads
# them: lane (g, r) of 4 x 16 holds, for the keys, of position r the values
# 32b + 8g + i in the order (b, i); for the values, of positions 4g + i the
# values 32b + 2r + e in the order (i, b, e).  A lane's bytes are cut into units
# of 16 (or the largest power of two that divides them), unit after unit.
# Quantized formats hold the rows' f16 block scales after the codes.
# ---------------------------------------------------------------------------
def _row_bytes(case):
    return case["dim"] * CODE_BITS[case["fmt"]] // 8


def _unit(case):
    return math.gcd(_row_bytes(case) // 4, 16)


def _side_bytes(case):
    """Bytes of one head's keys (or values) in one page."""
    scales = 0 if case["fmt"] == "f16" else case["dim"] // 32 * 2
    return case["page"] * (_row_bytes(case) + scales)


def _planes(pool, case):
    """Views of the pool: ((key codes, key scales), (value codes, value scales)); codes
    [pages][heads][page/16][unit][4][16][unit bytes] uint8, scales [pages][heads][page][dim/32] f16."""
    side, size, nb = _side_bytes(case), case["page"] * _row_bytes(case), case["dim"] // 32
    p = pool.view(-1, case["heads"], 2, side)

    def one(kv):
        codes = p[:, :, kv, :size].unflatten(-1, (case["page"] // 16, -1, 4, 16, _unit(case)))
        scales = None if case["fmt"] == "f16" else p[:, :, kv, size:].view(torch.float16).unflatten(-1, (-1, nb))
        return codes, scales
    return one(0), one(1)


def _numbers(raw, fmt, to):
    """What bytes (last dimension) stand for, before the scales."""
    if fmt == "f16":
        return raw.contiguous().view(torch.float16).to(to)
    if fmt == "q8_0":
        return raw.to(to) - 128
    return torch.stack([raw & 15, raw >> 4], -1).flatten(-2).to(to) - 8


def _bytes(x, fmt):
    """The inverse for codes from _quantized, or f32 values of an f16 cache."""
    if fmt == "f16":
        return x.half().contiguous().view(torch.uint8)
    x = x.to(torch.uint8)
    return x if fmt == "q8_0" else x[..., 0::2] | (x[..., 1::2] << 4)


def _scaled(x, scales):
    return x if scales is None else (x.unflatten(-1, (-1, 32)) * scales.to(x.dtype).unsqueeze(-1)).flatten(-2)


def _dense(codes, scales, values, case, to):
    """Whole pages as numbers: [...][page][dim] of codes [...][page/16][unit][4][16][unit bytes]."""
    nb = case["dim"] // 32
    lane = _numbers(codes.movedim(-4, -2).flatten(-2), case["fmt"], to)          # [..., page/16, 4, 16, 8 nb]
    if values:                                    # (g, r, i, b, e) -> (g, i, b, r, e)
        x = lane.unflatten(-1, (4, nb, 2)).movedim(-4, -2)
    else:                                         # (g, r, b, i) -> (r, b, g, i)
        x = lane.unflatten(-1, (nb, 8)).movedim(-4, -2)
    x = x.flatten(-3) if not values else x.flatten(-3).flatten(-3, -2)
    return _scaled(x.flatten(-3, -2), scales)


def _row_index(slots, values, case):
    """The index of the tokens' rows into a side's codes: keys [tokens][heads][unit][4][unit bytes],
    values [tokens][bytes of a position][heads][16]."""
    page, at = slots // case["page"], slots % case["page"]
    group, r = at // 16, at % 16
    if not values:
        return (page, slice(None), group, slice(None), slice(None), r)
    width, unit = _row_bytes(case) // 16, _unit(case)
    byte = (r % 4)[:, None] * width + torch.arange(width, device=slots.device)
    return (page[:, None], slice(None), group[:, None], byte // unit, (r // 4)[:, None], slice(None), byte % unit)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _freqs(rot, device):
    return 1e4 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / max(rot, 1))


def _fresh_pool(case, pages, gen):
    """A pool as a running server has it: every row written at some time."""
    n = pages * case["heads"] * 2 * _side_bytes(case)
    if case["fmt"] == "f16":
        return torch.randn(n // 2, generator=gen, device=DEVICE, dtype=torch.float16).view(torch.uint8)
    pool = torch.empty(n, dtype=torch.uint8, device=DEVICE)
    for codes, scales in _planes(pool, case):
        if case["fmt"] == "q8_0":     # codes spread like a normal value's, whose block maximum is 127
            codes.copy_((torch.randn(codes.shape, generator=gen, device=DEVICE, dtype=torch.float16) * 52 + 128)
                       .round_().clamp_(1, 255))
            scales.copy_(torch.rand(scales.shape, generator=gen, device=DEVICE) * 0.008 + 0.016)
        else:
            codes.copy_(torch.randint(0, 256, codes.shape, generator=gen, device=DEVICE, dtype=torch.uint8))
            scales.copy_((torch.rand(scales.shape, generator=gen, device=DEVICE) * 0.1 + 0.2)
                         * (torch.randint(0, 2, scales.shape, generator=gen, device=DEVICE) * 2 - 1))
    return pool


def _slots(case, pages, gen):
    """Slots of consecutive tokens in pages of any order."""
    order = torch.randperm(pages, generator=gen, device=DEVICE)
    at = torch.arange(case["tokens"], device=DEVICE)
    return order[at // case["page"]] * case["page"] + at % case["page"]


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(int(seed))
    dt = TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEVICE).to(dt)

    s = dict(case=case)
    op = case["op"]
    if op in ("rope", "write"):
        t = case["tokens"]
        s["freqs"] = _freqs(case["rot"], DEVICE)
    if op == "rope":
        s["x"] = normal(t, case["heads"], case["dim"])
        s["y"] = torch.empty_like(s["x"])
        s["positions"] = torch.arange(case["start"], case["start"] + t, device=DEVICE, dtype=torch.int32)
    if op == "write":
        hq, h, d = case["q_heads"], case["heads"], case["dim"]
        qkv = normal(t, hq + 2 * h, d)            # the fused projection's output: strided views
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + h], qkv[:, hq + h:]
        s["q_out"] = torch.empty(t, hq, d, dtype=dt, device=DEVICE)
        s["positions"] = torch.randint(0, 100000, (t,), generator=gen, device=DEVICE, dtype=torch.int32)
    if op in ("write", "read"):
        pages = -(-case["tokens"] // case["page"]) + 3
        s["pool"] = _fresh_pool(case, pages, gen)
        s["slots"] = _slots(case, pages, gen)
        if op == "read":
            s["slots"][case["tokens"] - 1 - case["tokens"] // 8:-1:3] = -1       # padding
        out = (case["tokens"], case["heads"], case["dim"])
        s["k_out"] = torch.empty(out, dtype=dt, device=DEVICE)
        s["v_out"] = torch.empty(out, dtype=dt, device=DEVICE)
    if op == "attn":
        lens = lengths(case)
        width = -(-case["length"] // case["page"])
        used = [-(-n // case["page"]) for n in lens]
        s["pool"] = _fresh_pool(case, sum(used) + 3, gen)
        order = torch.randperm(sum(used) + 3, generator=gen, device=DEVICE).to(torch.int32)
        table = torch.full((case["batch"], width), -1, dtype=torch.int32)        # padding past a sequence's pages
        inside = torch.arange(width)[None, :] < torch.tensor(used)[:, None]
        table = table.to(DEVICE)
        table[inside.to(DEVICE)] = order[:sum(used)]
        s["pages"], s["lens"] = table, torch.tensor(lens, dtype=torch.int32, device=DEVICE)
        s["q"] = normal(case["batch"], case["q_heads"], case["dim"]) * 1.5
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(case["batch"], case["q_heads"], dtype=torch.float32, device=DEVICE)
        s["scale"] = case["dim"] ** -0.5
        s["mask"] = None
        if case["mask"]:                          # added to the scores; a tenth of the positions is taken out
            m = torch.randn(case["batch"], case["length"], generator=gen, device=DEVICE)
            hidden = torch.rand(m.shape, generator=gen, device=DEVICE) < 0.1
            s["mask"] = m.masked_fill_(hidden, -math.inf)
    if own:                                       # what a program keeps: the cache's and the rotation's handles
        import matmul_quantize_q8_amd as qmm
        if op in ("rope", "write"):
            s["plan"] = qmm.RopePlan(s["freqs"], case["order"])
        if op != "rope":
            s["cache"] = qmm.KVCache(case["fmt"], s["pool"], case["page"], case["heads"], case["dim"])
        if op == "attn":
            s["workspace"] = qmm.attn_workspace(case["batch"], case["q_heads"], case["heads"], case["dim"],
                                                case["length"], case["window"])
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    return _run_own(s) if own else _PLAIN[s["case"]["op"]](s)


def _run_own(s):
    import matmul_quantize_q8_amd as qmm
    case = s["case"]
    op = case["op"]
    if op == "rope":
        qmm.qmm_rope(s["x"], s["y"], s["positions"], s["plan"], inverse=case["inverse"])
        return s["y"]
    if op == "write":
        if case["rope"]:
            qmm.ROPE_KV_WRITE[case["fmt"]](s["q"], s["q_out"], s["k"], s["v"], s["cache"], s["slots"],
                                           s["positions"], s["plan"])
        else:
            qmm.KV_WRITE[case["fmt"]](s["k"], s["v"], s["cache"], s["slots"])
    if op in ("write", "read"):
        qmm.KV_READ[case["fmt"]](s["cache"], s["slots"], s["k_out"], s["v_out"])
        return dict(q=s["q_out"] if op == "write" and case["rope"] else None, k=s["k_out"], v=s["v_out"])
    qmm.ATTN_DECODE[case["fmt"]](s["q"], s["out"], s["cache"], s["pages"], s["lens"], case["length"], s["workspace"],
                                 s["scale"], softcap=case["softcap"], window=case["window"], mask=s["mask"],
                                 lse=s["lse"])
    return dict(out=s["out"], lse=s["lse"])


def _rotated(x, positions, freqs, order, inverse=False):
    """x f32 [tokens][heads][dim], its first 2 * len(freqs) values rotated."""
    angle = positions.double()[:, None] * freqs
    c, s = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    if inverse:
        s = -s
    half = freqs.numel()
    part, rest = x[..., :2 * half], x[..., 2 * half:]
    if order == "half":
        a, b = part[..., :half], part[..., half:]
        return torch.cat([a * c - b * s, a * s + b * c, rest], -1)
    a, b = part[..., 0::2], part[..., 1::2]
    return torch.cat([torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2), rest], -1)


def _plain_rope(s):
    case = s["case"]
    return _rotated(s["x"].float(), s["positions"], s["freqs"], case["order"], case["inverse"]).to(s["x"].dtype)


def _quantized(x, fmt):
    """Codes (offset binary, f32) and f16 scales of f32 rows, a block of 32 at a time."""
    b = x.unflatten(-1, (-1, 32))
    mag = b.abs()
    top = mag.amax(-1, keepdim=True)
    if fmt == "q8_0":                             # d = top/127, code = round(x * (127/top))
        inv = torch.where(top > 0, torch.full_like(top, 127.0) / top, torch.zeros_like(top))
        return (torch.round(b * inv) + 128).flatten(-2), (top / 127.0).squeeze(-1).half()
    at = torch.arange(32, device=x.device).expand_as(b)
    first = torch.where(mag == top, at, 32).amin(-1, keepdim=True)               # ties: the lowest index
    d = b.gather(-1, first) / -8.0                # the value of largest magnitude keeps its sign
    code = torch.where(top > 0, torch.round(b / torch.where(top > 0, d, 1.0)), 0.0)
    return (code + 8).clamp(0, 15).flatten(-2), torch.where(top > 0, d, 0.0).squeeze(-1).half()


def _store(x, values, planes, slots, case):
    codes, scales = planes
    fmt, nb = case["fmt"], case["dim"] // 32
    if fmt != "f16":
        x, scales[slots // case["page"], :, slots % case["page"]] = _quantized(x, fmt)
    if values:                                    # (b, r, e) -> [tokens][byte of (b, e)][heads][r]
        rows = _bytes(x.unflatten(-1, (nb, 16, 2)).transpose(-3, -2).flatten(-2), fmt).permute(0, 3, 1, 2)
    else:                                         # (b, g, i) -> [tokens][heads][unit][g][unit bytes]
        rows = _bytes(x.unflatten(-1, (nb, 4, 8)).transpose(-3, -2).flatten(-2), fmt)
        rows = rows.unflatten(-1, (-1, _unit(case))).transpose(-3, -2)
    codes[_row_index(slots, values, case)] = rows


def _load(planes, values, slots, case, to):
    codes, scales = planes
    nb, valid = case["dim"] // 32, slots >= 0
    slots = slots.clamp(min=0)
    raw = codes[_row_index(slots, values, case)]
    if values:
        x = _numbers(raw.permute(0, 2, 3, 1), case["fmt"], torch.float32).unflatten(-1, (nb, 2))
    else:
        x = _numbers(raw.transpose(-3, -2).flatten(-2), case["fmt"], torch.float32).unflatten(-1, (nb, 8))
    x = x.transpose(-3, -2).flatten(-3)
    x = _scaled(x, None if scales is None else scales[slots // case["page"], :, slots % case["page"]])
    return torch.where(valid[:, None, None], x, math.nan).to(to)


def _plain_read(s):
    case, dt = s["case"], s["k_out"].dtype
    kp, vp = _planes(s["pool"], case)
    return dict(q=None, k=_load(kp, False, s["slots"], case, dt), v=_load(vp, True, s["slots"], case, dt))


def _plain_write(s):
    case = s["case"]
    k, q = s["k"].float(), None
    if case["rope"]:
        k = _rotated(k, s["positions"], s["freqs"], case["order"])
        q = _rotated(s["q"].float(), s["positions"], s["freqs"], case["order"]).to(s["q"].dtype)
    kp, vp = _planes(s["pool"], case)
    _store(k, False, kp, s["slots"], case)
    _store(s["v"].float(), True, vp, s["slots"], case)
    return dict(_plain_read(s), q=q)


def _plain_attn(s):
    case = s["case"]
    b, h, d = case["batch"], case["heads"], case["dim"]
    table = s["pages"].clamp(min=0).long()

    def dense(planes, values):                    # [batch][heads][positions][dim]
        codes, scales = planes
        x = _dense(codes[table], None if scales is None else scales[table], values, case, torch.float32)
        return x.transpose(1, 2).flatten(2, 3)
    kp, vp = _planes(s["pool"], case)
    k, v = dense(kp, False), dense(vp, True)
    q = s["q"].float().view(b, h, -1, d)
    score = torch.matmul(q, k.transpose(-1, -2).contiguous()) * s["scale"]
    if case["softcap"]:
        score = torch.tanh(score / case["softcap"]) * case["softcap"]
    at, n = torch.arange(k.shape[2], device=k.device)[None, :], s["lens"][:, None]
    seen = at < n
    if case["window"]:
        seen = seen & (at >= n - case["window"])
    if s["mask"] is not None:
        extra = torch.nn.functional.pad(s["mask"], (0, k.shape[2] - case["length"]))
        seen = seen & (extra > -math.inf)
        score = score + extra[:, None, None, :]
    score = score.masked_fill(~seen[:, None, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, torch.where(seen[:, None, :, None], v, 0.0))
    out = torch.where(total > 0, out / total, 0.0)
    lse = (top + torch.log(total)).squeeze(-1)
    return dict(out=out.reshape(s["q"].shape).to(s["q"].dtype), lse=lse.reshape(b, -1))


_PLAIN = {"rope": _plain_rope, "write": _plain_write, "read": _plain_read, "attn": _plain_attn}


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    size = {"f32": 4, "f16": 2, "bf16": 2}[case["dtype"]]
    op = case["op"]
    if op == "rope":
        n = case["tokens"] * case["heads"] * case["dim"]
        return dict(bytes=2 * n * size + case["tokens"] * 4 + case["rot"] * 4,
                    flops=3 * case["tokens"] * case["heads"] * case["rot"])
    row = 2 * (_side_bytes(case) // case["page"])                      # a token's keys and values of one head
    if op in ("write", "read"):
        t, kv = case["tokens"], case["tokens"] * case["heads"] * case["dim"] * 2
        read = t * case["heads"] * row + kv * size + t * 8             # cache in, rows out
        if op == "read":
            return dict(bytes=read, flops=kv)
        q = t * case["q_heads"] * case["dim"]
        return dict(bytes=read + (2 * q + kv) * size + t * case["heads"] * row + t * 12 + case["rot"] * 4,
                    flops=3 * t * (case["q_heads"] + case["heads"]) * case["rot"] + 4 * kv)
    seen = sum(min(n, case["window"]) if case["window"] else n for n in lengths(case))
    qo = case["batch"] * case["q_heads"] * case["dim"]
    return dict(bytes=seen * case["heads"] * row + 2 * qo * size + case["batch"] * case["q_heads"] * 4
                + 4 * -(-seen // case["page"]) + (4 * seen if case["mask"] else 0),
                flops=4 * seen * case["q_heads"] * case["dim"])


# ---------------------------------------------------------------------------
# The same from the definitions, in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return _EXACT[case["op"]](s)


def _turned64(x, s, sign):
    """Each pair (a, b) as a complex number times e^(i * angle)."""
    case = s["case"]
    rot, x = case["rot"], x.double()
    if rot == 0:
        return x
    first = torch.arange(rot // 2, device=x.device)
    i, j = (first, first + rot // 2) if case["order"] == "half" else (2 * first, 2 * first + 1)
    w = torch.polar(torch.ones((), dtype=torch.float64, device=x.device),
                    sign * torch.outer(s["positions"].double(), s["freqs"]))
    z = torch.complex(x[..., i], x[..., j]) * w[:, None, :]
    y = x.clone()
    y[..., i], y[..., j] = z.real, z.imag
    return y


def _exact_rope(s):
    return _turned64(s["x"], s, -1.0 if s["case"]["inverse"] else 1.0)


def _rows64(pool, case, slots, values):
    """Rows of the cache at `slots`, every head: f64 [slots][heads][dim], from the bytes' offsets."""
    p, h, d, fmt = case["page"], case["heads"], case["dim"], case["fmt"]
    side, rb, unit = _side_bytes(case), _row_bytes(case), _unit(case)
    n, head = torch.arange(d, device=slots.device), torch.arange(h, device=slots.device)
    block, rest = n // 32, n % 32
    base = ((slots // p)[:, None] * h + head) * 2 * side + (side if values else 0)
    at = slots % p
    t = (at % 16)[:, None]
    if values:
        g, r, j = t // 4, rest // 2, (t % 4) * (d // 16) + 2 * block + rest % 2
    else:
        g, r, j = rest // 8, t, 0 * t + 8 * block + rest % 8
    byte = j * CODE_BITS[fmt] // 8
    byte = (at // 16)[:, None] * 16 * rb + ((byte // unit * 4 + g) * 16 + r) * unit + byte % unit
    byte = base[..., None] + byte[:, None, :]
    if fmt == "f16":
        return pool.view(torch.float16)[byte // 2].double()
    scale = pool.view(torch.float16)[(base[..., None] + p * rb + at[:, None, None] * (d // 16) + 2 * block) // 2]
    if fmt == "q8_0":
        return (pool[byte].double() - 128) * scale.double()
    return ((pool[byte].int() >> (4 * (j % 2)).int()[:, None, :] & 15).double() - 8) * scale.double()


def _exact_read(s):
    case = s["case"]
    slots = s["slots"].clamp(min=0)
    gone = (s["slots"] < 0)[:, None, None]
    return dict(q=None, k=_rows64(s["pool"], case, slots, False).masked_fill(gone, math.nan),
                v=_rows64(s["pool"], case, slots, True).masked_fill(gone, math.nan))


def _through64(x, fmt):
    """What is left of f64 rows after the cache's format."""
    if fmt == "f16":
        return x.half().double()
    b = x.reshape(*x.shape[:-1], -1, 32)
    low, high = b.amin(-1, keepdim=True), b.amax(-1, keepdim=True)
    top = torch.maximum(high, -low)
    if fmt == "q8_0":
        code = torch.round(b * 127 / top.clamp(min=1e-300))
        y = code * (top / 127).half().double()
    else:
        # equal magnitudes of both signs: the earlier one sets the sign
        pos = torch.arange(32, device=x.device).double()
        up, down = (torch.where(b == e, pos, 99.0).amin(-1, keepdim=True) for e in (top, -top))
        d = torch.where(up < down, top, -top) / -8
        code = torch.round(b / torch.where(d == 0, 1.0, d)).clamp(-8, 7)
        y = code * d.half().double()
    return y.reshape(x.shape)


def _exact_write(s):
    case = s["case"]
    k = _turned64(s["k"], s, 1.0)
    return dict(q=_turned64(s["q"], s, 1.0) if case["rope"] else None, k=_through64(k, case["fmt"]),
                v=_through64(s["v"].double(), case["fmt"]))


def _exact_attn(s):
    case = s["case"]
    outs, lses = [], []
    for b, n in enumerate(lengths(case)):
        lo = max(0, n - case["window"]) if case["window"] else 0
        pos = torch.arange(lo, n, device=s["q"].device)
        extra = None
        if s["mask"] is not None:
            extra = s["mask"][b, lo:n].double()
            pos, extra = pos[extra > -math.inf], extra[extra > -math.inf]
        q = s["q"][b].double().reshape(case["heads"], -1, case["dim"])
        if pos.numel() == 0:
            outs.append(torch.zeros_like(q).flatten(0, 1))
            lses.append(torch.full((case["q_heads"],), -math.inf, dtype=torch.float64, device=q.device))
            continue
        slots = s["pages"][b].long()[pos // case["page"]] * case["page"] + pos % case["page"]
        parts = []
        for values in (False, True):              # a slice of positions at a time: the offsets are 64-bit
            parts.append(torch.cat([_rows64(s["pool"], case, c, values) for c in slots.split(8192)]).transpose(0, 1))
        z = torch.bmm(q, parts[0].transpose(1, 2).contiguous()) * s["scale"]
        if case["softcap"]:
            z = case["softcap"] * torch.tanh(z / case["softcap"])
        if extra is not None:
            z = z + extra
        lses.append(torch.logsumexp(z, -1).flatten())
        outs.append(torch.bmm(torch.softmax(z, -1), parts[1].contiguous()).flatten(0, 1))
    return dict(out=torch.stack(outs), lse=torch.stack(lses))


_EXACT = {"rope": _exact_rope, "write": _exact_write, "read": _exact_read, "attn": _exact_attn}
