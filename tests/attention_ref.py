"""Plain numpy forms of the attention operators, in 64 bits, from the formulas
and the byte layout that include/qmm.h states."""
import numpy as np

BITS = {"f16": 16, "q8_0": 8, "q4_0": 4}


def side_bytes(fmt, page, dim):
    return page * dim * BITS[fmt] // 8 + (0 if fmt == "f16" else page * dim // 32 * 2)


def code_places(fmt, dim, t, values):
    """Byte offsets in a side (int64 [dim]) of the codes of position t's row, and
    for each value whether it is a byte's high half."""
    n = np.arange(dim)
    b, rest, nb = n // 32, n % 32, dim // 32
    if values:
        g, r, number = np.full(dim, t % 16 // 4), rest // 2, t % 4 * 2 * nb + b * 2 + rest % 2
    else:
        g, r, number = rest // 8, np.full(dim, t % 16), b * 8 + rest % 8
    lane_bytes = dim // 4 * BITS[fmt] // 8
    unit = 16
    while lane_bytes % unit:
        unit //= 2
    byte = number * BITS[fmt] // 8
    at = t // 16 * 64 * lane_bytes + ((byte // unit * 4 + g) * 16 + r) * unit + byte % unit
    return at.astype(np.int64), (number % 2 == 1) & (fmt == "q4_0")


def read_row(pool, fmt, page, heads, dim, slot, head, values):
    """f64 [dim]: what the pool's bytes (uint8) hold at a slot."""
    side = side_bytes(fmt, page, dim)
    base = (slot // page * heads + head) * 2 * side + (side if values else 0)
    at, high = code_places(fmt, dim, slot % page, values)
    at = at + base
    if fmt == "f16":
        raw = pool[at].astype(np.uint16) | pool[at + 1].astype(np.uint16) << 8
        return raw.view(np.float16).astype(np.float64)
    scale_at = base + page * dim * BITS[fmt] // 8 + (slot % page) * dim // 32 * 2
    d = pool[scale_at:scale_at + dim // 32 * 2].copy().view(np.float16).astype(np.float64)
    code = pool[at].astype(np.int64)
    code = code - 128 if fmt == "q8_0" else np.where(high, code >> 4, code & 15) - 8
    return code * np.repeat(d, 32)


def read_rows(pool, fmt, page, heads, dim, slots, values):
    return np.stack([[read_row(pool, fmt, page, heads, dim, int(s), h, values) for h in range(heads)] for s in slots])


def through_cache(x, fmt, orc):
    """f64 rows that f32 rows x [..., dim] become in the cache (the weight
    formats' quantizers: the oracle's)."""
    x = np.ascontiguousarray(x, dtype=np.float32)
    if fmt == "f16":
        with np.errstate(over="ignore"):
            return x.astype(np.float16).astype(np.float64)
    rows = x.reshape(-1, x.shape[-1])
    raw = (orc.quantize_q8_0(rows) if fmt == "q8_0" else orc.quantize_q4_0_w(rows)).reshape(rows.shape[0], -1)
    blocks = raw.reshape(rows.shape[0], -1, 34 if fmt == "q8_0" else 18)
    d = blocks[..., :2].copy().view(np.float16).astype(np.float64)
    qs = blocks[..., 2:]
    if fmt == "q8_0":
        code = qs.copy().view(np.int8).astype(np.float64)
    else:
        code = np.concatenate([qs & 15, qs >> 4], -1).astype(np.float64) - 8
    return (code * d).reshape(x.shape)


def rotated(x, positions, freqs, order, mscale=1.0, inverse=False):
    """f32 rows x [T][H][D] rotated as stated: f64 angles, one rounding of each
    cosine and sine, f32 products and sums."""
    rot = 2 * len(freqs)
    ang = positions.astype(np.float64)[:, None] * freqs
    c = (np.cos(ang) * np.float64(np.float32(mscale))).astype(np.float32)[:, None]
    s = (np.sin(ang) * np.float64(np.float32(mscale))).astype(np.float32)[:, None]
    if inverse:
        s = -s
    i = np.arange(rot // 2)
    ia, ib = (i, i + rot // 2) if order == "half" else (2 * i, 2 * i + 1)
    y = x.astype(np.float32).copy()
    a, b = y[..., ia].copy(), y[..., ib].copy()
    y[..., ia] = a * c - b * s
    y[..., ib] = a * s + b * c
    return y


def attention(q, keys, vals, scale, softcap=0.0, mask=None):
    """One sequence, f64: q [Hq][D], keys and vals [n][H][D] of the positions
    that are seen, mask [n].  Returns out, lse and a bound's ingredients: the
    largest sum of |q||k| and the weighted sum of |v|."""
    Hq, D = q.shape
    n, H, _ = keys.shape
    out, lse = np.zeros((Hq, D)), np.full(Hq, -np.inf)
    reach, mag = np.zeros(Hq), np.zeros((Hq, D))
    if n == 0:
        return out, lse, reach, mag
    for h in range(Hq):
        k, v = keys[:, h // (Hq // H)], vals[:, h // (Hq // H)]
        z = k @ q[h] * scale
        if softcap:
            z = softcap * np.tanh(z / softcap)
        if mask is not None:
            z = z + mask
        m = z.max()
        p = np.exp(z - m)
        out[h], lse[h] = p @ v / p.sum(), m + np.log(p.sum())
        reach[h] = (np.abs(k) @ np.abs(q[h])).max() * abs(scale)
        mag[h] = p @ np.abs(v) / p.sum()
    return out, lse, reach, mag
