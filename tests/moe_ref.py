"""Plain 64-bit forms of the mixture-of-experts operators (numpy)."""
import math

import numpy as np

VALUES = {"q8_0": 32, "q8_k": 256}
STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}       # half a step, relative


def norm(s, weight, eps, offset=0.0):
    """y of rows s, in 64 bits."""
    s = s.astype(np.float64)
    w = offset + (np.ones(s.shape[1]) if weight is None else weight.astype(np.float64))
    return s / np.sqrt((s * s).mean(1, keepdims=True) + eps) * w


def activation(g, act):
    g = g.astype(np.float64)
    with np.errstate(over="ignore"):
        if act == "silu":
            return g / (1 + np.exp(-g))
        if act == "gelu":
            return 0.5 * g * np.vectorize(math.erfc)(-g / math.sqrt(2))
        return g / (1 + np.exp(-2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))


def decoded(xq, fmt):
    """(values, scales) of packed rows [rows][bytes]: f64 [rows][K] and [rows][blocks]."""
    if fmt == "q8_0":
        b = xq.reshape(xq.shape[0], -1, 34)
        d, q = np.ascontiguousarray(b[..., :2]).view(np.float16)[..., 0], np.ascontiguousarray(b[..., 2:]).view(np.int8)
    else:
        b = xq.reshape(xq.shape[0], -1, 292)
        d = np.ascontiguousarray(b[..., :4]).view(np.float32)[..., 0]
        q = np.ascontiguousarray(b[..., 4:260]).view(np.int8)
    d = d.astype(np.float64)
    return (q.astype(np.float64) * d[..., None]).reshape(xq.shape[0], -1), d


def route(logits, top, score="softmax", bias=None, groups=1, kept=1, group_top=1, renorm=True, scale=1.0):
    """(ids, weights) by the definition, a token at a time; scores are exact enough that ties are ties of the
    formula: without a bias the order is that of the logits."""
    T, E = logits.shape
    ids, weights = np.full((T, top), -1, np.int32), np.zeros((T, top))
    for t in range(T):
        x = logits[t].astype(np.float64)
        can = x != -math.inf
        with np.errstate(over="ignore", invalid="ignore"):
            if score == "softmax":
                m = np.max(x[can]) if can.any() and not np.isnan(x).any() else math.nan
                p = np.where(can, np.exp(x - m), 0)
                p = p / math.fsum(p) if not np.isnan(p).any() else p * math.nan
            else:
                p = 1 / (1 + np.exp(-x))
        c = p if bias is None else p + bias.astype(np.float64)
        can &= ~np.isneginf(c)
        order = x if bias is None else c

        def key(v):                                  # NaN above all
            return (1, 0.0) if v != v else (0, v)
        allowed = list(range(E))
        if groups > 1:
            per, ranked = E // groups, []
            for g in range(groups):
                best = sorted((c[e] for e in range(g * per, (g + 1) * per) if can[e]), key=key, reverse=True)[:group_top]
                if best:
                    ranked.append((key(sum(best)), -g))
            keep = {-g for _, g in sorted(ranked, reverse=True)[:kept]}
            allowed = [e for e in allowed if e // per in keep]
        chosen = sorted((e for e in allowed if can[e]), key=lambda e: (key(order[e]), -e), reverse=True)[:top]
        w = p[chosen]
        if renorm and chosen:
            xs = x[chosen]
            if not np.isnan(xs).any():               # shares, whatever the scores' size
                m = xs.max()
                if score == "softmax":
                    w = np.exp(xs - m)
                elif m < 0:
                    w = np.exp(xs - m) / (1 + np.exp(xs))
            w = w / w.sum()
        ids[t, :len(chosen)], weights[t, :len(chosen)] = chosen, w * scale
    return ids, weights


def experts(orc, fmt, w, xq, ids, N, K, per_pair):
    """(y, mag) [T][top][N]: exact products and the sum of their terms' magnitudes; w: a list of packed matrices."""
    T, top = ids.shape
    y, mag = np.zeros((T, top, N)), np.zeros((T, top, N))
    for e in range(len(w)):
        t, j = np.nonzero(ids == e)
        if t.size:
            rows = np.ascontiguousarray(xq[t * top + j] if per_pair else xq[t])
            r = orc.matmul(fmt, w[e], rows, t.size, N, K, threads=4, want=("y64", "mag"))
            y[t, j], mag[t, j] = r["y64"], r["mag"]
    return y, mag
