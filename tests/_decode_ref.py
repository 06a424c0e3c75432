"""Plain 64-bit references of the operators in include/mnb_decode.h (numpy; nothing of the package)."""
from __future__ import annotations

import numpy as np

import _ops_ref as ref


def places(lengths, starts):
    """(sequence, position) of every row of the sequences; starts None: one row each."""
    out = []
    for b, total in enumerate(lengths):
        n = 1 if starts is None else starts[b + 1] - starts[b]
        out += [(b, total - n + i) for i in range(n)]
    return out


def table(n, rot, base=10000.0):
    inv = base ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    a = np.arange(n, dtype=np.float64)[:, None] * inv
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def norm_rotate(x, weight, eps, rows, interleaved):
    """x [T, H, D], rows [T, rot] of the table (or None)."""
    x = np.asarray(x, np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    if rows is None or rows.shape[1] == 0:
        return x
    rot = rows.shape[1]
    cos, sin = rows[:, None, :rot // 2].astype(np.float64), rows[:, None, rot // 2:].astype(np.float64)
    y = x.copy()
    a = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    b = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    y[..., a], y[..., b] = x[..., a] * cos - x[..., b] * sin, x[..., b] * cos + x[..., a] * sin
    return y


def fp4(x):
    """The values that x [..., D] has as MX FP4 (NaN blocks as NaN)."""
    flat = np.asarray(x, np.float64).reshape(-1, x.shape[-1])
    q, s = ref.quantize(flat, 0)
    return (q * np.repeat(ref.scale_values(s), 32, -1)).reshape(x.shape)


def attention(q, k, v, first, scale, window=0):
    """q [n, Hq, D] at positions first.., k and v [total, Hkv, D]: (y, sum of |p v|) in 64 bits."""
    n, hq, d = q.shape
    total, hkv, _ = k.shape
    y, size = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    for i in range(n):
        p = first + i
        lo = max(0, p - window + 1) if window else 0
        if p < 0:
            continue
        for h in range(hq):
            kh, vh = k[lo:p + 1, h // (hq // hkv)], v[lo:p + 1, h // (hq // hkv)]
            with np.errstate(invalid="ignore", over="ignore"):
                s = (kh @ q[i, h]) * scale
                e = np.exp(s - s.max())
                e = e / e.sum()
                y[i, h] = (e[:, None] * vh).sum(0)
                size[i, h] = (e[:, None] * np.abs(vh)).sum(0)
    return y, size


def sample(x, u, temperature, top_k, top_p, min_p):
    """One row: the token, by sorting; ordinary rows."""
    x = np.asarray(x, np.float64)
    order = np.argsort(-x, kind="stable")
    if temperature == 0:
        return int(order[0])
    if top_k > 0:
        order = order[:top_k]
    p = np.exp((x[order] - x[order[0]]) / temperature)
    if top_p < 1:
        before = np.cumsum(p) - p
        keep = before < top_p * p.sum()
        keep[0] = True
        order, p = order[keep], p[keep]
    keep = p >= min(min_p, 1.0)
    order, p = order[keep], p[keep]
    index = np.sort(order)
    w = np.zeros(len(x))
    w[order] = p
    c = np.cumsum(w[index])
    return int(index[min(np.searchsorted(c, min(max(u, 0.0), np.float32(1) - np.float32(2) ** -24) * c[-1], side="right"), len(index) - 1)])
