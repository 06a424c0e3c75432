"""Plain 64-bit references of the operators in include/mnb_ops.h (numpy; nothing of the
package).  Numbers in, numbers out: ``bits`` helpers turn them into the device's types."""
from __future__ import annotations

import numpy as np

FP4 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])
# fmt: (mantissa bits, lowest exponent, largest value, largest exponent)
FORMATS = {0: (1, 0, 6.0, 2), 1: (3, -6, 448.0, 8)}


def e4m3(codes):
    c = np.asarray(codes).astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e > 0, np.ldexp(1 + m / 8.0, e - 7), np.ldexp(m / 8.0, -6))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >= 128, -v, v)


def round_elements(v, fmt):
    """Nearest value of the element format, ties to even, clamped; v finite."""
    man, low, top, _ = FORMATS[fmt]
    a = np.minimum(np.abs(v), top)
    octave = np.frexp(a)[1] - 1
    q = np.ldexp(1.0, np.maximum(octave, low) - man)
    return np.copysign(np.rint(a / q) * q, v)


def block_scales(x, fmt):
    """int scale bytes of x [..., K] (float64), 255 for blocks with NaN or infinity."""
    b = np.abs(x.reshape(*x.shape[:-1], -1, 32))
    amax = b.max(-1)
    e = np.frexp(np.where(np.isfinite(amax), amax, 1))[1] - 1 - FORMATS[fmt][3]
    e = np.where(amax == 0, -127, np.clip(e, -127, 127))
    return np.where(np.isfinite(b).all(-1), e + 127, 255).astype(np.int64)


def quantize(x, fmt):
    """(element values [M, K] before scaling, scale bytes [M, K/32])."""
    x = np.asarray(x, np.float64)
    s = block_scales(x, fmt)
    bad = s == 255
    e = np.where(bad, 0, s - 127)
    b = np.where(bad[..., None], 0.0, x.reshape(*s.shape, 32))
    return round_elements(np.ldexp(b, -e[..., None]), fmt).reshape(x.shape), s


def element_codes(q, fmt):
    """Codes of exact element values: uint8 [M, K/2] (FP4) or [M, K]."""
    sign = np.signbit(q)
    a = np.abs(q)
    if fmt == 0:
        c = (np.searchsorted(FP4[:8], a) + 8 * sign).astype(np.uint8)
        return c[..., 0::2] | (c[..., 1::2] << 4)
    table = e4m3(np.arange(127))
    return (np.searchsorted(table, a) + 128 * sign).astype(np.uint8)


def element_values(codes, fmt):
    if fmt == 0:
        c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
        return FP4[c]
    return e4m3(codes)


def scale_values(s):
    s = np.asarray(s).astype(np.int64)
    return np.where(s == 255, np.nan, np.ldexp(1.0, s - 127))


def dequantize(codes, scales, fmt):
    return element_values(codes, fmt) * np.repeat(scale_values(scales), 32, -1)


def pack(codes, scales, N, K):
    """The device layout of include/mnb_ops.h: (wq bytes, sc bytes)."""
    ng, ks, kb = -(-N // 64), -(-K // 128), -(-K // 512)
    wq = np.zeros((ng, ks, 4, 64, 16), np.uint8)
    sc = np.zeros((ng, kb, 4, 64, 4), np.uint8)
    for g in range(ng):
        for f in range(4):
            for lane in range(64):
                r, b = lane % 16, lane // 16
                n = 64 * g + 16 * (r // 4) + 4 * f + r % 4
                if n >= N:
                    continue
                for s in range(ks):
                    k = s * 4 + b
                    if k < K // 32:
                        wq[g, s, f, lane] = codes[n, k * 16:k * 16 + 16]
                        sc[g, s // 4, f, lane, s % 4] = scales[n, k]
    return wq.reshape(-1), sc.reshape(-1)


def rmsnorm(x, residual, w, eps):
    h = x if residual is None else x + residual
    return h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * w, h


def logprobs(x, tokens, top):
    """(logprob, entropy, sum p |x - m|, top values, top indices), 64 bits; ordinary rows."""
    with np.errstate(invalid="ignore", over="ignore"):
        m = x.max(-1, keepdims=True)
        d = x - m
        e = np.exp(d)
        S = e.sum(-1)
        lse = np.log(S)
        p = e / S[:, None]
        spread = np.where(p > 0, p * np.abs(np.where(p > 0, d, 0)), 0).sum(-1)
        lp = None if tokens is None else d[np.arange(len(x)), tokens] - lse
        idx = np.argsort(-x, axis=-1, kind="stable")[:, :top]
        return lp, lse + spread, spread, np.take_along_axis(d, idx, 1) - lse[:, None], idx
