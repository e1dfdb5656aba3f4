"""The 8-bit block format and its operators in 64 bits (numpy), written from
the definitions in include/sbl.h: the reference of the b8 tests."""
from __future__ import annotations

import numpy as np

E4M3, E5M2, I8 = 0, 1, 2
MAX = {E4M3: 448.0, E5M2: 57344.0, I8: 127.0}
MANT = {E4M3: 3, E5M2: 2}
EMIN = {E4M3: -6, E5M2: -14}
# half a step of the formats, relative to the value
HALF = {E4M3: 2.0 ** -4, E5M2: 2.0 ** -3, "bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


def code_values(typ):
    """The value of each of the 256 codes of a type (float64; NaN / Inf codes as such)."""
    out = np.empty(256)
    for c in range(256):
        if typ == I8:
            out[c] = c - 256 if c > 127 else c
            continue
        m, bias = MANT[typ], 1 - EMIN[typ]
        s, e, f = c >> 7, (c & 127) >> m, c & ((1 << m) - 1)
        v = f * 2.0 ** (1 - bias - m) if e == 0 else (1 + f / 2 ** m) * 2.0 ** (e - bias)
        if typ == E4M3 and (c & 127) == 127:
            v = np.nan
        if typ == E5M2 and e == 31:
            v = np.inf if f == 0 else np.nan
        out[c] = -v if s else v
    return out


def exponent(a, typ):
    """The block exponent for a largest magnitude a (finite)."""
    if a == 0:
        return 0
    e = -126
    while e < 127 and a > MAX[typ] * 2.0 ** e:
        e += 1
    return e


def round_to(y, typ):
    """y (float64, |y| <= MAX) to the nearest value of the type, ties to even."""
    if typ == I8:
        return np.rint(y)
    a = np.abs(y)
    _, x = np.frexp(np.where(a > 0, a, 1.0))
    step = np.ldexp(1.0, np.maximum(x - 1, EMIN[typ]) - MANT[typ])
    return np.copysign(np.rint(a / step) * step, y)


def quantize(x, typ, tiles=False):
    """x float64 [R, C] -> (values of the codes, exponents [R, B]; 128 marks a block that is not finite)."""
    r, c = x.shape
    b = -(-c // 128)
    e = np.zeros((r, b), dtype=np.int64)
    y = np.zeros_like(x)
    step = 128 if tiles else 1
    for j in range(b):
        for i in range(0, r, step):
            blk = x[i:i + step, 128 * j:128 * (j + 1)]
            if not np.isfinite(blk).all():
                e[i:i + step, j] = 128
                continue
            ee = exponent(np.abs(blk).max(), typ)
            e[i:i + step, j] = ee
            y[i:i + step, 128 * j:128 * (j + 1)] = round_to(blk * 2.0 ** -ee, typ)
    return y, e


def decode(y, e):
    s = np.where(e == 128, np.nan, np.ldexp(1.0, np.where(e == 128, 0, e)))
    return y * np.repeat(s, 128, axis=1)[:, :y.shape[1]]


def value(x, typ, tiles=False):
    return decode(*quantize(x, typ, tiles))


def scale_bytes(e, rows=None):
    """Exponents -> the scale bytes in memory order."""
    r, b = e.shape
    rp, w = -(-r // 128) * 128, -(-b // 4)
    out = np.full(4 * rp * w, 127, dtype=np.uint8)
    for j in range(b):
        i = np.arange(r)
        out[4 * ((j // 4) * rp + 128 * (i // 128) + 4 * (i % 32) + (i % 128) // 32) + j % 4] = (e[:, j] + 127).astype(np.uint8)
    return out


def act(g, kind):
    """act(g), act'(g): 0 silu, 1 squared ReLU."""
    if kind == 1:
        p = np.maximum(g, 0)
        return p * p, 2 * p
    s = np.where(g >= 0, 1 / (1 + np.exp(-np.abs(g))), np.exp(-np.abs(g)) / (1 + np.exp(-np.abs(g))))
    return g * s, s + g * s * (1 - s)


def rmsnorm_backward(x, g, eps, du, dr=None):
    """dX, dg of u = x r g, r = 1 / sqrt(mean x^2 + eps)."""
    k = x.shape[1]
    r = 1 / np.sqrt((x * x).sum(1, keepdims=True) / k + eps)
    v = du * g
    dx = r * v - x * r ** 3 * (v * x).sum(1, keepdims=True) / k
    if dr is not None:
        dx = dx + dr
    return dx, (du * x * r).sum(0)
