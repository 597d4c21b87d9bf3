"""Rotary positions and the norms before them in fp64, from the definitions in include/np.h, and what the kernels may be off."""
from __future__ import annotations

import numpy as np

U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}  # half a step, relative
# What fp32 leaves out, in 2^-24 of amplitude * (|a| + |b|): the norm's factor 13 (a sum of squares of 16 values a lane and 4
# joins: 20, a division and a sum: 22, halved by the root, then the root and the reciprocal) and 2 products; the sine and cosine
# 4 (the angle's conversion and product with 2 pi, the last step of the series, the terms left out); the amplitude 1; two products and their sum 2.
STEPS = 22


def freqs(rot, base=10000.0, scaling="none", factor=1.0, context=0, low=0.0, high=0.0):
    got = []
    for i in range(rot // 2):
        f = base ** (-2 * i / rot)
        if scaling == "linear":
            f /= factor
        elif scaling == "ntk":
            f = (base * factor ** (rot / (rot - 2))) ** (-2 * i / rot)
        elif scaling == "blend":
            n = context * f / (2 * np.pi)
            g = 0.0 if n <= low else 1.0 if n >= high else (n - low) / (high - low)
            f = g * f + (1 - g) * f / factor
        got.append(f)
    return np.array(got, dtype=np.float64)


def turned(x, pos, f, layout="half", amplitude=1.0, weight=None, eps=0.0):
    """x fp64 [rows, heads, hd] -> (y, scale of what its errors are relative to)."""
    x = x.astype(np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    h, rot = len(f), 2 * len(f)
    a = np.arange(h) if layout == "half" else 2 * np.arange(h)
    b = a + h if layout == "half" else a + 1
    # the angle as a fraction of a turn: p * f / (2 pi) mod 1 in extended precision
    t = np.asarray(pos, dtype=np.longdouble)[:, None] * (f.astype(np.longdouble) / (2 * np.longdouble("3.14159265358979323846264338327950288")))
    t = (t - np.floor(t)).astype(np.float64) * 2 * np.pi
    c, s = np.cos(t)[:, None], np.sin(t)[:, None]
    y, mag = x.copy(), np.abs(x)
    with np.errstate(invalid="ignore"):
        y[..., a] = (x[..., a] * c - x[..., b] * s) * amplitude
        y[..., b] = (x[..., a] * s + x[..., b] * c) * amplitude
        mag[..., a] = mag[..., b] = (np.abs(x[..., a]) + np.abs(x[..., b])) * amplitude
    return y, mag


def bound(y, mag, dtype):
    tiny = 2.0 ** -25 if dtype == "f16" else 2.0 ** -126   # half a step of subnormal results
    return U[dtype] * np.abs(y) * 1.01 + STEPS * 2.0 ** -24 * mag * 1.01 + tiny
