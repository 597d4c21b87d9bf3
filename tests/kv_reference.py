"""Plain fp64 implementation of the 8-bit key/value cache's operators, from the definitions in include/np.h: what the
GPU tests compare with. It stores codes and exponents per block (page, head, K or V) in natural order."""
from __future__ import annotations

import numpy as np


def e4m3_values() -> np.ndarray:
    b = np.arange(256)
    x, f = (b >> 3) & 15, b & 7
    v = np.where(x == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (x - 10.0))
    return np.where((b & 127) == 127, np.nan, v) * np.where(b > 127, -1.0, 1.0)


def round_e4m3(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value (ties to even) of |x| <= 448; NaN stays."""
    a = np.abs(x)
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.where(np.isnan(a), 1.0, a), 2.0 ** -6))) - 3)
    return np.copysign(np.rint(a / step) * step, x)


def exponent_for(top: float) -> int:
    if top == 0:
        return -120
    m, e = np.frexp(top)                      # top = m * 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    return int(min(120, max(-120, e - 9 + (m > 0.875))))


def quantise(x: np.ndarray, old: np.ndarray, e_old: int | None):
    """Block rule: new values x [n, hd], earlier code values old [m, hd] at e_old -> (code values [m + n, hd], e)."""
    x = x.astype(np.float64)
    fin = np.abs(x[np.isfinite(x)])
    e = exponent_for(fin.max() if fin.size else 0.0)
    if e_old is not None:
        e = max(e, e_old)
        old = round_e4m3(old * 2.0 ** (e_old - e))
    scaled = np.where(np.isinf(x), np.copysign(448.0, x), x / 2.0 ** e)
    return np.concatenate([old, round_e4m3(scaled)]), e


class RefSeq:
    """One sequence of one layer: code values and exponents per page, heads and K/V."""

    def __init__(self, n_kv: int, hd: int, page: int):
        self.n_kv, self.hd, self.page = n_kv, hd, page
        self.codes = np.zeros((0, 2, n_kv, hd))  # [tokens]
        self.exps = np.zeros((0, 2, n_kv), dtype=np.int64)  # [pages]

    def append(self, k: np.ndarray, v: np.ndarray) -> None:
        n0, n, pt = len(self.codes), len(k), self.page
        self.codes = np.concatenate([self.codes, np.zeros((n, 2, self.n_kv, self.hd))])
        for p in range(n0 // pt, -(-(n0 + n) // pt)):
            if p >= len(self.exps):
                self.exps = np.concatenate([self.exps, np.zeros((1, 2, self.n_kv), dtype=np.int64)])
            lo, hi = max(n0, p * pt), min(n0 + n, (p + 1) * pt)
            for side, x in ((0, k), (1, v)):
                for h in range(self.n_kv):
                    fresh = lo == p * pt
                    c, e = quantise(x[lo - n0:hi - n0, h], self.codes[p * pt:lo, side, h], None if fresh else int(self.exps[p, side, h]))
                    self.codes[p * pt:hi, side, h] = c
                    self.exps[p, side, h] = e

    def values(self):
        """k, v [tokens, n_kv, hd] in fp64."""
        e = np.repeat(self.exps, self.page, axis=0)[:len(self.codes)]
        x = self.codes * 2.0 ** e[..., None].astype(np.float64)
        return x[:, 0], x[:, 1]


def attention(q, k, v, before: int, scale: float, window: int = 0, sinks: int = 0, held=None):
    """q [n, H, hd], k, v [before + n, Hk, hd] fp64 -> out [n, H, hd], lse [n, H], and per output the scale of its terms
    (sum p |v| / l) and per row the largest sum |q||k| * scale (for error bounds). Only visible tokens enter."""
    n, H, hd = q.shape
    Hk = k.shape[1]
    out, terms = np.zeros((n, H, hd)), np.zeros((n, H, hd))
    lse, mag = np.full((n, H), -np.inf), np.zeros((n, H))
    for i in range(n):
        pos = before + i
        j = np.arange(pos + 1)
        ok = np.ones(pos + 1, bool) if held is None else held[:pos + 1].copy()
        if window:
            ok &= (pos - j < window) | (j < sinks)
        j = j[ok]
        if not j.size:
            continue
        for h in range(H):
            kk, vv = k[j, h // (H // Hk)], v[j, h // (H // Hk)]
            with np.errstate(all="ignore"):
                s = kk @ q[i, h] * scale
                p = np.exp(s - s.max())
                l = p.sum()
                out[i, h] = p @ vv / l
                terms[i, h] = p @ np.abs(vv) / l
                lse[i, h] = np.log(l) + s.max()
                mag[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * scale
    return out, lse, terms, mag


U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}  # half a step, relative


def bound(out, terms, mag, n_tokens: int, hd: int, dtype: str):
    """|error| of an output: its own rounding; the weights' rounding (fp16 for 16-bit types, 3 x 8 bits for fp32); the
    scores' fp32 error, which exp turns into a relative one (hd products, then the scale, the exponent's argument and
    the exponential: 8 more steps of 2^-24, on magnitudes up to mag and on the exponent's own size); fp32 sums over
    n_tokens terms in the numerator and the denominator. First-order terms, doubled for the products of them."""
    weights = 2.0 ** -11 if dtype != "f32" else 2.0 ** -24
    scores = ((hd + 8) * mag + 8 * (1 + mag))[..., None] * 2.0 ** -24
    sums = 2 * (n_tokens + 16) * 2.0 ** -24
    tiny = 2.0 ** -24 if dtype == "f16" else 2.0 ** -126  # subnormal outputs
    return U[dtype] * np.abs(out) * 1.01 + 2 * terms * (weights + 2 * scores + sums) + tiny


def lse_bound(lse, mag, n_tokens: int, hd: int):
    return 2 * ((hd + 8) * mag + (n_tokens + 16) + 8 * np.abs(lse) + 8) * 2.0 ** -24
