"""Oracle: the quantised cache's rows and attention with changed scores, float64 numpy.

TEST INFRASTRUCTURE (see the package docstring): nothing in the CUDA library uses this file.

A row is stored as e4m3 codes times a power of two: the smallest exponent e in [-32, 31] with
max |x| <= 448 * 2^e, each x * 2^-e rounded to the nearest e4m3 value (ties to the even code).  A row
with a value that is not finite is NaN as a whole: exponent byte 255, codes 0x7f.  The 256 values are spelled out from the format: sign, 4 exponent bits with bias 7, 3 fraction bits, no
infinities, 0x7f and 0xff NaN.
"""
from __future__ import annotations

import math

import numpy as np

LOW, HIGH, BIAS, NAN = -32, 31, 127, 255


def e4m3_table() -> np.ndarray:
    """The value of each of the 256 codes."""
    out = np.empty(256)
    for code in range(256):
        sign, e, m = code >> 7, (code >> 3) & 15, code & 7
        x = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        if e == 15 and m == 7:
            x = math.nan
        out[code] = -x if sign else x
    return out


_TABLE = e4m3_table()


def to_code(x: np.ndarray) -> np.ndarray:
    """The nearest code of each float64 value (clamped to +-448; NaN to 0x7f), ties to the even code."""
    x = np.asarray(x, dtype=np.float64)
    mag = np.minimum(np.abs(x), 448.0)
    grid = _TABLE[:127]                     # 0 .. 448, ascending
    hi = np.clip(np.searchsorted(grid, mag), 1, 126)
    lo = hi - 1
    below, above = mag - grid[lo], grid[hi] - mag
    code = np.where(below < above, lo, np.where(above < below, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(np.isnan(x), 0x7F, code + np.where(np.signbit(x), 128, 0))
    return code.astype(np.uint8)


def exponents(rows: np.ndarray) -> np.ndarray:
    """The exponent of each finite row's scale: from LOW on, one more for every power that is too small."""
    top = np.max(np.abs(rows), axis=-1, initial=0.0)
    e = np.full(top.shape, LOW)
    for k in range(LOW, HIGH):
        e = e + (top > 448.0 * 2.0 ** k)
    return e


def quantise(x: np.ndarray):
    """x float64 [..., D]: codes uint8 [..., D] and stored exponent bytes uint8 [...]."""
    x = np.asarray(x, dtype=np.float64)
    dead = ~np.isfinite(x).all(-1)
    x = np.where(dead[..., None], 0.0, x)
    e = exponents(x)
    codes = to_code(x * 2.0 ** -e.astype(np.float64)[..., None])
    codes[dead] = 0x7F
    return codes, np.where(dead, NAN, e + BIAS).astype(np.uint8)


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """The values that codes [..., D] with exponent bytes [...] stand for."""
    f = np.where(scales == NAN, np.nan, 2.0 ** (scales.astype(np.float64) - BIAS))
    return _TABLE[codes] * f[..., None]


def scored_attention(q, K, V, ctx: int, scale: float, softcap: float = 0.0, slopes=None,
                     visible: int = 0, window: int = 0):
    """One sequence: q [n, Hq, D] at positions ctx .., K and V [kv, Hkv, D] -> out [n, Hq, D], lse
    [n, Hq], and the size of each row's weighted values, sum_j p_j |v_j| [n, Hq, D]."""
    n, hq, _ = q.shape
    kv, hkv, _ = K.shape
    out, size = np.empty(q.shape), np.empty(q.shape)
    lse = np.empty((n, hq))
    keys = np.arange(kv)
    pos = ctx + np.arange(n)
    seen = (keys[None] <= pos[:, None]) | (keys[None] < visible)
    if window > 0:
        seen &= keys[None] > pos[:, None] - window
    for h in range(hq):
        g = h // (hq // hkv)
        x = q[:, h] @ K[:, g].T * scale
        if softcap > 0:
            x = softcap * np.tanh(x / softcap)
        if slopes is not None:
            x = x + float(slopes[h]) * (keys[None] - pos[:, None])
        x = np.where(seen, x, -np.inf)
        m = x.max(axis=1, keepdims=True)
        p = np.exp(x - m)
        total = p.sum(axis=1, keepdims=True)
        p /= total
        v = np.where(np.isfinite(V[:, g]), V[:, g], 0) if not seen.all() else V[:, g]
        out[:, h] = p @ v
        size[:, h] = p @ np.abs(v)
        lse[:, h] = (m + np.log(total))[:, 0]
    return out, lse, size
