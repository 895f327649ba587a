"""Oracle of the paged 8-bit K/V cache and of single-token attention over it: plain
numpy, in 64 bits, one row or one query at a time, written from the definitions.

The formats: a row's e4m3 scale is 2^max(-126, ceil(log2(a / 448))) for its largest
magnitude a, its code x / scale rounded to nearest even; an int8 row's scale is
a' * (1 / 127) with a' = max(a, 127 * 2^-126), its code rint(x * (127 * (1 / a'))),
where each operation is rounded to 32 bits.
"""
from __future__ import annotations

import math

import numpy as np

E4M3, INT8 = "e4m3", "int8"


def e4m3_values() -> np.ndarray:
    """The values of the 256 e4m3 codes (bias 7; codes 0x7f and 0xff are NaN)."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        if (c & 0x7F) == 0x7F:
            v = math.nan
        out[c] = -v if c & 0x80 else v
    return out


def values(codes: np.ndarray, dtype: str) -> np.ndarray:
    """What uint8 bit patterns of codes stand for, in 64 bits."""
    if dtype == E4M3:
        return e4m3_values()[codes]
    return codes.view(np.int8).astype(np.float64)


def quantise(x: np.ndarray, dtype: str):
    """(values of the codes [..., D], scale [...]) of bf16 rows x given in 64 bits."""
    x = np.asarray(x, np.float64)
    a = np.max(np.abs(x), axis=-1)
    bad = ~np.isfinite(a)
    x = np.where(bad[..., None], 0.0, x)
    a = np.where(bad, 0.0, a)
    if dtype == E4M3:
        mant, exp = np.frexp(a)                              # a = mant 2^exp, 448 = 0.875 * 2^9
        e = np.where(a > 0, exp - 9 + (mant > 0.875), -126)
        scale = np.exp2(np.maximum(e, -126).astype(np.float64))
        y = x / scale[..., None]
        _, ye = np.frexp(np.maximum(np.abs(y), 2.0 ** -6))   # at least the smallest normal's exponent
        step = np.exp2((ye - 4).astype(np.float64))
        codes = np.rint(y / step) * step
    else:
        f = np.float32
        a32 = np.maximum(a.astype(f), f(127) * f(2.0) ** f(-126))
        scale = (a32 * (f(1) / f(127))).astype(np.float64)
        codes = np.rint(x.astype(f) * (f(127) * (f(1) / a32))[..., None]).astype(np.float64)
    return codes, np.where(bad, np.nan, scale)


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float):
    """(out [D], lse, spread) of one query over keys k, v [n, D]; spread = sum p |v| [D]."""
    if len(k) == 0:
        return np.zeros(v.shape[1]), -math.inf, np.zeros(v.shape[1])
    s = scale * (k @ q)
    m = np.max(s)
    e = np.exp(s - m)
    l = float(np.sum(e))
    p = e / l
    return p @ v, float(m + math.log(l)), p @ np.abs(v)


def gather(codes: np.ndarray, scales: np.ndarray, table, h: int, positions, dtype: str) -> np.ndarray:
    """64-bit cached rows [n, D] of head h at positions; a page outside the cache yields no row."""
    page = codes.shape[2]
    rows = []
    for p in positions:
        pg = int(table[p // page])
        if 0 <= pg < codes.shape[0]:
            rows.append(values(codes[pg, h, p % page], dtype) * float(scales[pg, h, p % page]))
    return np.array(rows).reshape(-1, codes.shape[3])
