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


def chunk_mask(n: int, m: int, kind: int, window: int = 0, sinks: int = 0, prefix: int = 0) -> np.ndarray:
    """[m, n]: whether the query at position n - m + t meets key j (kinds numbered as in the C ABI:
    0 all keys, 1 causal, 2 sliding window with sink tokens, 4 prefix)."""
    i, j = np.arange(n - m, n)[:, None], np.arange(n)[None]
    if kind == 0:
        return np.ones((m, n), bool)
    if kind == 1:
        return j <= i
    if kind == 2:
        return (j <= i) & ((i - j < window) | (j < sinks))
    if kind == 4:
        return (j < prefix) | (j <= i)
    raise ValueError(kind)


def attend_rows(q: np.ndarray, k: np.ndarray, v: np.ndarray, mask: np.ndarray, scale: float):
    """``attend`` of every row of q [r, D] over the keys its row of mask [r, n] names: (out, lse, spread)."""
    out = np.zeros((len(q), v.shape[1]))
    lse, spread = np.full(len(q), -math.inf), np.zeros_like(out)
    for r in range(len(q)):
        out[r], lse[r], spread[r] = attend(q[r], k[mask[r]], v[mask[r]], scale)
    return out, lse, spread


def weigh(q: np.ndarray, lse: np.ndarray, k: np.ndarray, mask: np.ndarray, scale: float) -> np.ndarray:
    """[n]: the weight that the rows of q [r, D], with their lse [r], give to keys k [n, D]."""
    w = np.zeros(len(k))
    for r in range(len(q)):
        if lse[r] != -math.inf:
            w[mask[r]] += np.exp(scale * (k[mask[r]] @ q[r]) - lse[r])
    return w


def evict(weights: np.ndarray, keep: int, recent: int, sinks: int) -> np.ndarray:
    """The ascending positions that stay of keys with these weights [n]; a weight None stands for a key that
    cannot be read."""
    n = len(weights)
    if n <= keep:
        return np.arange(n)
    first = [j for j in range(n) if j < sinks or j >= n - recent]

    def rank(j):
        w = weights[j]
        if w is None:
            return (2, 0.0, j)
        return (0, 0.0, j) if math.isnan(w) else (1, -float(w), j)
    rest = sorted((j for j in range(n) if sinks <= j < n - recent), key=rank)
    return np.array(sorted(first + rest[:keep - len(first)]))
