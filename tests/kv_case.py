"""Seeded cases of the paged cache for the GPU tests: pools, tables, lists, and the
oracle's answers with the tolerances that their arithmetic gives."""
from __future__ import annotations

import math

import numpy as np
import torch

import block_sparse_flashattention_gb300 as bsa
from oracle import kv_cache as okv

DT = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


class Pool:
    """A cache of random rows, its host copy, and page tables of random pages."""

    def __init__(self, seed, pages, H, D, page, dtype, spread=0.3, device="cuda"):
        self.rng = np.random.default_rng(seed)
        self.dtype, self.page, self.H, self.D = dtype, page, H, D
        self.codes, self.scales = {}, {}
        tens = {}
        for n in ("k", "v"):
            x = self.rng.standard_normal((pages, H, page, D)) * np.exp(spread * self.rng.standard_normal((pages, H, page, 1)))
            x = bf16(x).float().numpy().astype(np.float64)
            val, s = okv.quantise(x, dtype)
            if dtype == "e4m3":
                c = torch.from_numpy(val.astype(np.float32)).to(torch.float8_e4m3fn)
            else:
                c = torch.from_numpy(val.astype(np.int8))
            self.codes[n] = c.view(torch.uint8).numpy().copy()
            self.scales[n] = s.astype(np.float32)
            tens[n] = c.to(device)
        self.device = device
        self.cache = bsa.KVCache(tens["k"], tens["v"], *(torch.from_numpy(self.scales[n]).to(device) for n in ("k", "v")))
        self.free = list(self.rng.permutation(pages))

    def take(self, n):
        return [int(self.free.pop()) for _ in range(n)]

    def tables(self, lens, cols=None):
        """(host table, device table): random pages for every length; unused entries are -1."""
        need = [-(-max(n, 0) // self.page) for n in lens]
        t = np.full((len(lens), cols or max(max(need), 1)), -1, np.int32)
        for b, n in enumerate(need):
            t[b, :n] = self.take(n)
        return t, torch.from_numpy(t).to(self.device)

    def host(self, name, table, h, positions):
        """64-bit rows of head h at positions; a page outside the cache yields no row (okv.gather, vectorised)."""
        pos = np.asarray(positions, np.int64)
        pg = np.asarray(table, np.int64)[pos // self.page] if len(pos) else pos
        on = (pg >= 0) & (pg < len(self.codes[name]))
        pg, row = pg[on], pos[on] % self.page
        return okv.values(self.codes[name][pg, h, row], self.dtype) * self.scales[name][pg, h, row].astype(np.float64)[:, None]


def pages_for(lens, page):
    return sum(-(-max(n, 0) // page) for n in lens)


def expect(pool, q, G, parts, scale, coarse=0.0):
    """Oracle (out, lse, out tolerance, lse tolerance) [B, Hq, ...]; parts(b, h): list of (table, positions).

    Scores: a dot product of D fp32 terms, accumulated in any order, is off by at most
    D 2^-24 of sum |q k|, and the three multiplications by scales, the subtraction of the
    maximum and the base-2 exponential's argument add 8 more such steps of the score's
    own size: ds = (D + 8) 2^-24 scale sum_d |q_d k_d|, largest over the keys.  A weight
    exp(s - m) is then off by 2 ds (numerator and sum) + 2^-20 (the exponentials' and
    sums' own rounding) relatively, by its rounding to fp16, 2^-11 of it, and absolutely
    by 2^-32 of the largest weight times its value where it is too small for fp16.

    coarse: relative error of every element of V that the call may make (long prefixes
    whose value scales are rounded with the codes: 2 * 2^-11)."""
    B, Hq, D = q.shape
    out, lse = np.zeros((B, Hq, D)), np.full((B, Hq), -math.inf)
    to, tl = np.zeros((B, Hq, D)), np.zeros((B, Hq))
    for b in range(B):
        for h in range(Hq // G):
            k = np.concatenate([pool.host("k", t, h, p) for t, p in parts(b, h)] or [np.zeros((0, D))])
            v = np.concatenate([pool.host("v", t, h, p) for t, p in parts(b, h)] or [np.zeros((0, D))])
            for g in range(G):
                x = q[b, h * G + g]
                o, l, spread = okv.attend(x, k, v, scale)
                out[b, h * G + g], lse[b, h * G + g] = o, l
                if len(k):
                    ds = (D + 8) * 2.0 ** -24 * scale * float(np.max(np.abs(k) @ np.abs(x)))
                    to[b, h * G + g] = spread * (2.0 ** -11 + 2 * ds + coarse + 2.0 ** -20) + len(k) * 2.0 ** -32 * np.max(np.abs(v))
                    tl[b, h * G + g] = ds + 2.0 ** -20 + abs(l) * 2.0 ** -22
    return out, lse, to, tl


def agree(out, lse, ref):
    """Asserts device results against expect()'s; a bf16 output is rounded once more (half a step, 2^-8)."""
    o, l, to, tl = ref
    got, gl = f64(out), f64(lse)
    if out.dtype == torch.bfloat16:
        to = to + 2.0 ** -8 * (np.abs(o) + to)
    empty = np.isneginf(l)
    assert np.array_equal(np.isneginf(gl), empty)
    assert not got[empty].any()
    assert np.all(np.abs(gl[~empty] - l[~empty]) <= tl[~empty]), np.max(np.abs(gl - l)[~empty] / tl[~empty])
    assert np.all(np.isfinite(got))
    bad = np.abs(got - o) > to
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], o[bad][:4], to[bad][:4])


def lists(pool_H, lens, tiles, *, valid=None, kind="varlen", mask_every=0, device="cuda"):
    """A Meta whose full (and, with mask_every, mask) lists hold tiles(b, h), one query row per sequence.

    mask_every = m > 0: every m-th listed tile goes to the mask list."""
    B, H = len(lens), pool_H
    nn = [-(-max(n, 0) // 128) for n in lens]
    num_n = max(max(nn), 1)
    off = np.concatenate([[0], np.cumsum(nn)]).astype(np.int32)
    if kind == "varlen":
        cnt = np.zeros((2, H, B), np.int32)
        idx = np.full((2, H, max(int(off[-1]), 1)), -1, np.int32)
    else:
        cnt = np.zeros((2, B, H, 1), np.int32)
        idx = np.full((2, B, H, 1, num_n), -1, np.int32)
    for b in range(B):
        for h in range(H):
            put = [[], []]
            for i, t in enumerate(tiles(b, h)):
                put[1 if mask_every and i % mask_every == 0 else 0].append(t)
            for m in range(2):
                if kind == "varlen":
                    cnt[m, h, b] = len(put[m])
                    idx[m, h, off[b]:off[b] + len(put[m])] = put[m]
                else:
                    cnt[m, b, h, 0] = len(put[m])
                    idx[m, b, h, 0, :len(put[m])] = put[m]
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(device)  # noqa: E731
    kw = dict(varlen=1, num_m=0, num_n=num_n, total_m_blocks=B, total_n_blocks=idx.shape[-1],
              cu_total_m_blocks=d(np.arange(B + 1, dtype=np.int32)), cu_block_idx_offsets=d(off)) \
        if kind == "varlen" else dict(varlen=0, num_m=1, num_n=num_n)
    return bsa.Meta(d(cnt[0]), d(idx[0]), d(cnt[1]), d(idx[1]), B=B, H=H, **kw)
