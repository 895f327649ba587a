"""Seeded cases of chunks over the paged cache for the GPU tests: the oracle's answers with the
tolerances that their arithmetic gives."""
from __future__ import annotations

import math

import numpy as np
import torch

import block_sparse_flashattention_gb300 as bsa
from oracle import kv_cache as okv
from tests.kv_case import Pool, bf16, pages_for


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Chunks:
    """A cache with sequences of lens keys, and queries of their news newest tokens."""

    def __init__(self, seed, dtype, H, G, D, page, lens, news, kind=bsa.MASK_CAUSAL, window=0, sinks=0, prefix=0,
                 spread=0.3, size=1.5, scale=None):
        self.H, self.G, self.D, self.lens, self.news = H, G, D, lens, news
        self.pool = Pool(seed, pages_for(lens, page) + 1, H, D, page, dtype, spread=spread)
        self.host_table, self.table = self.pool.tables(lens)
        self.first = np.concatenate([[0], np.cumsum(news)]).astype(int)
        self.q = bf16(size * np.random.default_rng(seed + 1).standard_normal((self.first[-1], H * G, D))).cuda()
        self.cu, self.seqlens = i32(self.first.tolist()), i32(lens)
        self.scale = scale or 1 / math.sqrt(D)
        self.mask_args = (kind, window, sinks, prefix)
        self.kw = dict(kind=kind, mask_params=bsa.MaskParams(window_left=window, sink_tokens=sinks, prefix_len=prefix),
                       softmax_scale=self.scale)

    def parts(self, b, h):
        """(q [m G, D], k, v [keys, D], mask [m G, keys]) of sequence b, head h in 64 bits: tokens, then heads."""
        n, m, G = max(self.lens[b], 0), self.news[b], self.G
        pos = np.arange(n)
        pg = self.host_table[b][pos // self.pool.page]
        ok = (pg >= 0) & (pg < len(self.pool.codes["k"]))
        q = self.q[self.first[b]:self.first[b] + m, h * G:(h + 1) * G].float().cpu().numpy().astype(np.float64)
        mask = okv.chunk_mask(n, m, *self.mask_args) if n else np.zeros((m, 0), bool)
        return (q.reshape(m * G, self.D), self.pool.host("k", self.host_table[b], h, pos),
                self.pool.host("v", self.host_table[b], h, pos), np.repeat(mask[:, ok], G, axis=0), ok)

    def expect(self, coarse=None):
        """Oracle (out, lse, out tolerance, lse tolerance) [total, Hq, ...].

        Scores: a dot product of D fp32 terms in any order is off by at most D 2^-24 of sum |q k|;
        scales, the maximum's subtraction and the exponential's argument add 8 such steps: ds = (D + 8)
        2^-24 scale sum_d |q_d k_d|, largest over the keys.  A weight is then off by 2 ds + 2^-20
        relatively, by its rounding to fp16, 2^-11, and by the value's where its scale is not a power of two
        (int8), 2^-11 more (`coarse`: what both come to where it is not that), and absolutely by at most 2^-32 of the largest weight where it is too small for fp16, times at most 2^5 where the values
        of its tile are smaller than those of another."""
        if coarse is None:
            coarse = 2.0 ** -10 if self.pool.dtype == "int8" else 2.0 ** -11
        total, Hq = self.q.shape[:2]
        out, lse = np.zeros((total, Hq, self.D)), np.full((total, Hq), -math.inf)
        to, tl = np.zeros_like(out), np.zeros_like(lse)
        for b in range(len(self.lens)):
            m = self.news[b]
            for h in range(self.H):
                q, k, v, mask, _ = self.parts(b, h)
                if not m or not mask.any():
                    continue
                o, l, spread = okv.attend_rows(q, k, v, mask, self.scale)
                ds = (self.D + 8) * 2.0 ** -24 * self.scale * np.max(np.abs(q) @ np.abs(k).T, axis=1)
                rows, hq = slice(self.first[b], self.first[b] + m), slice(h * self.G, (h + 1) * self.G)
                out[rows, hq], lse[rows, hq] = o.reshape(m, self.G, -1), l.reshape(m, self.G)
                t = spread * (coarse + 2 * ds[:, None] + 2.0 ** -20) + len(k) * 2.0 ** -27 * np.max(np.abs(v))
                to[rows, hq] = t.reshape(m, self.G, -1)
                l0 = np.where(np.isneginf(l), 0.0, l)
                tl[rows, hq] = (ds + 2.0 ** -20 + np.abs(l0) * 2.0 ** -22).reshape(m, self.G)
        return out, lse, to, tl

    def expect_weights(self, lse):
        """Oracle (weights, tolerance) as arrays like k_scale, given the lse [total, Hq] that the call gets; NaN
        where no sequence has a key.

        A weight exp(s - lse): ds as above, the argument in base 2 is off by another 4 steps of its size and the
        exponential by 2^-20; their sum over r queries in any order by r 2^-24 of itself."""
        w = np.full(self.pool.scales["k"].shape, math.nan)
        tol = np.zeros_like(w)
        lse = lse.detach().cpu().numpy().astype(np.float64)
        for b in range(len(self.lens)):
            m = self.news[b]
            if not m or self.lens[b] <= 0:
                continue
            for h in range(self.H):
                q, k, _, mask, ok = self.parts(b, h)
                l = lse[self.first[b]:self.first[b] + m, h * self.G:(h + 1) * self.G].reshape(-1)
                pos = np.flatnonzero(ok)
                pg, row = self.host_table[b][pos // self.pool.page], pos % self.pool.page
                got = okv.weigh(q, l, k, mask, self.scale)
                l0 = np.where(np.isfinite(l), l, 0.0)
                ds = (self.D + 8) * 2.0 ** -24 * self.scale * np.max(np.abs(q) @ np.abs(k).T)
                rel = 2 * ds + 8 * 2.0 ** -24 * np.max(np.abs(l0)) + 2.0 ** -20 + len(q) * 2.0 ** -24
                w[pg, h, row] = got
                tol[pg, h, row] = got * rel + len(q) * 2.0 ** -120
        return w, tol
