"""Operators over a paged 8-bit K/V cache for chunks of new tokens and for a bounded cache: the calls that are
measured, and their plain forms.

Three operators, each reached through the package's public calls:

  prefill  prefill: the queries of each sequence's newest tokens (one or thousands) attend over its cached keys, their
           own among them, under a causal or sliding-window mask
  weigh    kv_weigh: the attention weight that those queries give to every cached key, summed over queries and over
           the query heads of a KV head
  evict    kv_evict: per sequence and KV head, the keys of most weight (with the first and the newest ones) are kept and
           moved, in order, to other pages

A cache holds, per page and KV head, `page` rows of D one-byte codes (e4m3 or int8) and one fp32 scale per row
([pages, H, page, D] and [pages, H, page], for K and for V); position p of sequence b is row p % page of page
page_table[b][p // page], and its value is code * scale.  Weights lie like a scale: fp32 [pages, H, page].

A sequence of n keys with m new tokens has its queries at the positions i = n - m .. n - 1.  Query i meets the keys
j <= i, with a window only those with i - j < window or j < sinks:

  s_ij = q_i . k_j / sqrt(D),  lse_i = ln sum_j exp(s_ij),  out_i = sum_j exp(s_ij - lse_i) v_j,
  weight_j = sum_i exp(s_ij - lse_i)

`own` False: elementary torch operations.  `own` True: the package's operators.
"""
import math

import torch

own = False

E4M3, INT8 = torch.float8_e4m3fn, torch.int8


def _cdiv(a, b):
    return -(-a // b)


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # eight sequences check a draft of four tokens each (latency)
        dict(name="prefill_draft", op="prefill", dtype="e4m3", B=8, H=8, G=4, D=128, page=64, old_lo=100, old_hi=4096,
             new_lo=4, new_hi=4, window=0, sinks=0),
        # a step of a server that mixes single tokens with chunks of prompts; small pages
        dict(name="prefill_mixed", op="prefill", dtype="int8", B=16, H=8, G=4, D=128, page=16, old_lo=0, old_hi=4096,
             new_lo=1, new_hi=512, window=0, sinks=0),
        # whole prompts of 100 to 4096 tokens at once, as many KV heads as query heads, heads of 64
        dict(name="prefill_prompts", op="prefill", dtype="e4m3", B=8, H=16, G=1, D=64, page=128, old_lo=0, old_hi=0,
             new_lo=100, new_hi=4096, window=0, sinks=0),
        # a chunk of a long prompt behind what has been cached of it
        dict(name="prefill_long", op="prefill", dtype="int8", B=1, H=8, G=4, D=128, page=64, old_lo=61440,
             old_hi=61440, new_lo=2048, new_hi=2048, window=0, sinks=0),
        # the last chunk of the long-context workload: its length and heads, its window and its sink tokens
        dict(name="prefill_window", op="prefill", dtype="e4m3", B=1, H=32, G=1, D=128, page=128, old_lo=126976,
             old_hi=126976, new_lo=4096, new_hi=4096, window=4096, sinks=512),
        # the weights of one decoding step of two short sequences (latency)
        dict(name="weigh_small", op="weigh", dtype="e4m3", B=2, H=4, G=1, D=128, page=128, old_lo=1023, old_hi=1023,
             new_lo=1, new_hi=1, window=0, sinks=0),
        # the weights of a serving batch's decoding step, four query heads a KV head
        dict(name="weigh_step", op="weigh", dtype="int8", B=64, H=8, G=4, D=128, page=64, old_lo=100, old_hi=4096,
             new_lo=1, new_hi=1, window=0, sinks=0),
        # the last 64 tokens of one long sequence say what its cache is to keep
        dict(name="weigh_last", op="weigh", dtype="e4m3", B=1, H=24, G=1, D=128, page=128, old_lo=61376,
             old_hi=61376, new_lo=64, new_hi=64, window=0, sinks=0),
        # every token of a chunk counts
        dict(name="weigh_chunk", op="weigh", dtype="int8", B=1, H=8, G=4, D=128, page=64, old_lo=31744,
             old_hi=31744, new_lo=2048, new_hi=2048, window=0, sinks=0),
        # two short sequences are cut in half (latency), heads of 64
        dict(name="evict_small", op="evict", dtype="e4m3", B=2, H=4, D=64, page=128, lo=1024, hi=1024, keep=512,
             recent=64, sinks=4),
        # a serving batch: sequences of 100 to 4096 keys are bounded by 1024
        dict(name="evict_batch", op="evict", dtype="int8", B=64, H=8, D=128, page=64, lo=100, hi=4096, keep=1024,
             recent=128, sinks=4),
        # one sequence at the long-context workload's length and heads keeps a quarter, window and sink tokens among it
        dict(name="evict_long", op="evict", dtype="e4m3", B=1, H=32, D=128, page=128, lo=131072, hi=131072,
             keep=32768, recent=4096, sinks=512),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


# What a drawn case stays under: (query, key) pairs x query heads x D of the largest listed ones, cached elements.
PAIRS = {"prefill": 2048 * 61440 * 32 * 128, "weigh": 2048 * 32768 * 32 * 128}
KEYS = 65536 * 24 * 128


def draw(rng):
    op = rng.choice(["prefill", "prefill", "prefill", "weigh", "weigh", "evict", "evict"])
    c = dict(op=op, dtype=rng.choice(["e4m3", "int8"]), D=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]))
    c["B"], c["H"] = _log_int(rng, 1, 32), _log_int(rng, 1, 32)
    most = max(1, min(131072, KEYS // (c["B"] * c["H"] * c["D"])))
    if op == "evict":
        c["hi"] = _log_int(rng, 1, most)
        c["lo"] = _log_int(rng, 1, c["hi"])
        c["keep"] = _log_int(rng, 1, c["hi"])
        c["recent"] = rng.randint(0, c["keep"] // 2)
        c["sinks"] = rng.randint(0, min(4, c["keep"] - c["recent"]))
        return c
    c["G"] = rng.choice([1, 1, 2, 3, 4, 4, 5, 6, 7, 8, 12, 16])
    c["old_hi"] = _log_int(rng, 1, most) - 1
    c["old_lo"] = _log_int(rng, 1, c["old_hi"] + 1) - 1
    # with m new tokens behind p others: m p + m^2 pairs at most
    room = max(1, PAIRS[op] // (c["B"] * c["H"] * c["G"] * c["D"]))
    p = c["old_hi"]
    new = max(1, min(4096, most, int((math.sqrt(p * p + 4.0 * room) - p) / 2)))
    c["new_hi"] = _log_int(rng, 1, new)
    c["new_lo"] = _log_int(rng, 1, c["new_hi"])
    near = rng.random() < 0.3
    c["window"], c["sinks"] = (_log_int(rng, 1, 8192), rng.choice([0, 4, 128, 500])) if near else (0, 0)
    return c


def _spread(lo, hi, n, at):
    """n numbers spread over lo..hi by the golden ratio (the same for every seed)."""
    return [lo + int((hi - lo + 1) * ((at + i * 0.6180339887498949) % 1.0)) for i in range(n)]


def _lengths(c):
    """(keys, new tokens) of a case's sequences."""
    if c["op"] == "evict":
        return _spread(c["lo"], c["hi"], c["B"], 0.5), None
    new = _spread(c["new_lo"], c["new_hi"], c["B"], 0.25)
    return [o + m for o, m in zip(_spread(c["old_lo"], c["old_hi"], c["B"], 0.5), new)], new


def _first_seen(c, n, m):
    """(sinks, first): the keys that some query of the sequence meets are 0 .. sinks - 1 and first .. n - 1."""
    if not c["window"]:
        return 0, 0
    first = max(0, n - m - c["window"] + 1)
    return min(c["sinks"], first), first


# ------------------------------------------------------------------ inputs --

def _cache_rows(shape, dtype, g, dev):
    """Codes (uint8) and scales of normal rows whose magnitudes vary from row to row, as quantised rows have them."""
    x = torch.randn(shape, generator=g, device=dev, dtype=torch.float32)
    x *= torch.exp(0.3 * torch.randn(shape[:-1], generator=g, device=dev, dtype=torch.float32))[..., None]
    a = x.abs().amax(-1).clamp(min=1e-20)
    if dtype == "int8":
        s = a / 127.0
        return torch.round(x / s[..., None]).clamp(-127, 127).to(INT8).view(torch.uint8), s
    s = torch.exp2(torch.ceil(torch.log2(a / 448.0)))
    return (x / s[..., None]).clamp(-448, 448).to(E4M3).view(torch.uint8), s


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev).manual_seed(7368787 * int(seed) + 29)
    lens, new = _lengths(c)
    cols = [_cdiv(n, c["page"]) for n in lens]
    fresh = [_cdiv(min(n, c["keep"]), c["page"]) for n in lens] if c["op"] == "evict" else []
    pages = sum(cols) + sum(fresh)
    perm = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    at = 0

    def table(need):
        nonlocal at
        t = torch.zeros((c["B"], max(need)), device=dev, dtype=torch.int32)
        for b, n in enumerate(need):
            t[b, :n] = perm[at:at + n]
            at += n
        return t

    st = dict(case=dict(c), page_table=table(cols), lens=lens, new=new, pages=pages,
              seqlens=torch.tensor(lens, device=dev, dtype=torch.int32))
    shape = (pages, c["H"], c["page"], c["D"])
    for name in ("k", "v"):
        codes = torch.empty(shape, device=dev, dtype=torch.uint8)
        scale = torch.empty(shape[:-1], device=dev, dtype=torch.float32)
        step = max(1, (64 << 20) // (shape[1] * shape[2] * shape[3]))
        for p in range(0, pages, step):
            r = (min(step, pages - p),) + shape[1:]
            codes[p:p + step], scale[p:p + step] = _cache_rows(r, c["dtype"], g, dev)
        st[name], st[name + "_scale"] = codes.view(E4M3 if c["dtype"] == "e4m3" else INT8), scale
    if c["op"] == "evict":
        st["out_table"] = table(fresh)
        # sums of many softmax weights: a few keys hold most, many hold next to nothing, some exactly nothing
        w = torch.exp(2.0 * torch.randn(shape[:-1], generator=g, device=dev) - 4.0)
        st["weights"] = w * (torch.rand(shape[:-1], generator=g, device=dev) > 0.1)
        return st
    total = sum(new)
    st["cu"] = torch.tensor([0] + new, device=dev, dtype=torch.int32).cumsum(0).to(torch.int32)
    # queries: normal rows, somewhat longer than 1 so that the softmax is neither flat nor one key
    st["q"] = (1.5 * torch.randn((total, c["H"] * c["G"], c["D"]), generator=g, device=dev)).to(torch.bfloat16)
    if c["op"] == "weigh":
        st["weights"] = torch.zeros(shape[:-1], device=dev, dtype=torch.float32)
        st["lse"] = _plain_prefill(st, lse_only=True)       # what prefill or decode gave for these queries
    return st


# -------------------------------------------------------------- plain forms --

SCORES = 1 << 28   # scores that a plain form holds at a time


def _seen(st, b):
    """Positions of the keys that some query of sequence b meets, and their page and row."""
    n, m = st["lens"][b], st["new"][b]
    sinks, first = _first_seen(st["case"], n, m)
    dev, page = st["page_table"].device, st["case"]["page"]
    pos = torch.arange(first, n, device=dev)
    if sinks:
        pos = torch.cat([torch.arange(sinks, device=dev), pos])
    return pos, st["page_table"][b].long()[pos // page], pos % page


def _values(st, name, pg, row, heads):
    """fp32 values [heads, keys, D] of cached rows."""
    codes = st[name].view(torch.uint8)[pg[None], heads[:, None], row[None]].view(st[name].dtype)
    return codes.float() * st[name + "_scale"][pg[None], heads[:, None], row[None]][..., None]


def _pieces(st, b, keys):
    """(heads h0 .. h1, new tokens t0 .. t1) of sequence b, as many scores at a time as are held."""
    H, m = st["case"]["H"], st["new"][b]
    tokens = min(m, max(1, SCORES // (keys * st["case"]["G"])))
    step = min(H, max(1, SCORES // (keys * st["case"]["G"] * tokens)))
    for h in range(0, H, step):
        yield h, min(H, h + step), [(t, min(m, t + tokens)) for t in range(0, m, tokens)]


def _scores(st, b, pos, k, h0, h1, t0, t1):
    """fp32 scores [heads, (t1 - t0) G, keys] of the new tokens t0 .. t1 of sequence b, -inf where a key is not met."""
    c = st["case"]
    G, first = c["G"], sum(st["new"][:b])
    q = st["q"][first + t0:first + t1, h0 * G:h1 * G].float()
    q = q.view(t1 - t0, h1 - h0, G, c["D"]).transpose(0, 1).reshape(h1 - h0, -1, c["D"])
    s = torch.matmul(q, k.transpose(1, 2)) * (1.0 / math.sqrt(c["D"]))
    i = (st["lens"][b] - st["new"][b] + torch.arange(t0, t1, device=q.device)).repeat_interleave(G)[:, None]
    off = pos > i
    if c["window"]:
        off |= (i - pos >= c["window"]) & (pos >= c["sinks"])
    return s.masked_fill_(off, -math.inf)


def _plain_prefill(st, lse_only=False):
    c = st["case"]
    H, G, D = c["H"], c["G"], c["D"]
    lse = torch.empty((st["q"].shape[0], H * G), device=st["q"].device, dtype=torch.float32)
    out = None if lse_only else torch.empty_like(st["q"])
    first = 0
    for b in range(c["B"]):
        pos, pg, row = _seen(st, b)
        for h0, h1, tokens in _pieces(st, b, len(pos)):
            heads = torch.arange(h0, h1, device=pos.device)
            k = _values(st, "k", pg, row, heads)
            v = None if lse_only else _values(st, "v", pg, row, heads)
            for t0, t1 in tokens:
                s = _scores(st, b, pos, k, h0, h1, t0, t1)
                m = s.amax(-1, keepdim=True)
                e = torch.exp(s.sub_(m))
                l = e.sum(-1, keepdim=True)
                at = slice(first + t0, first + t1), slice(h0 * G, h1 * G)
                lse[at] = (m + torch.log(l)).view(h1 - h0, t1 - t0, G).transpose(0, 1).reshape(t1 - t0, -1)
                if out is not None:
                    o = (torch.matmul(e, v) / l).view(h1 - h0, t1 - t0, G, D).transpose(0, 1)
                    out[at] = o.reshape(t1 - t0, -1, D).to(out.dtype)
        first += st["new"][b]
    return lse if lse_only else {"out": out, "lse": lse}


def _plain_weigh(st):
    c = st["case"]
    G, first = c["G"], 0
    for b in range(c["B"]):
        pos, pg, row = _seen(st, b)
        for h0, h1, tokens in _pieces(st, b, len(pos)):
            heads = torch.arange(h0, h1, device=pos.device)
            k = _values(st, "k", pg, row, heads)
            w = torch.zeros((h1 - h0, len(pos)), device=pos.device)
            for t0, t1 in tokens:
                s = _scores(st, b, pos, k, h0, h1, t0, t1)
                lse = st["lse"][first + t0:first + t1, h0 * G:h1 * G]
                lse = lse.view(t1 - t0, h1 - h0, G).transpose(0, 1).reshape(h1 - h0, -1, 1)
                w += torch.exp(s.sub_(lse)).sum(1)
            st["weights"][pg[None], heads[:, None], row[None]] = w
        first += st["new"][b]
    return {"weights": st["weights"]}


def _plain_evict(st):
    c = st["case"]
    H, page, keep = c["H"], c["page"], c["keep"]
    dev = st["weights"].device
    kept = torch.full((c["B"], H, keep), -1, device=dev, dtype=torch.int32)
    heads = torch.arange(H, device=dev)[:, None]
    for b, n in enumerate(st["lens"]):
        p = torch.arange(n, device=dev)
        m = min(n, keep)
        w = st["weights"][st["page_table"][b].long()[p // page], :, p % page].t().contiguous()
        # the first and the newest keys first, then by weight; equal ones in the order of their positions
        w[:, (p < c["sinks"]) | (p >= n - c["recent"])] = math.inf
        at = torch.sort(w, dim=1, descending=True, stable=True).indices[:, :m].sort(dim=1).values     # [H, m]
        kept[b, :, :m] = at.to(torch.int32)
        src_pg, src_row = st["page_table"][b].long()[at // page], at % page
        to = torch.arange(m, device=dev)
        dst_pg, dst_row = st["out_table"][b].long()[to // page][None], (to % page)[None]
        for name in ("k", "v"):
            codes = st[name].view(torch.uint8)
            codes[dst_pg, heads, dst_row] = codes[src_pg, heads, src_row]
        for name in ("k_scale", "v_scale", "weights"):
            st[name][dst_pg, heads, dst_row] = st[name][src_pg, heads, src_row]
    out = {n: st[n] for n in ("k", "v", "k_scale", "v_scale", "weights")}
    out.update(kept=kept, lens=st["seqlens"].clamp(max=keep))
    return out


# ------------------------------------------------------- the package's calls --

def _own(st):
    import block_sparse_flashattention_gb300 as bsa

    c = st["case"]
    if "cache" not in st:                        # what a serving loop keeps from step to step
        st["cache"] = bsa.KVCache(st["k"], st["v"], st["k_scale"], st["v_scale"])
        if c["op"] != "evict":
            st["mask"] = dict(kind=bsa.MASK_CAUSAL)
            if c["window"]:
                st["mask"] = dict(kind=bsa.MASK_SLIDING_WINDOW, mask_params=bsa.MaskParams(
                    window_left=c["window"], sink_tokens=c["sinks"]))
        if c["op"] == "prefill":
            st["keys"] = sum(st["lens"])
            st["workspace"] = bsa.alloc_prefill_workspace(st["cache"], st["q"].shape[0], c["B"], c["H"] * c["G"],
                                                          st["keys"])
    if c["op"] == "prefill":
        out, lse = bsa.prefill(st["q"], st["cache"], st["page_table"], st["seqlens"], st["cu"], keys=st["keys"],
                               workspace=st["workspace"], **st["mask"])
        return {"out": out, "lse": lse}
    if c["op"] == "weigh":
        bsa.kv_weigh(st["q"], st["lse"], st["cache"], st["weights"], st["page_table"], st["seqlens"],
                     cu_seqlens=st["cu"], accumulate=False, **st["mask"])
        return {"weights": st["weights"]}
    kept, lens = bsa.kv_evict(st["cache"], st["weights"], st["page_table"], st["seqlens"], c["keep"],
                              recent=c["recent"], sinks=c["sinks"], out_table=st["out_table"])
    out = {n: st[n] for n in ("k", "v", "k_scale", "v_scale", "weights")}
    out.update(kept=kept, lens=lens)
    return out


def run(state):
    if own:
        return _own(state)
    return {"prefill": _plain_prefill, "weigh": _plain_weigh, "evict": _plain_evict}[state["case"]["op"]](state)


# ---------------------------------------------------------------- work, exact --

def _pairs(c, n, m):
    """(query, key) pairs of a sequence of n keys with m new tokens."""
    if not c["window"]:
        return m * n - m * (m - 1) // 2
    return sum(min(i + 1, c["window"]) + min(c["sinks"], max(0, i + 1 - c["window"])) for i in range(n - m, n))


def work(case):
    c = case
    lens, new = _lengths(c)
    H, D = c["H"], c["D"]
    row = D + 4                                       # codes and scale of one cached row of one head
    if c["op"] == "evict":
        kept = sum(min(n, c["keep"]) for n in lens)   # rows and weights in and out, kept positions out; all weights in
        return {"bytes": H * (sum(lens) * 4 + kept * (2 * 2 * row + 4 + 4)), "flops": 0}
    seen = sum(n - f + s for n, m in zip(lens, new) for s, f in [_first_seen(c, n, m)])
    pairs = sum(_pairs(c, n, m) for n, m in zip(lens, new))
    rows = sum(new) * H * c["G"]
    if c["op"] == "prefill":
        return {"bytes": seen * H * 2 * row + rows * (4 * D + 4), "flops": 4 * H * c["G"] * D * pairs}
    return {"bytes": seen * H * (row + 4) + rows * (2 * D + 4), "flops": 2 * H * c["G"] * D * pairs}


def exact(case, seed):
    """The operators' definitions in 64 bits, one sequence, head and block of queries at a time."""
    c = case
    lens, new = _lengths(c)
    H, D, page, f64 = c["H"], c["D"], c["page"], torch.float64
    st = prepare(case, seed)
    table = st["page_table"].tolist()
    if c["op"] == "evict":
        res = {n: st[n].view(torch.uint8).clone().view(st[n].dtype).to(torch.float32).to(f64) for n in ("k", "v")}
        res.update({n: st[n].to(f64) for n in ("k_scale", "v_scale", "weights")})
        if res["k"].numel() > 1 << 30:                # too much to hold in 64 bits
            res = {n: res[n] for n in ("k_scale", "v_scale", "weights")}
        out = st["out_table"].tolist()
        kept = torch.full((c["B"], H, c["keep"]), -1, dtype=torch.int32, device="cuda")
        for b, n in enumerate(lens):
            own_pages = torch.tensor(table[b][:_cdiv(n, page)], device="cuda")
            w = res["weights"][own_pages].transpose(0, 1).reshape(H, -1)[:, :n].clone()
            m = min(n, c["keep"])
            new_pages = torch.tensor(out[b][:_cdiv(m, page)], device="cuda")
            for h in range(H):
                forced = torch.zeros(n, dtype=torch.bool, device="cuda")
                forced[:c["sinks"]] = True
                forced[max(0, n - c["recent"]):] = True
                others = torch.nonzero(~forced).flatten()
                rest = m - int(forced.sum())
                if rest > 0:
                    order = torch.argsort(-w[h][others], stable=True)
                    forced[others[order[:rest]]] = True
                pos = torch.nonzero(forced).flatten()[:m]
                kept[b, h, :m] = pos.to(torch.int32)
                to = torch.arange(m, device="cuda")
                for name in res:
                    res[name][new_pages[to // page], h, to % page] = res[name][own_pages[pos // page], h, pos % page]
        res.update(kept=kept, lens=torch.tensor([min(n, c["keep"]) for n in lens], dtype=torch.int32, device="cuda"))
        return {n: res.get(n) for n in ("k", "v", "k_scale", "v_scale", "weights", "kept", "lens")}

    def cached(name, b, h, lo, hi):
        """Rows lo .. hi of sequence b, head h, whole pages at a time."""
        pages = torch.tensor(table[b][lo // page:_cdiv(hi, page)], device="cuda", dtype=torch.long)
        codes = st[name].view(torch.uint8)[pages, h].view(st[name].dtype).to(torch.float32).to(f64)
        x = (codes * st[name + "_scale"][pages, h].to(f64)[..., None]).reshape(-1, D)
        return x[lo - lo // page * page:][:hi - lo]

    G = c["G"]
    lse = torch.empty((sum(new), H * G), dtype=f64, device="cuda")
    out = torch.empty((sum(new), H * G, D), dtype=f64, device="cuda")
    weights = st["weights"].to(f64) if c["op"] == "weigh" else None
    first = 0
    for b, (n, m) in enumerate(zip(lens, new)):
        block = max(1, (1 << 27) // (max(n, 1) * G))
        for h in range(H):
            for t0 in range(0, m, block):
                t1 = min(m, t0 + block)
                i = torch.arange(n - m + t0, n - m + t1, device="cuda")
                lo = max(0, n - m + t0 - c["window"] + 1) if c["window"] else 0
                hi = n - m + t1
                spans = [(0, min(c["sinks"], lo)), (lo, hi)] if c["window"] else [(0, hi)]
                at = torch.cat([torch.arange(x, y, device="cuda") for x, y in spans])
                k = torch.cat([cached("k", b, h, x, y) for x, y in spans if y > x])
                q = st["q"][first + t0:first + t1, h * G:(h + 1) * G].to(f64)
                s = torch.einsum("tgd,kd->tgk", q, k) / math.sqrt(D)
                ok = at[None] <= i[:, None]
                if c["window"]:
                    ok = ok & ((i[:, None] - at[None] < c["window"]) | (at[None] < c["sinks"]))
                s = torch.where(ok[:, None], s, torch.full_like(s, -math.inf))
                rows = slice(first + t0, first + t1), slice(h * G, (h + 1) * G)
                if weights is not None:
                    w = torch.exp(s - st["lse"][rows].to(f64)[..., None]).sum((0, 1))
                    pg = torch.tensor(table[b], device="cuda")[at // page]
                    before = weights[pg, h, at % page] if t0 else 0.0
                    weights[pg, h, at % page] = before + w
                    continue
                lse[rows] = torch.logsumexp(s, -1)
                v = torch.cat([cached("v", b, h, x, y) for x, y in spans if y > x])
                out[rows] = torch.einsum("tgk,kd->tgd", torch.exp(s - lse[rows][..., None]), v)
        first += m
    return {"weights": weights} if weights is not None else {"out": out, "lse": lse}
