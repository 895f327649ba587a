"""kv_weigh and kv_evict against the oracle at the sizes and masks where they can go wrong."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import block_sparse_flashattention_gb300 as bsa  # noqa: E402
from oracle import kv_cache as okv  # noqa: E402
from tests.chunk_case import Chunks, i32  # noqa: E402
from tests.kv_case import Pool, pages_for  # noqa: E402

pytestmark = pytest.mark.gpu


def _err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _lse(c):
    """The oracle's lse as a program has it, in 32 bits."""
    return torch.from_numpy(c.expect()[1].astype(np.float32)).cuda()


def _weigh(c, lse, weights=None, **kw):
    w = bsa.alloc_kv_weights(c.pool.cache) if weights is None else weights
    err = _err()
    got = bsa.kv_weigh(c.q, lse, c.pool.cache, w, c.table, c.seqlens, err_flag=err,
                       **{**c.kw, "cu_seqlens": c.cu, **kw})
    assert got is w
    return w, int(err)


def _near(w, ref, before=0.0):
    want, tol = ref
    on = ~np.isnan(want)
    got = w.cpu().numpy().astype(np.float64)
    diff = np.abs(got - before - want)[on]
    bad = diff > tol[on] + 2.0 ** -23 * abs(before)
    assert not bad.any(), (diff[bad][:4], want[on][bad][:4], tol[on][bad][:4])
    assert (got[~on] == before).all()


SHAPES = [
    # dtype, H, G, D, page, lens, news
    ("e4m3", 1, 1, 128, 128, [1], [1]),
    ("int8", 2, 1, 64, 16, [0, 1, 2, 15, 16, 17], [0, 1, 1, 3, 16, 2]),
    ("e4m3", 3, 4, 128, 64, [127, 128, 129, 0, 640], [1, 4, 129, 0, 33]),
    ("int8", 2, 5, 128, 32, [300, 31, 33], [60, 31, 1]),
    ("e4m3", 1, 16, 64, 64, [400], [1]),
    ("int8", 1, 17, 128, 128, [200, 3], [1, 3]),
    ("e4m3", 1, 128, 64, 128, [300], [3]),
    ("int8", 1, 3, 128, 16, [1100, 70], [500, 43]),
    ("e4m3", 2, 2, 64, 128, [2500], [64]),
    ("int8", 1, 7, 128, 64, [900, 12, 500], [0, 5, 100]),
]


@pytest.mark.parametrize("dtype,H,G,D,page,lens,news", SHAPES)
def test_weigh(dtype, H, G, D, page, lens, news):
    c = Chunks(61, dtype, H, G, D, page, lens, news)
    lse = _lse(c)
    ref = c.expect_weights(lse)
    w, err = _weigh(c, lse)
    assert err == 0
    _near(w, ref)
    w, _ = _weigh(c, lse, torch.full_like(w, 3.0))
    _near(w, ref, before=3.0)
    w, _ = _weigh(c, lse, torch.full_like(w, 3.0), accumulate=False)
    on = torch.from_numpy(~np.isnan(ref[0])).cuda()
    assert (w[~on] == 3.0).all()
    _near(torch.where(on, w, torch.zeros_like(w)), ref)


@pytest.mark.parametrize("mask", [
    dict(kind=bsa.MASK_NONE), dict(kind=bsa.MASK_SLIDING_WINDOW, window=1), dict(kind=bsa.MASK_SLIDING_WINDOW, window=0),
    dict(kind=bsa.MASK_SLIDING_WINDOW, window=0, sinks=3), dict(kind=bsa.MASK_SLIDING_WINDOW, window=100, sinks=130),
    dict(kind=bsa.MASK_SLIDING_WINDOW, window=2 ** 31 - 1), dict(kind=bsa.MASK_PREFIX, prefix=500)])
@pytest.mark.parametrize("dtype,H,G,D,page,lens,news", [
    ("e4m3", 2, 2, 128, 64, [700, 129, 1], [40, 129, 1]), ("int8", 1, 3, 64, 16, [1100, 300], [350, 2])])
def test_weigh_masks(mask, dtype, H, G, D, page, lens, news):
    c = Chunks(62, dtype, H, G, D, page, lens, news, **mask)
    lse = _lse(c)
    w, err = _weigh(c, lse, accumulate=False)
    assert err == 0
    _near(w, c.expect_weights(lse))


@pytest.mark.parametrize("G", [1, 4, 9])
def test_weigh_single_tokens(G):
    """A decoding step's queries without offsets: with them, and what decode's lse makes of it."""
    lens = [300, 1, 0, 77, 1000]
    c = Chunks(63, "int8", 2, G, 128, 64, lens, [1] * 5)
    out, lse = bsa.decode(c.q, c.pool.cache, c.table, c.seqlens)
    a, err = _weigh(c, lse, cu_seqlens=None)
    b, _ = _weigh(c, lse)
    assert err == 0 and torch.equal(a, b)
    assert abs(float(a.double().sum()) - 4 * 2 * G) < 1e-4 * 8 * G           # every query's weights sum to 1
    _near(a, c.expect_weights(lse))


def test_weigh_the_last_tokens_of_a_prompt():
    c = Chunks(64, "e4m3", 2, 4, 128, 128, [1500], [600])
    out, lse = bsa.prefill(c.q, c.pool.cache, c.table, c.seqlens, c.cu, keys=1500, **c.kw)
    d = Chunks(64, "e4m3", 2, 4, 128, 128, [1500], [32])
    d.q.copy_(c.q[-32:])
    w, err = _weigh(d, lse[-32:])
    assert err == 0
    _near(w, d.expect_weights(lse[-32:]))


def test_weigh_shared_pages_add_up():
    c = Chunks(65, "e4m3", 1, 2, 64, 64, [128, 128], [5, 9])
    lse = _lse(c)
    one, _ = _weigh(c, lse)
    table = c.table.clone()
    table[1] = table[0]                                              # both sequences are the first one's keys
    d = Chunks(65, "e4m3", 1, 2, 64, 64, [128, 128], [5, 9])
    d.table, d.host_table = table, table.cpu().numpy()
    w, _ = _weigh(d, lse)
    total = 0.0
    for b in range(2):
        q, k, _, mask, _ = d.parts(b, 0)
        total = total + okv.weigh(q, lse[d.first[b]:d.first[b + 1]].cpu().numpy().reshape(-1).astype(float), k, mask, d.scale)
    got = w[table[0].long(), 0].reshape(-1).cpu().numpy()
    assert np.allclose(got, total, rtol=1e-4, atol=1e-30)


def test_weigh_faults():
    c = Chunks(66, "int8", 2, 2, 128, 32, [200, 100, 64, 90], [30, 40, 64, 10])
    lse = _lse(c)
    base, _ = _weigh(c, lse)
    for lens, cu in [([200, 39, 64, 90], None), ([200, c.table.shape[1] * 32 + 1, 64, 90], None),
                     (c.lens, [0, 30, 20, 134, 144])]:
        w = torch.zeros_like(base)
        err = _err()
        bsa.kv_weigh(c.q, lse, c.pool.cache, w, c.table, i32(lens), cu_seqlens=i32(cu or c.first.tolist()), err_flag=err, **c.kw)
        assert int(err) == bsa.FLAG_BAD_SEQLENS
        bad = c.table[1][:4].long()
        assert not w[bad].any()                                      # the second sequence's pages
        if cu is None:
            ok = c.table[2][:2].long()
            assert torch.equal(w[ok], base[ok])
    c.host_table[0, 3], c.host_table[3, 0] = -1, 10 ** 6
    c.table.copy_(torch.from_numpy(c.host_table))
    w, err = _weigh(c, lse)
    assert err == bsa.FLAG_BAD_INDEX
    _near(w, c.expect_weights(lse))


def test_weigh_nan_and_infinite():
    c = Chunks(67, "e4m3", 1, 1, 64, 16, [50, 50], [4, 30])
    lse = _lse(c)
    lse[0] = -math.inf                                               # a query without weight
    ref = c.expect_weights(lse)
    pg, row = c.host_table[1][20 // 16], 20 % 16
    c.pool.cache.k_scale[pg, 0, row] = math.nan
    w, _ = _weigh(c, lse)
    assert math.isnan(float(w[pg, 0, row])) and int(torch.isnan(w).sum()) == 1
    w[pg, 0, row] = float(ref[0][pg, 0, row])
    _near(w, ref)
    lse[2] = math.nan                                                # query 2 of the first sequence: its keys 0 .. 48
    w, _ = _weigh(c, lse)
    pos = np.arange(49)
    assert torch.isnan(w[c.table[0].long()[pos // 16], 0, pos % 16]).all()


def test_weigh_strides_graph_and_stream():
    c = Chunks(68, "int8", 2, 3, 64, 32, [400, 90], [300, 4])
    lse = _lse(c)
    base, _ = _weigh(c, lse, accumulate=False)
    wide = torch.randn(304, 3 * 6 * 64 + 8, device="cuda").to(torch.bfloat16)
    q = wide[:, 8:8 + 6 * 64].unflatten(1, (6, 64))
    q.copy_(c.q)
    w = torch.zeros_like(base)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    bsa.kv_weigh(q, lse, c.pool.cache, w, c.table, c.seqlens, cu_seqlens=c.cu, stream=side, **c.kw)
    side.synchronize()
    assert torch.equal(w, base)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bsa.kv_weigh(q, lse, c.pool.cache, w, c.table, c.seqlens, cu_seqlens=c.cu, accumulate=False, **c.kw)
    w.fill_(5)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    on = base != 0
    assert torch.equal(w[on], base[on])


# ------------------------------------------------------------------ eviction --

def _state(pool, weights):
    """(codes K, V, scales K, V, weights) of a pool on the host, as bits."""
    return [t.view(torch.uint8 if t.element_size() == 1 else torch.int32).cpu().numpy().copy()
            for t in (pool.cache.k, pool.cache.v, pool.cache.k_scale, pool.cache.v_scale, weights)]


def _evict_case(seed, dtype, H, D, page, lens, keep, ties=False, extra=0):
    pool = Pool(seed, pages_for(lens, page) + pages_for([min(n, keep) for n in lens], page) + 1 + extra, H, D, page, dtype)
    ht, table = pool.tables(lens)
    rng = np.random.default_rng(seed + 1)
    shape = pool.scales["k"].shape
    w = rng.integers(0, 4, shape).astype(np.float32) if ties else np.exp(rng.standard_normal(shape)).astype(np.float32)
    return pool, ht, table, torch.from_numpy(w).cuda()


def _evict_check(pool, ht, lens, weights, before, keep, recent, sinks, out_host, kept, new_lens, cols=None):
    """Kept positions, lengths and every byte of the cache and the weights after an eviction."""
    page, H = pool.page, pool.H
    want = [x.copy() for x in before]
    in_place = out_host is None
    dst = ht if in_place else out_host
    wf = before[4].view(np.float32)
    kept, new_lens = kept.cpu().numpy(), new_lens.cpu().numpy()
    pages = len(before[0])
    for b, n in enumerate(lens):
        n = max(n, 0)
        m = min(n, keep)
        assert new_lens[b] == m
        for h in range(H):
            ws = [float(wf[ht[b, j // page], h, j % page]) if 0 <= ht[b, j // page] < pages else None for j in range(n)]
            pos = okv.evict(ws, keep, recent, sinks)
            assert kept[b, h, :m].tolist() == pos.tolist() and (kept[b, h, m:] == -1).all()
            for i, j in enumerate(pos):
                to, at = dst[b, i // page], ht[b, j // page]
                if not 0 <= to < pages or (in_place and i == j):
                    continue
                for x, y in zip(want, before):
                    x[to, h, i % page] = y[at, h, j % page] if 0 <= at < pages else 0
            if in_place:
                for j in range(m, n):
                    if 0 <= ht[b, j // page] < pages:
                        want[4][ht[b, j // page], h, j % page] = 0
    for name, x, y in zip(("k", "v", "k_scale", "v_scale", "weights"), want, _state(pool, weights)):
        assert np.array_equal(x, y), name


EVICT = [
    # dtype, H, D, page, lens, keep, recent, sinks
    ("e4m3", 1, 128, 128, [1], 1, 0, 0),
    ("int8", 2, 64, 16, [0, 1, 5, 16, 17, 100], 8, 2, 1),
    ("e4m3", 3, 128, 64, [127, 128, 129, 640], 128, 16, 4),
    ("int8", 1, 128, 32, [300, 31, 33], 32, 32, 0),
    ("e4m3", 2, 64, 128, [2500, 1000], 700, 0, 0),
    ("int8", 2, 128, 16, [3000], 2999, 100, 100),
    ("e4m3", 1, 64, 64, [5000, 60, 4097], 1, 0, 1),
    ("int8", 1, 64, 16, [1025], 1024, 1, 0),
    ("e4m3", 4, 128, 128, [1500, 1500], 513, 513, 0),
]


@pytest.mark.parametrize("dtype,H,D,page,lens,keep,recent,sinks", EVICT)
@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("in_place", [True, False])
def test_evict(dtype, H, D, page, lens, keep, recent, sinks, ties, in_place):
    pool, ht, table, w = _evict_case(71, dtype, H, D, page, lens, keep, ties)
    out_host, out = (None, None) if in_place else pool.tables([min(n, keep) for n in lens])
    before, err = _state(pool, w), _err()
    kept, new = bsa.kv_evict(pool.cache, w, table, i32(lens), keep, recent=recent, sinks=sinks, out_table=out, err_flag=err)
    assert int(err) == 0
    _evict_check(pool, ht, lens, w, before, keep, recent, sinks, out_host, kept, new)


@pytest.mark.parametrize("in_place", [True, False])
def test_evict_odd_weights(in_place):
    """NaN, infinities, zeros of both signs and equal weights."""
    lens, keep = [600, 64], 40
    pool, ht, table, w = _evict_case(72, "int8", 2, 64, 32, lens, keep)
    rng = np.random.default_rng(73)
    odd = np.array([math.nan, math.inf, -math.inf, 0.0, -0.0, 1e-45, -1.0, 3e38], np.float32)
    w.copy_(torch.from_numpy(odd[rng.integers(0, len(odd), w.shape)]))
    for share in (1.0, 0.02):                            # many of each kind, then few that stand out
        if share < 1:
            x = np.where(rng.random(w.shape) < share, odd[rng.integers(0, len(odd), w.shape)], np.float32(0.5))
            w.copy_(torch.from_numpy(x.astype(np.float32)))
        out_host, out = (None, None) if in_place else pool.tables([min(n, keep) for n in lens]) if share == 1 else (out_host, out)
        before = _state(pool, w)
        kept, new = bsa.kv_evict(pool.cache, w, table, i32(lens), keep, recent=3, sinks=2, out_table=out)
        _evict_check(pool, ht, lens, w, before, keep, 3, 2, out_host, kept, new)


@pytest.mark.parametrize("in_place", [True, False])
def test_evict_faults(in_place):
    lens, keep = [200, 100, 150], 60
    pool, ht, table, w = _evict_case(74, "e4m3", 2, 64, 16, lens, keep)
    out_host, out = (None, None) if in_place else pool.tables([60] * 3)
    ht[0, 2], ht[2, 9], ht[2, 0] = -1, 10 ** 6, -3
    if not in_place:
        out_host[1, 1] = 10 ** 6
        out.copy_(torch.from_numpy(out_host))
    table.copy_(torch.from_numpy(ht))
    before, err = _state(pool, w), _err()
    kept, new = bsa.kv_evict(pool.cache, w, table, i32(lens), keep, recent=5, out_table=out, err_flag=err)
    assert int(err) == bsa.FLAG_BAD_INDEX
    _evict_check(pool, ht, lens, w, before, keep, 5, 0, out_host, kept, new)
    # a sequence that outgrows its table, one without keys
    before, err = _state(pool, w), _err()
    kept, new = bsa.kv_evict(pool.cache, w, table, i32([table.shape[1] * 16 + 1, -5, 2 ** 31 - 1]), keep, out_table=out, err_flag=err)
    assert int(err) == bsa.FLAG_BAD_SEQLENS and new.tolist() == [0, 0, 0] and (kept == -1).all()
    for x, y in zip(before, _state(pool, w)):
        assert np.array_equal(x, y)


def test_evict_shared_source_pages():
    """Two sequences behind one common prefix move to pages of their own."""
    page, keep = 32, 70
    pool, ht, table, w = _evict_case(75, "int8", 2, 128, page, [200, 200], keep, extra=8)
    ht[1, :3] = ht[0, :3]
    table.copy_(torch.from_numpy(ht))
    out_host, out = pool.tables([keep, keep])
    before = _state(pool, w)
    kept, new = bsa.kv_evict(pool.cache, w, table, i32([200, 190]), keep, recent=10, out_table=out)
    _evict_check(pool, ht, [200, 190], w, before, keep, 10, 0, out_host, kept, new)


def test_evict_many_sequences_and_strides():
    lens = [(7 * i) % 50 for i in range(300)]
    pool, ht, table, w = _evict_case(76, "e4m3", 1, 64, 16, lens, 20)
    wide = torch.full((300, table.shape[1] + 3), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    before = _state(pool, w)
    kept, new = bsa.kv_evict(pool.cache, w, wide[:, :table.shape[1]], i32(lens), 20, recent=4)
    _evict_check(pool, ht, lens, w, before, 20, 4, 0, None, kept, new)


def test_evict_graph_and_stream():
    lens, keep = [900, 300], 256
    pool, ht, table, w = _evict_case(77, "int8", 2, 128, 64, lens, keep)
    out_host, out = pool.tables([keep, keep])
    before = _state(pool, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kept, new = bsa.kv_evict(pool.cache, w, table, i32(lens), keep, recent=8, out_table=out, stream=side)
    side.synchronize()
    _evict_check(pool, ht, lens, w, before, keep, 8, 0, out_host, kept, new)
    lens_t = i32(lens)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        k2, n2 = bsa.kv_evict(pool.cache, w, table, lens_t, keep, recent=8, out_table=out)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(k2, kept) and torch.equal(n2, new)
    _evict_check(pool, ht, lens, w, before, keep, 8, 0, out_host, k2, n2)


# ------------------------------------------------------------ used together --

def test_a_bounded_cache_serves():
    """Prompts are appended and attended chunk by chunk, their keys weighed; the cache is bounded and decoding
    goes on over what is left: every step against the oracle over the rows that the cache then holds."""
    H, G, D, page, keep = 2, 2, 64, 32, 150
    rng = np.random.default_rng(80)
    pool = Pool(81, 64, H, D, page, "int8")
    table = torch.from_numpy(np.array([pool.take(16), pool.take(16)], np.int32)).cuda()
    w = bsa.alloc_kv_weights(pool.cache)
    lens = [0, 0]

    def rows(m, heads):
        return torch.from_numpy(rng.standard_normal((m, heads, D)).astype(np.float32)).to(torch.bfloat16).cuda()

    def refresh():
        pool.codes = {"k": pool.cache.k.view(torch.uint8).cpu().numpy(), "v": pool.cache.v.view(torch.uint8).cpu().numpy()}
        pool.scales = {"k": pool.cache.k_scale.cpu().numpy(), "v": pool.cache.v_scale.cpu().numpy()}

    def step(new):
        nonlocal lens, w
        lens = [n + m for n, m in zip(lens, new)]
        cu = i32([0, new[0], sum(new)])
        bsa.kv_append(rows(sum(new), H), rows(sum(new), H), pool.cache, table, i32(lens), cu_seqlens=cu)
        refresh()
        c = Chunks.__new__(Chunks)
        c.H, c.G, c.D, c.lens, c.news, c.pool = H, G, D, lens, new, pool
        c.host_table, c.table, c.first = table.cpu().numpy(), table, np.array([0, new[0], sum(new)])
        c.q, c.scale, c.mask_args = rows(sum(new), H * G), D ** -0.5, (bsa.MASK_CAUSAL, 0, 0, 0)
        if max(new) == 1:
            out, lse = bsa.decode(c.q, pool.cache, table, i32(lens), out_dtype=torch.float32)
        else:
            out, lse = bsa.prefill(c.q, pool.cache, table, i32(lens), cu, keys=sum(lens), out_dtype=torch.float32)
        from tests.kv_case import agree
        agree(out, lse, c.expect())
        before = w.cpu().numpy().astype(np.float64)
        bsa.kv_weigh(c.q, lse, pool.cache, w, table, i32(lens), cu_seqlens=cu)
        want, tol = c.expect_weights(lse)
        on = ~np.isnan(want)
        got = w.cpu().numpy().astype(np.float64)
        assert np.all(np.abs(got - before - want)[on] <= tol[on] + 2.0 ** -23 * np.abs(before + want)[on])
        assert np.array_equal(got[~on], before[~on])

    for new in ([200, 90], [130, 3], [40, 40]):
        step(new)
    before = _state(pool, w)
    kept, t = bsa.kv_evict(pool.cache, w, table, i32(lens), keep, recent=32, sinks=4)
    _evict_check(pool, table.cpu().numpy(), lens, w, before, keep, 32, 4, None, kept, t)
    lens = t.tolist()
    assert lens == [150, 133]
    for new in ([1, 1], [1, 1], [20, 1]):
        step(new)
