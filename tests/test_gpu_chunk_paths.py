"""The variants of prefill, kv_weigh and kv_evict that sizes choose, and calls side by side; tolerances as derived in
chunk_case.Chunks."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import block_sparse_flashattention_gb300 as bsa  # noqa: E402
from oracle import kv_cache as okv  # noqa: E402
from tests.chunk_case import Chunks, i32  # noqa: E402
from tests.kv_case import agree  # noqa: E402
from tests.test_gpu_kv_weights import _evict_case, _evict_check, _lse, _near, _state, _weigh  # noqa: E402
from tests.test_gpu_prefill import _run  # noqa: E402

pytestmark = pytest.mark.gpu

WINDOWS = [dict(), dict(kind=bsa.MASK_SLIDING_WINDOW, window=37, sinks=20), dict(kind=bsa.MASK_PREFIX, prefix=70)]


def _check_weigh(c, **kw):
    lse = _lse(c)
    w, err = _weigh(c, lse, accumulate=False, **kw)
    assert err == 0
    _near(w, c.expect_weights(lse))
    w, err = _weigh(c, lse, torch.full_like(w, 2.0), **kw)
    _near(w, c.expect_weights(lse), before=2.0)


def _check_prefill(c, **kw):
    out, lse, err = _run(c, out_dtype=torch.float32, **kw)
    assert err == 0
    agree(out, lse, c.expect())


# Query rows of a KV head and sequence in the mean: each width of both kernels' products.
@pytest.mark.parametrize("mask", WINDOWS)
@pytest.mark.parametrize("G,m", [(1, 1), (3, 2), (8, 1), (9, 1), (4, 4), (5, 5), (16, 2), (11, 3), (2, 31), (13, 9)])
@pytest.mark.parametrize("dtype,D,page", [("e4m3", 128, 16), ("int8", 64, 128), ("int8", 128, 32)])
def test_weigh_rows(mask, G, m, dtype, D, page):
    c = Chunks(11, dtype, 2, G, D, page, [333, m, 70 + m, 16], [m, m, m, min(m, 16)], **mask)
    _check_weigh(c)


@pytest.mark.parametrize("dtype,D", [("e4m3", 128), ("int8", 64)])
@pytest.mark.parametrize("mask", WINDOWS)
def test_weigh_one_chunk_among_steps(dtype, D, mask):
    """Rows are few in the mean, many in one sequence: its blocks are taken one after the other."""
    lens = [(13 * i) % 90 + 1 for i in range(60)]
    news = [1] * 60
    lens[17], news[17] = 500, 213
    _check_weigh(Chunks(12, dtype, 1, 3, D, 16, lens, news, **mask))


@pytest.mark.parametrize("G", [1, 40])
@pytest.mark.parametrize("B", [129, 700, 2100])
def test_weigh_many_sequences(G, B):
    lens = [(7 * i) % 45 for i in range(B)]
    c = Chunks(13, "int8", 1, G, 64, 16, lens, [min(n, 1) for n in lens])
    _check_weigh(c)


@pytest.mark.parametrize("G", [1, 33])
def test_weigh_nan_codes(G):
    """A NaN code makes its key's weight NaN where a query meets the key, and no other."""
    c = Chunks(14, "e4m3", 1, G, 128, 32, [300], [2], kind=bsa.MASK_SLIDING_WINDOW, window=100, sinks=4)
    lse = _lse(c)
    ref = c.expect_weights(lse)
    bits = c.pool.cache.k.view(torch.uint8)
    at = {j: (int(c.host_table[0][j // 32]), j % 32) for j in (2, 50, 250)}
    for d, (pg, row) in zip((0, 127, 64), at.values()):
        bits[pg, 0, row, d] = 0xff if d else 0x7f
    w, err = _weigh(c, lse, accumulate=False)
    for j, (pg, row) in at.items():
        assert math.isnan(float(w[pg, 0, row])) == (j != 50)
        w[pg, 0, row] = float(ref[0][pg, 0, row])
    _near(w, ref)


@pytest.mark.parametrize("mask", WINDOWS + [dict(kind=bsa.MASK_NONE)])
@pytest.mark.parametrize("G,m", [(1, 16), (8, 2), (4, 8), (3, 11), (16, 4), (5, 25), (2, 64), (2, 65), (1, 300)])
@pytest.mark.parametrize("dtype,D,page", [("e4m3", 64, 16), ("int8", 128, 64)])
def test_prefill_rows(mask, G, m, dtype, D, page):
    c = Chunks(15, dtype, 2, G, D, page, [m + 400, m, m + 129], [m, m, m], **mask)
    _check_prefill(c)


@pytest.mark.parametrize("m", [2, 140])
@pytest.mark.parametrize("B", [129, 650])
def test_prefill_many_sequences(m, B):
    lens = [(7 * i) % 45 + (m if i % 5 else 0) for i in range(B)]
    news = [min(n, m) for n in lens] if m < 100 else [min(n, m) if i % 9 == 0 else 0 for i, n in enumerate(lens)]
    _check_prefill(Chunks(16, "e4m3", 1, 1, 64, 16, lens, news))


def test_prefill_one_chunk_among_steps():
    lens = [(13 * i) % 90 + 1 for i in range(60)]
    news = [1] * 60
    lens[17], news[17] = 700, 600
    _check_prefill(Chunks(17, "int8", 2, 2, 128, 16, lens, news))


@pytest.mark.parametrize("m", [3, 200])
def test_prefill_nan_codes(m):
    """NaN codes reach the queries that meet their key, and no others."""
    c = Chunks(18, "e4m3", 1, 2, 128, 32, [400], [m], kind=bsa.MASK_SLIDING_WINDOW, window=m, sinks=1)
    first = 400 - m
    j = first - m // 2                                       # some of the queries meet it
    met = [i for i in range(m) if first + i - j < m]
    assert 0 < len(met) < m
    pg, row = int(c.host_table[0][j // 32]), j % 32
    far, fr = int(c.host_table[0][0]), 5                     # a key that none meets
    rest = [i for i in range(m) if i not in met]
    o, l, to, tl = c.expect()
    for name in ("k", "v"):
        bits = getattr(c.pool.cache, name).view(torch.uint8)
        kept = int(bits[pg, 0, row, 77])
        if m == 3:
            bits[far, 0, fr, 3] = 0x7f
        bits[pg, 0, row, 77] = 0x7f
        out, lse, err = _run(c, out_dtype=torch.float32)
        bits[pg, 0, row, 77] = kept
        bad = torch.isnan(out[met])
        assert bad.all() if name == "k" else bad[..., 77].all()
        assert torch.isnan(lse[met]).all() == (name == "k")
        if name == "v":
            assert np.all(np.abs(lse[met].cpu().numpy() - l[met]) <= tl[met])
        agree(out[rest], lse[rest], (o[rest], l[rest], to[rest], tl[rest]))


@pytest.mark.parametrize("m", [1, 5, 150])
def test_padded_batch(m):
    """Sequences of length 0 that have rows all the same: 0 and -inf, and no weight."""
    c = Chunks(19, "int8", 2, 2, 64, 32, [0, 200, -3, 170], [m, m, m, m])
    _check_prefill(c)
    _check_weigh(c)


@pytest.mark.parametrize("lens,H,keep,recent,sinks", [
    ([100000], 1, 50000, 100, 4),                            # clusters of 8, all keys in shared memory
    ([100000] + [5] * 200, 1, 99000, 0, 0),                  # one CTA, more keys than it holds
    ([90000, 17] + [3] * 50, 1, 700, 64, 0),                 # two
    ([20000] * 40, 1, 300, 10, 10)])
@pytest.mark.parametrize("in_place", [True, False])
def test_evict_long(lens, H, keep, recent, sinks, in_place):
    pool, ht, table, w = _evict_case(21, "int8", H, 64, 128, lens, keep, ties=True)
    w += torch.rand_like(w).round(decimals=1)                # many equal ones
    out_host, out = (None, None) if in_place else pool.tables([min(n, keep) for n in lens])
    before = _state(pool, w)
    kept, new = bsa.kv_evict(pool.cache, w, table, i32(lens), keep, recent=recent, sinks=sinks, out_table=out)
    wf = before[4].view(np.float32)
    page = 128
    assert new.tolist() == [min(n, keep) for n in lens]
    want = [x.copy() for x in before]
    for b, n in enumerate(lens):
        pos = np.arange(n)
        x = wf[ht[b, pos // page], 0, pos % page]
        free = np.zeros(n, bool)
        free[min(sinks, n):max(n - recent, min(sinks, n))] = True
        m = min(n, keep)
        if n <= keep:
            on = pos
        else:
            order = np.lexsort((pos[free], -x[free].astype(np.float64)))
            on = np.sort(np.concatenate([pos[~free], pos[free][order[:m - (~free).sum()]]]))
        assert np.array_equal(kept[b, 0, :m].cpu().numpy(), on) and (kept[b, 0, m:] == -1).all()
        dst, i = (ht if in_place else out_host), np.arange(m)
        for y, z in zip(want, before):
            y[dst[b, i // page], 0, i % page] = z[ht[b, on // page], 0, on % page]
        if in_place:
            want[4][ht[b, pos[m:] // page], 0, pos[m:] % page] = 0
    for y, z in zip(want, _state(pool, w)):
        assert np.array_equal(y, z)


def test_evict_table_given_twice():
    """out_table the same tensor as page_table: in place."""
    lens, keep = [300, 20, 129], 64
    pool, ht, table, w = _evict_case(22, "e4m3", 2, 128, 32, lens, keep)
    before = _state(pool, w)
    kept, new = bsa.kv_evict(pool.cache, w, table, i32(lens), keep, recent=4, out_table=table)
    _evict_check(pool, ht, lens, w, before, keep, 4, 0, None, kept, new)


@pytest.mark.parametrize("m", [2, 20, 200])
def test_far_pages(m):
    """Pages whose codes lie beyond 2^31 bytes answer as the same rows at the start of a small cache do."""
    H, D, page, n, G = 2, 128, 128, 700, 2
    cols = -(-n // page)
    pages = 2 ** 31 // (H * page * D) + cols
    g = torch.Generator(device="cuda").manual_seed(3)

    def rand(*s):
        return torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)

    k, v, q = rand(n, H, D), rand(n, H, D), rand(m, H * G, D)
    cu_k, cu_q, lens = i32([0, n]), i32([0, m]), i32([n])
    got = []
    for count, first in ((cols, 0), (pages, pages - cols)):
        cache = bsa.alloc_kv_cache(count, H, D, page_size=page, dtype=torch.int8)
        table = torch.arange(first, first + cols, dtype=torch.int32, device="cuda")[None]
        bsa.kv_append(k, v, cache, table, lens, cu_seqlens=cu_k)
        w = bsa.alloc_kv_weights(cache)
        out, lse = bsa.prefill(q, cache, table, lens, cu_q, keys=n)
        bsa.kv_weigh(q, lse, cache, w, table, lens, cu_seqlens=cu_q, accumulate=False)
        before = w[first:].clone()
        kept, new = bsa.kv_evict(cache, w, table, lens, 300, recent=10)
        got.append([out, lse, before, kept, new, w[first:].clone()] +
                   [x[first:first + 3].clone() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale)])
        del cache, w
    for a, b in zip(*got):
        assert torch.equal(a, b)
    torch.cuda.empty_cache()


@pytest.mark.parametrize("m", [1, 30, 200])
def test_two_calls_at_once(m):
    """Calls on two streams, each with a workspace of its own, answer as they do one after the other."""
    cs = [Chunks(30 + i, "e4m3", 2, 2, 128, 64, [1500, 900], [m, m]) for i in range(2)]
    ws = [bsa.alloc_prefill_workspace(c.pool.cache, 2 * m, 2, 4, 2400) for c in cs]

    def calls(c, ws):
        out, lse = bsa.prefill(c.q, c.pool.cache, c.table, c.seqlens, c.cu, keys=2400, workspace=ws)
        w = bsa.kv_weigh(c.q, lse, c.pool.cache, bsa.alloc_kv_weights(c.pool.cache), c.table, c.seqlens, cu_seqlens=c.cu)
        return out, lse, w

    want = [calls(c, x) for c, x in zip(cs, ws)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(calls(cs[i], ws[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for x in got[i]:
            for a, b in zip(x, want[i]):
                assert torch.equal(a, b)


@pytest.mark.parametrize("m", [1, 24, 180])
def test_stream_as_a_number_and_the_plain_call(m):
    """The native call, the one through ctypes and one on another stream, given as a number, are the same."""
    c = Chunks(33, "int8", 2, 2, 64, 32, [400, 250], [m, m])
    ws = bsa.alloc_prefill_workspace(c.pool.cache, 2 * m, 2, 4, 650)
    side = torch.cuda.Stream()
    got = []
    for kw in (dict(), dict(err_flag=i32([0])), dict(stream=side.cuda_stream)):
        torch.cuda.synchronize()
        out, lse = bsa.prefill(c.q, c.pool.cache, c.table, c.seqlens, c.cu, keys=650, workspace=ws, **kw)
        torch.cuda.synchronize()
        w = bsa.alloc_kv_weights(c.pool.cache)
        torch.cuda.synchronize()
        bsa.kv_weigh(c.q, lse, c.pool.cache, w, c.table, c.seqlens, cu_seqlens=c.cu, **kw)
        torch.cuda.synchronize()
        w2, state = w.clone(), [x.clone() for x in (c.pool.cache.k, c.pool.cache.v, c.pool.cache.k_scale, c.pool.cache.v_scale)]
        kept, new = bsa.kv_evict(c.pool.cache, w2, c.table, c.seqlens, 128, recent=8, **kw)
        torch.cuda.synchronize()
        got.append((out, lse, w, w2, kept, new, c.pool.cache.k.clone(), c.pool.cache.v_scale.clone()))
        for x, y in zip((c.pool.cache.k, c.pool.cache.v, c.pool.cache.k_scale, c.pool.cache.v_scale), state):
            x.copy_(y)
    for x in got[1:]:
        for a, b in zip(x, got[0]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("m", [1, 24, 180])
def test_replayed_with_other_lengths(m):
    """A captured call reads lengths, offsets and tables anew."""
    c = Chunks(34, "e4m3", 2, 2, 128, 32, [300, 700, 100 + m], [m, m, m])
    ws = bsa.alloc_prefill_workspace(c.pool.cache, 3 * m, 3, 4, 2000)
    w = bsa.alloc_kv_weights(c.pool.cache)
    g = torch.cuda.CUDAGraph()

    def call():
        out, lse = bsa.prefill(c.q, c.pool.cache, c.table, c.seqlens, c.cu, keys=2000, workspace=ws)
        bsa.kv_weigh(c.q, lse, c.pool.cache, w, c.table, c.seqlens, cu_seqlens=c.cu, accumulate=False)
        return out, lse

    call()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        out, lse = call()
    for lens in ([300, 700, 100 + m], [250, 690, m], [m, 0, 100]):
        c.lens = lens
        c.seqlens.copy_(i32(lens))
        cu = [0, m, 2 * m, 2 * m + min(m, lens[2])]
        c.cu.copy_(i32(cu))
        c.news, c.first = [m, m, min(m, lens[2])], np.array(cu)
        w.zero_()
        g.replay()
        torch.cuda.synchronize()
        end = cu[-1]
        ref = c.expect()
        agree(out[:end], lse[:end], tuple(x[:end] for x in ref))
        _near(w, c.expect_weights(lse))


@pytest.mark.parametrize("m", [2, 100, 300])
def test_offsets_that_go_back_and_forth(m):
    """Sequences that claim the same rows over and over: flagged, and nothing outside the workspace is written."""
    B = 64
    c = Chunks(40, "e4m3", 1, 2, 64, 16, [320] * B, [m] + [0] * (B - 1))
    cu = i32([0 if b % 2 == 0 else m for b in range(B + 1)])
    n = bsa.bsattn_prefill_workspace_size(c.pool.cache.ref, m, B, 2, 320 * B)
    buf = torch.full((n + (1 << 20),), 77, dtype=torch.uint8, device="cuda")
    wide = torch.full((m + 8, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    err = i32([0])
    bsa.prefill(c.q, c.pool.cache, c.table, c.seqlens, cu, keys=320 * B, workspace=buf[:n], out=wide[:m], err_flag=err)
    torch.cuda.synchronize()
    assert int(err) == bsa.FLAG_BAD_SEQLENS
    assert (buf[n:] == 77).all() and (wide[m:] == 5).all()
    w, err = _weigh(c, torch.zeros(m, 2, device="cuda"), cu_seqlens=cu)
    assert err == bsa.FLAG_BAD_SEQLENS
