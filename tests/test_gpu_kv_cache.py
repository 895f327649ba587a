"""kv_append and kv_read against the oracle: codes and scales equal to its values, rows
read back equal to code * scale rounded to bf16, everything else left as it was."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import block_sparse_flashattention_gb300 as bsa  # noqa: E402
from oracle import kv_cache as okv  # noqa: E402
from tests.kv_case import DT, Pool, bf16, f64, pages_for  # noqa: E402

pytestmark = pytest.mark.gpu


def _fill(cache, byte=0x2A, scale=7.5):
    for t in (cache.k, cache.v):
        t.view(torch.uint8).fill_(byte)
    for t in (cache.k_scale, cache.v_scale):
        t.fill_(scale)


def _empty(pages, H, D, page, dtype):
    c = bsa.alloc_kv_cache(pages, H, D, page_size=page, dtype=DT[dtype])
    _fill(c)
    return c


def _host(cache, dtype):
    return {n: (okv.values(getattr(cache, n).view(torch.uint8).cpu().numpy(), dtype),
                getattr(cache, n + "_scale").cpu().numpy().astype(np.float64)) for n in ("k", "v")}


def _rows(rng, T, H, D):
    """bf16 rows of all kinds: normal ones, zeros, tiny and huge ones, a row at e4m3's 448 border."""
    x = rng.standard_normal((T, H, D)) * np.exp(2.0 * rng.standard_normal((T, H, 1)))
    flat = x.reshape(-1, D)
    special = [np.zeros(D), np.full(D, 2.0 ** -133), flat[0] * 1e-38, flat[0] * 1e37,
               np.linspace(-448, 448, D), np.linspace(-450, 450, D), -np.full(D, 3.0 * 2.0 ** 100)]
    for i, s in enumerate(special[:len(flat) // 2]):
        flat[2 * i] = s
    return bf16(x)


CASES = [
    # dtype, H, D, page, lens (after the append), new tokens of each (None: one each, without cu_seqlens), fused rows
    ("e4m3", 1, 128, 128, [1], None, False),
    ("int8", 3, 64, 16, [5, 16, 17, 40], None, True),
    ("e4m3", 16, 128, 64, [100, 0, 65, 64, 63], None, False),
    ("e4m3", 2, 64, 32, [33, 70, 7], [33, 1, 0], True),
    ("int8", 9, 128, 128, [300, 129, 128, 127], [300, 128, 1, 126], False),
    ("e4m3", 8, 64, 16, [3] * 70, [3, 2] * 35, False),
    ("int8", 17, 64, 128, [1], [1], True),
]


@pytest.mark.parametrize("dtype,H,D,page,lens,new,fused", CASES)
def test_append(dtype, H, D, page, lens, new, fused):
    pool = Pool(1, pages_for(lens, page) + 2, 1, 64, page, dtype)   # its tables only
    rng = np.random.default_rng(2)
    host_table, table = pool.tables(lens)
    cache = _empty(len(pool.free) + pages_for(lens, page), H, D, page, dtype)
    before = _host(cache, dtype)
    counts = [1] * len(lens) if new is None else new
    T = sum(counts)
    if fused:
        qkv = _rows(rng, T, 3 * H, D).cuda()
        k, v = qkv[:, H:2 * H], qkv[:, 2 * H:]
    else:
        k, v = _rows(rng, T, H, D).cuda(), _rows(rng, T, H, D).cuda()
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = bsa.kv_append(k, v, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                        cu_seqlens=None if new is None else torch.from_numpy(cu).cuda(), err_flag=err)
    assert got is cache and int(err) == 0
    after = _host(cache, dtype)
    for name, x in (("k", f64(k)), ("v", f64(v))):
        codes, scales = (a.copy() for a in before[name])
        c, s = okv.quantise(x, dtype)
        for b, n in enumerate(lens):
            for i in range(counts[b] if n > 0 else 0):
                p = n - counts[b] + i
                codes[host_table[b, p // page], :, p % page] = c[cu[b] + i]
                scales[host_table[b, p // page], :, p % page] = s[cu[b] + i]
        assert np.array_equal(after[name][1], scales)
        assert np.array_equal(after[name][0], codes)


@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
def test_append_rows_that_are_not_finite(dtype):
    cache = _empty(1, 4, 64, 16, dtype)
    x = np.ones((1, 4, 64), np.float32)
    x[0, 0, 3], x[0, 1, 5], x[0, 2, 7] = np.nan, np.inf, -np.inf
    k = bf16(x).cuda()
    table, n = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    bsa.kv_append(k, k, cache, table, n)
    k2, v2 = bsa.kv_read(cache, table, torch.tensor([0, 1], dtype=torch.int32, device="cuda"), total=1)
    for t in (k2, v2):
        t = t.float().cpu()[0]
        assert t[:3].isnan().all() and (t[3] - 1).abs().max() <= 2.0 ** -8


def test_append_faults_leave_the_cache():
    """Bad pages, lengths and offsets: flagged, nothing else written, the good sequences served."""
    H, D, page, dtype = 2, 64, 16, "int8"
    cases = [  # table row, length, new tokens, expected flag (0: served)
        ([0, 1], 20, 2, 0), ([99, 2], 18, 3, bsa.FLAG_BAD_INDEX), ([-1], 4, 1, bsa.FLAG_BAD_INDEX),
        ([3, 4], 2, 3, bsa.FLAG_BAD_SEQLENS), ([3, 4], 33, 1, bsa.FLAG_BAD_SEQLENS), ([3, 4], 0, 2, 0),
        ([3, 4], -5, 1, 0)]
    for row, n, new, flag in cases:
        cache = _empty(6, H, D, page, dtype)
        table = torch.full((2, 2), 5, dtype=torch.int32)
        table[0, :len(row)] = torch.tensor(row, dtype=torch.int32)
        k = bf16(np.random.default_rng(4).standard_normal((new + 1, H, D))).cuda()
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        bsa.kv_append(k, k, cache, table.cuda(), torch.tensor([n, 9], dtype=torch.int32, device="cuda"),
                      cu_seqlens=torch.tensor([0, new, new + 1], dtype=torch.int32, device="cuda"), err_flag=err)
        assert int(err) == flag, (row, n)
        got = cache.k.cpu().numpy()
        c, _ = okv.quantise(f64(k), dtype)
        assert np.array_equal(got[5, :, 8], c[new])      # the second sequence's token
        written = {(5, 8)}
        if n > 0 and flag != bsa.FLAG_BAD_SEQLENS:
            for i in range(new):
                p = n - new + i
                if 0 <= row[p // page] < 6:
                    assert np.array_equal(got[row[p // page], :, p % page], c[i])
                    written.add((row[p // page], p % page))
        for pg in range(6):
            for r in range(page):
                assert (pg, r) in written or (got[pg, :, r] == 0x2A).all()


@pytest.mark.parametrize("cu", [[0, -1, 4], [0, 3, 2], [0, 2, 5], [-1, 2, 4]])
def test_bad_offsets_are_flagged(cu):
    cache = _empty(2, 2, 64, 16, "e4m3")
    table = torch.tensor([[0], [1]], dtype=torch.int32, device="cuda")
    k = torch.ones((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    bsa.kv_append(k, k, cache, table, torch.tensor([9, 9], dtype=torch.int32, device="cuda"), cu_seqlens=cud, err_flag=err)
    assert int(err) == bsa.FLAG_BAD_SEQLENS
    err.zero_()
    bsa.kv_read(cache, table, cud, total=4, err_flag=err)
    assert int(err) == bsa.FLAG_BAD_SEQLENS


@pytest.mark.parametrize("dtype,H,D,page,lens", [
    ("e4m3", 1, 128, 128, [1]), ("int8", 3, 64, 16, [5, 0, 16, 17, 40]), ("e4m3", 16, 64, 64, [100, 64, 63, 1]),
    ("int8", 9, 128, 32, [300, 129]), ("e4m3", 5, 128, 16, [2] * 40 + [31])])
def test_read(dtype, H, D, page, lens):
    pool = Pool(5, pages_for(lens, page) + 1, H, D, page, dtype)
    host_table, table = pool.tables(lens, cols=max(-(-n // page) for n in lens) + 2)
    cu = np.concatenate([[2], 2 + np.cumsum(lens)]).astype(np.int32)    # rows 0, 1 and the last 3 belong to nobody
    T = int(cu[-1]) + 3
    k, v = (torch.full((T, H, D), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    bsa.kv_read(pool.cache, table, torch.from_numpy(cu).cuda(), k=k, v=v, err_flag=err)
    assert int(err) == 0
    for name, got in (("k", k), ("v", v)):
        want = np.full((T, H, D), 9.0)
        for b, n in enumerate(lens):
            for h in range(H):
                want[cu[b]:cu[b + 1], h] = pool.host(name, host_table[b], h, range(n))
        # code * scale is exact in fp64; the device multiplies in fp32, then rounds: bf16 of an fp32 rounding
        want32 = torch.from_numpy(want.astype(np.float32)).to(torch.bfloat16)
        assert torch.equal(got.cpu(), want32)


def test_read_faults():
    pool = Pool(6, 3, 2, 64, 16, "e4m3")
    table = torch.tensor([[0, 77], [1, 2], [1, 2]], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 20, 53, 55], dtype=torch.int32, device="cuda")     # 20 over a bad page, 33 > 2 pages, 2
    k, v = (torch.full((55, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    bsa.kv_read(pool.cache, table, cu, k=k, v=v, err_flag=err)
    assert int(err) == bsa.FLAG_BAD_INDEX | bsa.FLAG_BAD_SEQLENS
    assert (k[16:20] == 0).all() and (v[16:20] == 0).all() and (k[20:53] == 9.0).all()
    for h in range(2):
        assert np.array_equal(f64(k)[53:, h], pool.host("k", [1, 2], h, range(2)))


@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
def test_append_then_read_is_within_half_a_step(dtype):
    """|x - read| <= half a code step of the row's scale plus the read's bf16 rounding (e4m3: none)."""
    H, D, page, T = 4, 128, 64, 130
    cache = bsa.alloc_kv_cache(3, H, D, page_size=page, dtype=DT[dtype])
    x = bf16(np.random.default_rng(7).standard_normal((T, H, D))).cuda()
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    cu, n = (torch.tensor(a, dtype=torch.int32, device="cuda") for a in ([0, T], [T]))
    bsa.kv_append(x, x, cache, table, n, cu_seqlens=cu)
    k, _ = bsa.kv_read(cache, table, cu, total=T)
    x, k = f64(x), f64(k)
    a = np.abs(x).max(-1, keepdims=True)
    if dtype == "int8":
        tol = a / 127 * 0.5 * (1 + 2.0 ** -20) + 2.0 ** -8 * np.abs(k)
    else:
        s = 2.0 ** np.ceil(np.log2(a / 448))
        tol = np.maximum(2.0 ** -4 * np.abs(x), s * 2.0 ** -10)
    assert np.all(np.abs(x - k) <= tol)


def test_wide_strides_and_other_stream():
    """A table cut from a wider one, token strides above H * D, a stream of its own."""
    H, D, page, lens = 2, 64, 16, [20, 3]
    cache, plain = (_empty(8, H, D, page, "e4m3") for _ in range(2))
    wide = torch.full((2, 9), -1, dtype=torch.int32, device="cuda")
    wide[0, 3:5] = torch.tensor([6, 1], dtype=torch.int32)
    wide[1, 3] = 4
    buf = torch.randn((2, 5, H, D), device="cuda").to(torch.bfloat16)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    bsa.kv_append(buf[:, 1], buf[:, 3], cache, wide[:, 3:5], n, stream=s)
    s.synchronize()
    bsa.kv_append(buf[:, 1].contiguous(), buf[:, 3].contiguous(), plain, wide[:, 3:5].contiguous(), n)
    for name in ("k", "v", "k_scale", "v_scale"):
        assert torch.equal(getattr(cache, name).view(torch.uint8), getattr(plain, name).view(torch.uint8))
    assert not torch.equal(cache.k.view(torch.uint8), _empty(8, H, D, page, "e4m3").k.view(torch.uint8))


@pytest.mark.parametrize("native", [True, False])
def test_calls_without_a_row(native, monkeypatch):
    """No sequence has a new token, no row is read back: nothing happens; offsets that promise rows are flagged."""
    from block_sparse_flashattention_gb300 import kv_cache
    cache = _empty(2, 2, 64, 16, "e4m3")
    if not native:
        monkeypatch.setattr(kv_cache, "_calls", None)
    before = [t.view(torch.uint8).clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    table, n, cu = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([[0], [1], [0]], [3, 0, 16], [0, 0, 0, 0]))
    none = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for e in (None, err):
        assert bsa.kv_append(none, none, cache, table, n, cu_seqlens=cu, err_flag=e) is cache
        for kw in (dict(total=0), dict(k=none.clone(), v=none.clone())):
            k, v = bsa.kv_read(cache, table, cu, err_flag=e, **kw)
            assert k.shape == v.shape == none.shape
    assert int(err) == 0
    assert all(torch.equal(a, t.view(torch.uint8)) for a, t in zip(before, (cache.k, cache.v, cache.k_scale, cache.v_scale)))
    bad = torch.tensor([0, 0, 1, 1], dtype=torch.int32, device="cuda")
    for call in (lambda: bsa.kv_append(none, none, cache, table, n, cu_seqlens=bad, err_flag=err),
                 lambda: bsa.kv_read(cache, table, bad, total=0, err_flag=err)):
        err.zero_()
        call()
        assert int(err) == bsa.FLAG_BAD_SEQLENS
