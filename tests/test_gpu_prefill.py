"""prefill against the oracle at the sizes and masks where it can go wrong; tolerances as derived in
chunk_case.Chunks.expect."""
import math

import pytest

torch = pytest.importorskip("torch")

import block_sparse_flashattention_gb300 as bsa  # noqa: E402
from tests.chunk_case import Chunks, i32  # noqa: E402
from tests.kv_case import agree  # noqa: E402

pytestmark = pytest.mark.gpu


def _run(c, **kw):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = bsa.prefill(c.q, c.pool.cache, c.table, c.seqlens, c.cu, keys=sum(max(n, 0) for n in c.lens),
                           err_flag=err, **{**c.kw, **kw})
    return out, lse, int(err)


SHAPES = [
    # dtype, H, G, D, page, lens, news
    ("e4m3", 1, 1, 128, 128, [1], [1]),
    ("int8", 2, 1, 64, 16, [0, 1, 2, 15, 16, 17], [0, 1, 1, 3, 16, 2]),
    ("e4m3", 3, 4, 128, 64, [127, 128, 129, 0, 640], [1, 4, 129, 0, 33]),
    ("int8", 2, 5, 128, 32, [300, 31, 33], [60, 31, 1]),
    ("e4m3", 2, 8, 64, 128, [257, 1000], [17, 16]),
    ("int8", 1, 3, 128, 16, [513, 70], [171, 43]),
    ("e4m3", 1, 16, 64, 64, [400], [9]),
    ("int8", 1, 17, 128, 128, [200, 3], [8, 3]),
    ("e4m3", 1, 128, 128, 128, [300], [3]),
    ("int8", 1, 100, 64, 64, [140], [2]),
    ("e4m3", 5, 2, 128, 128, [2500], [64]),
    ("int8", 4, 1, 64, 64, [3000, 1, 60], [128, 1, 60]),
    ("e4m3", 1, 1, 128, 16, [5000], [700]),
    ("int8", 1, 4, 128, 128, [1300], [1300]),
    ("e4m3", 2, 1, 64, 32, [1024, 255, 256, 257], [1024, 255, 256, 257]),
    ("int8", 1, 7, 128, 64, [900, 12], [400, 5]),
    ("e4m3", 1, 2, 64, 128, [130] * 40, [1 + 3 * i for i in range(40)]),
]


@pytest.mark.parametrize("dtype,H,G,D,page,lens,news", SHAPES)
def test_causal(dtype, H, G, D, page, lens, news):
    c = Chunks(41, dtype, H, G, D, page, lens, news)
    ref = c.expect()
    out, lse, err = _run(c, out_dtype=torch.float32)
    assert err == 0
    agree(out, lse, ref)
    o16, l16, _ = _run(c)
    assert o16.dtype == torch.bfloat16 and torch.equal(l16, lse)
    assert torch.equal(o16, out.to(torch.bfloat16))


MASKS = [
    dict(kind=bsa.MASK_NONE), dict(kind=bsa.MASK_SLIDING_WINDOW, window=1), dict(kind=bsa.MASK_SLIDING_WINDOW, window=0),
    dict(kind=bsa.MASK_SLIDING_WINDOW, window=0, sinks=3), dict(kind=bsa.MASK_SLIDING_WINDOW, window=100, sinks=130),
    dict(kind=bsa.MASK_SLIDING_WINDOW, window=129), dict(kind=bsa.MASK_SLIDING_WINDOW, window=300, sinks=1),
    dict(kind=bsa.MASK_SLIDING_WINDOW, window=2 ** 31 - 1, sinks=2 ** 31 - 1),
    dict(kind=bsa.MASK_PREFIX, prefix=0), dict(kind=bsa.MASK_PREFIX, prefix=500), dict(kind=bsa.MASK_PREFIX, prefix=2 ** 31 - 1),
]


@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("dtype,H,G,D,page,lens,news", [
    ("e4m3", 2, 2, 128, 64, [700, 129, 1], [40, 129, 1]),
    ("int8", 1, 3, 64, 16, [1100, 300], [350, 2]),
])
def test_masks(mask, dtype, H, G, D, page, lens, news):
    c = Chunks(42, dtype, H, G, D, page, lens, news, **mask)
    out, lse, err = _run(c, out_dtype=torch.float32)
    assert err == 0
    agree(out, lse, c.expect())


def test_single_tokens_are_decode():
    """A chunk of one token each, like a decoding step: the same answers up to their roundings."""
    lens = [300, 1, 77, 1000]
    c = Chunks(43, "int8", 2, 4, 128, 64, lens, [1] * 4)
    out, lse, _ = _run(c, out_dtype=torch.float32)
    ref = c.expect()
    agree(out, lse, ref)
    o, l = bsa.decode(c.q, c.pool.cache, c.table, c.seqlens, out_dtype=torch.float32)
    agree(o, l, ref)


def test_rows_of_no_sequence_stay():
    c = Chunks(44, "e4m3", 1, 2, 64, 16, [40, 300], [5, 260])
    total = 300
    q = torch.zeros(total, 2, 64, dtype=torch.bfloat16, device="cuda")
    q[10:15], q[20:280] = c.q[:5], c.q[5:]
    # offsets with gaps are offsets of three sequences, the middle one (without keys) in between
    cu, lens = i32([10, 15, 20, 280]), i32([40, 0, 300])
    table = torch.stack([c.table[0], c.table[0], c.table[1]])
    out = torch.full((total, 2, 64), 7.0, device="cuda")
    lse = torch.full((total, 2), 7.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    bsa.prefill(q, c.pool.cache, table, lens, cu, keys=340, out=out, lse=lse, err_flag=err)
    assert int(err) == 0
    agree(torch.cat([out[10:15], out[20:280]]), torch.cat([lse[10:15], lse[20:280]]), c.expect())
    assert (out[:10] == 7).all() and (lse[:10] == 7).all() and (out[280:] == 7).all() and (lse[280:] == 7).all()
    assert not out[15:20].any() and torch.isneginf(lse[15:20]).all()      # queries of a sequence without keys


def test_faulty_sequences_are_left_and_flagged():
    c = Chunks(45, "int8", 2, 2, 128, 32, [200, 100, 64, 90], [30, 40, 64, 10])
    base_o, base_l, _ = _run(c, out_dtype=torch.float32)
    first, ref = c.first, c.expect()
    for lens, cu in [([200, 39, 64, 90], None),                             # more new tokens than keys
                     ([200, c.table.shape[1] * 32 + 1, 64, 90], None),      # outgrows the table
                     (c.lens, [0, 30, 20, 134, 144]),                       # offsets decrease
                     (c.lens, [0, 30, 70, 134, 145]), (c.lens, [-1, 30, 70, 134, 144])]:
        out = torch.full_like(base_o, 7.0)
        lse = torch.full_like(base_l, 7.0)
        cu_t = i32(cu or first.tolist())
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        bsa.prefill(c.q, c.pool.cache, c.table, i32(lens), cu_t, keys=2000, out=out, lse=lse, err_flag=err, **c.kw)
        assert int(err) == bsa.FLAG_BAD_SEQLENS
        off = cu or first.tolist()
        for b in range(4):
            good = 0 <= off[b] <= off[b + 1] <= 144 and lens[b] == c.lens[b] and off[b + 1] - off[b] <= lens[b]
            same = off[b] == first[b] and off[b + 1] == first[b + 1]
            r = slice(first[b], first[b + 1])
            if good and same:
                # What the others are worth moves the places where this sequence's keys are divided, and with
                # them the order of its sums: each division is within the tolerance that any order has.
                agree(out[r], lse[r], tuple(x[r] for x in ref))
            elif not good and cu is None:
                assert (out[r] == 7).all() and (lse[r] == 7).all()


def test_a_workspace_for_fewer_keys_leaves_sequences_out():
    c = Chunks(46, "e4m3", 1, 4, 128, 128, [2000, 3000], [600, 700])
    ref = c.expect()
    out = torch.full((1300, 4, 128), 7.0, device="cuda")
    lse = torch.full((1300, 4), 7.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    bsa.prefill(c.q, c.pool.cache, c.table, c.seqlens, c.cu, keys=2000, out=out, lse=lse, err_flag=err, **c.kw)
    left = (lse == 7).all(1)
    if int(err):
        assert int(err) == bsa.FLAG_BAD_SEQLENS and left[600:].all() and (out[600:] == 7).all()
    on = (~left).cpu().numpy()
    assert on[:600].all()
    agree(out[~left], lse[~left], tuple(x[on] for x in ref))


def test_bad_pages_are_left_out_and_flagged():
    for m in (3, 300):
        c = Chunks(47, "e4m3", 2, 1, 64, 16, [700], [m])
        for j, page in ((3, -1), (20, 10 ** 6), (43, -7)):
            c.host_table[0, j] = page
        c.table.copy_(torch.from_numpy(c.host_table))
        out, lse, err = _run(c, out_dtype=torch.float32)
        assert err == bsa.FLAG_BAD_INDEX
        agree(out, lse, c.expect())


def test_strided_queries_and_tables():
    c = Chunks(48, "int8", 2, 3, 64, 32, [400, 90], [300, 4])
    wide = torch.randn(304, 3 * 6 * 64 + 8, device="cuda").to(torch.bfloat16)
    q = wide[:, 8:8 + 6 * 64].unflatten(1, (6, 64))
    q.copy_(c.q)
    table = torch.full((2, c.table.shape[1] + 9), 5, dtype=torch.int32, device="cuda")[:, :c.table.shape[1]]
    table.copy_(c.table)
    out, lse = bsa.prefill(q, c.pool.cache, table, c.seqlens, c.cu, keys=490, out_dtype=torch.float32, **c.kw)
    agree(out, lse, c.expect())


def test_no_queries():
    c = Chunks(49, "e4m3", 1, 1, 64, 16, [10, 20], [0, 0])
    out, lse, err = _run(c)
    assert out.shape == (0, 1, 64) and lse.shape == (0, 1) and err == 0


@pytest.mark.parametrize("m", [2, 400])
def test_nan_scales_and_values(m):
    """A NaN key scale makes the queries that meet the key NaN, and no others."""
    c = Chunks(50, "int8", 1, 2, 128, 64, [500], [m])
    pg, row = c.host_table[0][499 // 64], 499 % 64                      # the last key: only the last query meets it
    c.pool.cache.k_scale[pg, 0, row] = math.nan
    out, lse, err = _run(c, out_dtype=torch.float32)
    assert torch.isnan(out[-1]).all() and torch.isnan(lse[-1]).all()
    o, l, to, tl = c.expect()
    agree(out[:-1], lse[:-1], (o[:-1], l[:-1], to[:-1], tl[:-1]))
    c.pool.cache.k_scale[pg, 0, row] = 0.01
    c.pool.cache.v_scale[pg, 0, row] = math.nan
    out, lse, err = _run(c, out_dtype=torch.float32)
    assert torch.isnan(out[-1]).all() and torch.isfinite(lse).all()
    agree(out[:-1], lse[:-1], (o[:-1], l[:-1], to[:-1], tl[:-1]))


@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
@pytest.mark.parametrize("m", [3, 300])
@pytest.mark.parametrize("size", [0.0, 40.0])
def test_flat_and_peaked(dtype, m, size):
    """Queries of zeros weigh all keys alike; long ones pick one key."""
    c = Chunks(51, dtype, 1, 2, 64, 32, [600], [m], size=size)
    out, lse, err = _run(c, out_dtype=torch.float32)
    agree(out, lse, c.expect())


def _scales(c, name, f):
    """Multiplies the scales of sequence 0's keys by f(j), on both sides."""
    for j in range(c.lens[0]):
        pg, row = c.host_table[0][j // c.pool.page], j % c.pool.page
        c.pool.scales[name][pg, :, row] *= f(j)
    getattr(c.pool.cache, name + "_scale").copy_(torch.from_numpy(c.pool.scales[name]))


@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
@pytest.mark.parametrize("m", [2, 260])
@pytest.mark.parametrize("name,f", [
    ("k", lambda j: 0.75 + 0.5 * (j % 3)),
    ("k", lambda j: 2.0 ** -(j % 60)),
    ("k", lambda j: 2.0 ** -90),
    ("v", lambda j: 1.0 if j else 2.0 ** -7),
    ("v", lambda j: 2.0 ** (j // 128)),
    ("v", lambda j: 2.0 ** -(j // 100)),
    ("v", lambda j: 2.0 ** -115),
    ("v", lambda j: 1.3 * 2.0 ** (30 * (j % 2) - 15)),
    ("v", lambda j: 2.0 ** (20 * (j // 128))),
    ("v", lambda j: 2.0 ** (-20 * (j // 128))),
])
def test_scales_of_every_size(dtype, m, name, f):
    """Weights and values are each rounded to 11 bits."""
    c = Chunks(52, dtype, 1, 1, 64, 128, [560], [m])
    _scales(c, name, f)
    out, lse, err = _run(c, out_dtype=torch.float32)
    agree(out, lse, c.expect(2 * 2.0 ** -11))


def test_graph_and_stream():
    c = Chunks(53, "int8", 2, 2, 128, 64, [900, 40], [300, 3])
    ws = bsa.alloc_prefill_workspace(c.pool.cache, 303, 2, 4, 940)
    out, lse = torch.empty_like(c.q), torch.empty(303, 4, device="cuda")
    args = (c.q, c.pool.cache, c.table, c.seqlens, c.cu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    bsa.prefill(*args, keys=940, workspace=ws, out=out, lse=lse, stream=side, **c.kw)
    side.synchronize()
    want = out.clone(), lse.clone()
    agree(*want, c.expect())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bsa.prefill(*args, keys=940, workspace=ws, out=out, lse=lse, **c.kw)
    out.zero_(), lse.zero_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    c.q.copy_(c.q.flip(0))
    ws.fill_(255)                                                            # it carries nothing
    g.replay()
    o2, l2 = bsa.prefill(*args, keys=940, **c.kw)
    assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_runs_are_alike():
    c = Chunks(54, "e4m3", 3, 4, 128, 64, [4000, 1500, 200], [500, 20, 1])
    a = _run(c)
    for _ in range(3):
        b = _run(c)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_wide_table_and_default_keys():
    c = Chunks(55, "e4m3", 1, 2, 64, 16, [300], [280])
    out, lse = bsa.prefill(c.q, c.pool.cache, c.table, c.seqlens, c.cu, out_dtype=torch.float32, **c.kw)
    agree(out, lse, c.expect())


def test_against_the_forward():
    """A whole prompt appended, then attended over the cache: the forward over the rows that kv_read gives."""
    H, D, lens = 2, 128, [300, 511]
    c = Chunks(56, "e4m3", H, 1, D, 128, lens, lens)
    out, lse, _ = _run(c, out_dtype=torch.float32)
    k, v = bsa.kv_read(c.pool.cache, c.table, c.cu, total=sum(lens))
    nm = [-(-n // 128) for n in lens]
    meta = bsa.alloc_meta(2, H, varlen=True, total_m_blocks=sum(nm), total_n_blocks=sum(n * n for n in nm), max_num_n=max(nm))
    bsa.build_meta(torch.ones(H, sum(n * n for n in nm), dtype=torch.uint8, device="cuda"), meta, cu_seqlens_q=c.cu,
                   cu_seqlens_k=c.cu, kind=bsa.MASK_CAUSAL)
    o, l = bsa.forward(c.q, k, v, meta, cu_seqlens_q=c.cu, cu_seqlens_k=c.cu, kind=bsa.MASK_CAUSAL,
                       out_dtype=torch.float32)
    # the forward rounds its weights to bf16, 2^-8 of each; its sums and exponentials are as in prefill
    agree(o, l.t(), c.expect(2.0 ** -8))
    agree(out, lse, c.expect())
