"""decode and decode_shared_prefix against the oracle, at the sizes and masks where they
can go wrong; tolerances as derived in kv_case.expect."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import block_sparse_flashattention_gb300 as bsa  # noqa: E402
from oracle import kv_cache as okv  # noqa: E402
from tests.kv_case import DT, Pool, agree, bf16, expect, f64, lists, pages_for  # noqa: E402

pytestmark = pytest.mark.gpu


def _q(seed, B, Hq, D, size=1.5):
    return bf16(size * np.random.default_rng(seed).standard_normal((B, Hq, D))).cuda()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


DECODE = [
    # dtype, H, G, D, page, lens
    ("e4m3", 1, 1, 128, 128, [1]),
    ("int8", 2, 1, 64, 16, [0, 1, 2, 15, 16, 17]),
    ("e4m3", 3, 4, 128, 64, [127, 128, 129, 0, 640]),
    ("int8", 2, 5, 128, 32, [300, 31, 33]),
    ("e4m3", 2, 8, 64, 128, [257, 1000]),
    ("int8", 1, 9, 128, 16, [513, 70]),
    ("e4m3", 1, 16, 64, 64, [400]),
    ("int8", 1, 17, 128, 128, [200, 3]),
    ("e4m3", 2, 33, 64, 16, [150]),
    ("int8", 1, 64, 128, 64, [260, 5]),
    ("e4m3", 1, 128, 128, 128, [300]),
    ("e4m3", 5, 2, 128, 128, [2500]),
    ("int8", 4, 1, 64, 64, [5000, 1, 60]),
    ("e4m3", 1, 1, 128, 16, [9000]),
]


@pytest.mark.parametrize("dtype,H,G,D,page,lens", DECODE)
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_decode(dtype, H, G, D, page, lens, out_dtype):
    pool = Pool(11, pages_for(lens, page) + 1, H, D, page, dtype)
    ht, table = pool.tables(lens)
    q = _q(12, len(lens), H * G, D)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = bsa.decode(q, pool.cache, table, _i32(lens), out_dtype=out_dtype, err_flag=err)
    assert int(err) == 0
    agree(out, lse, expect(pool, f64(q), G, lambda b, h: [(ht[b], range(lens[b]))], 1 / math.sqrt(D)))


@pytest.mark.parametrize("kind", ["varlen", "batched"])
@pytest.mark.parametrize("dtype,H,G,D,page,lens,mask_every,valid", [
    ("e4m3", 2, 1, 128, 128, [1000, 130, 0, 128], 0, False),
    ("int8", 3, 4, 64, 16, [700, 700, 1], 2, True),
    ("e4m3", 1, 12, 128, 32, [1300, 257], 1, True),
    ("int8", 2, 2, 128, 64, [5000, 4000], 3, False),
])
def test_decode_lists(kind, dtype, H, G, D, page, lens, mask_every, valid):
    pool = Pool(13, pages_for(lens, page) + 1, H, D, page, dtype)
    ht, table = pool.tables(lens)
    rng = np.random.default_rng(14)
    sel = {(b, h): sorted((int(t) for t in np.flatnonzero(rng.random(-(-n // 128)) < 0.6)), reverse=True)
           for b, n in enumerate(lens) for h in range(H)}
    sel[0, 0] = []                                                  # a head that attends nothing
    meta = lists(H, lens, lambda b, h: sel[b, h], kind=kind, mask_every=mask_every)
    vl = rng.integers(0, 129, (len(lens), meta.num_n)).astype(np.int32) if valid else None

    def keys(b, h):
        out = []
        for i, t in enumerate(sel[b, h]):
            lim = min(128, lens[b] - 128 * t)
            if valid and mask_every and i % mask_every == 0:
                lim = min(lim, int(vl[b, t]))
            out += range(128 * t, 128 * t + max(lim, 0))
        return [(ht[b], out)]
    q = _q(15, len(lens), H * G, D)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = bsa.decode(q, pool.cache, table, _i32(lens), meta=meta, err_flag=err, out_dtype=torch.float32,
                          kv_valid_len=torch.from_numpy(vl).cuda() if valid else None)
    assert int(err) == 0
    agree(out, lse, expect(pool, f64(q), G, keys, 1 / math.sqrt(D)))


PREFIX = [
    # dtype, H, G, D, page, prefix, lens
    ("e4m3", 1, 1, 128, 128, 1, [1]),
    ("int8", 2, 1, 64, 16, 17, [0, 5, 40]),
    ("e4m3", 2, 4, 128, 64, 500, [1, 100, 0, 64]),
    ("int8", 1, 8, 128, 32, 1000, [300, 20, 1, 0, 7]),
    ("e4m3", 3, 2, 64, 128, 129, [3] * 20),
    ("int8", 1, 16, 64, 16, 300, [10, 20, 30]),
    ("e4m3", 2, 3, 128, 128, 700, [2] * 50),
    ("int8", 1, 4, 128, 64, 257, [1, 2] * 40),
    ("e4m3", 1, 20, 64, 128, 400, [5] * 9),
    ("int8", 1, 100, 128, 128, 140, [20, 130]),
    ("e4m3", 1, 8, 128, 128, 2000, [0] * 4),
]


@pytest.mark.parametrize("dtype,H,G,D,page,prefix,lens", PREFIX)
def test_shared_prefix(dtype, H, G, D, page, prefix, lens):
    pool = Pool(21, pages_for(lens + [prefix], page) + 1, H, D, page, dtype)
    hp = pool.take(-(-prefix // page))
    ht, table = pool.tables(lens)
    q = _q(22, len(lens), H * G, D)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    scale = 0.7 / math.sqrt(D)
    out, lse = bsa.decode_shared_prefix(q, pool.cache, _i32(hp), prefix, table, _i32(lens), err_flag=err,
                                        softmax_scale=scale, out_dtype=torch.float32)
    assert int(err) == 0
    ref = expect(pool, f64(q), G, lambda b, h: [(hp, range(prefix)), (ht[b], range(lens[b]))], scale)
    agree(out, lse, ref)
    o16, l16 = bsa.decode_shared_prefix(q, pool.cache, _i32(hp), prefix, table, _i32(lens), softmax_scale=scale)
    agree(o16, l16, ref)
    if not any(lens):
        o, l = bsa.decode_shared_prefix(q, pool.cache, _i32(hp), prefix, None, _i32(lens), softmax_scale=scale,
                                        out_dtype=torch.float32)
        assert torch.equal(o, out) and torch.equal(l, lse)


LONG = [
    # the same, at sizes that take the prefix in the streaming line or in its own kernel:
    # up to 128, 256 and more query rows a head, tails of every kind, one CTA to many
    ("int8", 8, 2, 128, 64, 5000, [3, 0, 7, 20, 1, 1, 40, 9]),
    ("e4m3", 5, 1, 64, 16, 30011, [2, 0, 33, 5]),
    ("e4m3", 1, 3, 128, 64, 2500, [1 + i % 5 for i in range(130)]),
    ("int8", 1, 1, 128, 16, 3001, [i % 3 for i in range(110)]),
    ("int8", 2, 8, 128, 128, 4500, [i % 4 for i in range(40)]),
    ("e4m3", 3, 2, 64, 32, 4097, [5] * 50),
    ("int8", 1, 16, 64, 16, 5000, [i % 2 for i in range(120)]),
    ("int8", 4, 5, 64, 128, 2049, [2] * 80),
    ("e4m3", 1, 1, 128, 128, 20000, [i for i in range(17)]),
    ("e4m3", 2, 4, 128, 32, 1300, [1] * 120),
]


@pytest.mark.parametrize("dtype,H,G,D,page,prefix,lens", LONG)
def test_shared_prefix_long(dtype, H, G, D, page, prefix, lens):
    assert len(lens) * H * prefix * 2 * (D + 4) > 76 << 20
    pool = Pool(121, pages_for(lens + [prefix], page) + 1, H, D, page, dtype)
    hp = pool.take(-(-prefix // page))
    ht, table = pool.tables(lens)
    q = _q(122, len(lens), H * G, D)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = bsa.decode_shared_prefix(q, pool.cache, _i32(hp), prefix, table, _i32(lens), err_flag=err,
                                        out_dtype=torch.float32)
    assert int(err) == 0
    # many rows: values whose scales are not powers of two carry two roundings to 11 bits more
    coarse = 2.0 ** -10 if dtype == "int8" and len(lens) * G > 16 else 0.0
    agree(out, lse, expect(pool, f64(q), G, lambda b, h: [(hp, range(prefix)), (ht[b], range(lens[b]))],
                           1 / math.sqrt(D), coarse))
    again = bsa.decode_shared_prefix(q, pool.cache, _i32(hp), prefix, table, _i32(lens), out_dtype=torch.float32)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("B,G", [(120, 1), (120, 4), (4, 2)])
@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
def test_long_prefix_with_faults_and_odd_scales(B, G, dtype):
    """Bad prefix pages are left out and flagged, rows behind the prefix's end may be NaN, value and key scales
    differ by 2^40, some are 0."""
    H, D, page = 1 if B > 4 else 30, 128, 64
    prefix = 2700
    pool = Pool(123, 44, H, D, page, dtype, spread=0.0)
    rng = np.random.default_rng(124)
    for name in ("k", "v"):
        e = rng.integers(-30, 12, pool.scales[name].shape) if name == "v" else rng.integers(-6, 3, pool.scales[name].shape)
        s = (2.0 ** np.floor(np.log2(pool.scales[name])) if dtype == "int8" else pool.scales[name]) * 2.0 ** e
        pool.scales[name] = s.astype(np.float32)
        pool.scales[name][..., 5] = 0.0
    hp = pool.take(43)
    last = hp[-1]
    for name in ("k", "v"):
        t = torch.from_numpy(pool.scales[name]).clone()
        t[last, :, prefix % page:] = float("nan")
        getattr(pool.cache, name + "_scale").copy_(t)
        getattr(pool.cache, name).view(torch.uint8)[last, :, prefix % page:] = 0x7F
    hp[3], hp[20] = 10 ** 6, -1
    lens = [0] * B
    q = _q(125, B, H * G, D)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = bsa.decode_shared_prefix(q, pool.cache, _i32(hp), prefix, None, _i32(lens), err_flag=err, out_dtype=torch.float32)
    assert int(err) == bsa.FLAG_BAD_INDEX
    agree(out, lse, expect(pool, f64(q), G, lambda b, h: [(hp, range(prefix))], 1 / math.sqrt(D)))


@pytest.mark.parametrize("dtype,D", [("e4m3", 64), ("int8", 128)])
def test_long_prefix_many_tiles_per_block(dtype, D):
    """Two blocks of query rows and two heads over 313 tiles: pieces of eight tiles and more, some of which hold
    the end of one block's line and the beginning of the next."""
    H, G, page, prefix, B = 2, 2, 128, 40000, 150
    pool = Pool(126, pages_for([prefix], page), H, D, page, dtype)
    hp = pool.take(-(-prefix // page))
    q = _q(127, B, H * G, D)
    out, lse = bsa.decode_shared_prefix(q, pool.cache, _i32(hp), prefix, None, _i32([0] * B), out_dtype=torch.float32)
    some = [0, 63, 64, 127, 128, 149]
    coarse = 2.0 ** -10 if dtype == "int8" else 0.0
    agree(out[some], lse[some], expect(pool, f64(q[some]), G, lambda b, h: [(hp, range(prefix))], 1 / math.sqrt(D), coarse))


class _Heads:
    """Some heads of a pool, as expect() asks for rows."""

    def __init__(self, pool, heads):
        self.pool, self.heads = pool, heads

    def host(self, name, table, h, positions):
        return self.pool.host(name, table, self.heads[h], positions)


def _some_heads(pool, q, G, heads, parts, scale, coarse=0.0):
    """(columns of the query heads of KV heads `heads`, expect() for them)."""
    cols = [h * G + g for h in heads for g in range(G)]
    return cols, expect(_Heads(pool, heads), f64(q[:, cols]), G, parts, scale, coarse)


@pytest.mark.parametrize("dtype,H,G,D,B,prefix", [
    ("int8", 600, 20, 64, 2, 100),     # one tile a segment, several segments a block
    ("e4m3", 600, 20, 64, 6, 128),
    ("e4m3", 32, 1, 128, 128, 640),    # pieces of one tile, some of two segments
    ("int8", 90, 18, 64, 3, 300),      # three tiles a segment: pieces with the last tile of one, the first of the next
])
def test_long_prefix_with_one_tile_of_a_segment_in_a_block(dtype, H, G, D, B, prefix):
    """At most 128 query rows a head and one tile of a segment in a block: one of the two slots has no key there,
    in one segment after the other.  The workspace holds NaN before each call: no part may be left out."""
    page = 64
    pool = Pool(170, pages_for([prefix], page), H, D, page, dtype)
    hp = pool.take(-(-prefix // page))
    q = _q(171, B, H * G, D)
    ws = bsa.alloc_decode_workspace(pool.cache, B, H * G, prefix_len=prefix)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    first = None
    for _ in range(8):
        ws.fill_(255)
        got = bsa.decode_shared_prefix(q, pool.cache, _i32(hp), prefix, None, _i32([0] * B), workspace=ws, err_flag=err,
                                       out_dtype=torch.float32)
        first = first or got
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])
    assert int(err) == 0
    cols, ref = _some_heads(pool, q, G, sorted({0, 1, 2, H // 3, H // 2, H - 2, H - 1}), lambda b, h: [(hp, range(prefix))],
                            1 / math.sqrt(D), 2.0 ** -10 if dtype == "int8" else 0.0)
    agree(first[0][:, cols], first[1][:, cols], ref)


OWN_KERNEL = [(120, 1, 2, 1500), (3, 20, 3, 300), (60, 5, 2, 2700)]   # B, G, H, keys: rows in both slots alike, in both halves


def _own_kernel(seed, B, G, H, n, page, dtype, spread=0.3, more=2):
    """A pool of heads of 128 for a prefix of about n keys that has a kernel of its own, and its pages."""
    assert G > 16 or B * H * n * 2 * 132 > 76 << 20
    pool = Pool(seed, pages_for([n], page) + more, H, 128, page, dtype, spread=spread)
    return pool, pool.take(-(-n // page))


def _set_row(pool, name, page, row, scale, zero=True):
    """Row `row` of a page: zeros (or its codes), with this scale, in the cache and in its host copy."""
    pool.scales[name][page, :, row] = scale
    getattr(pool.cache, name + "_scale")[page, :, row] = scale
    if zero:
        pool.codes[name][page, :, row] = 0
        getattr(pool.cache, name).view(torch.uint8)[page, :, row] = 0


@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
@pytest.mark.parametrize("page", [128, 32])
@pytest.mark.parametrize("B,G,H,n", OWN_KERNEL)
def test_a_tile_of_a_long_prefix_without_a_key(B, G, H, n, page, dtype):
    """Every page of a tile bad (with pages of 128: one entry): its keys are left out and flagged, whether they
    come first, amid others or are all there are; the sequences' own keys are attended all the same."""
    pool, hp = _own_kernel(172, B, G, H, n, page, dtype, more=B)
    lens = [i % 3 for i in range(B)]
    ht, table = pool.tables(lens)
    q = _q(173, B, H * G, 128)
    per, coarse = 128 // page, 2.0 ** -10 if dtype == "int8" else 0.0
    some = [0, 1, 2, B - 1]
    for tiles in ([1], [0], range(-(-n // 128))):
        bad = list(hp)
        for t in tiles:
            for i in range(t * per, min((t + 1) * per, len(bad))):
                bad[i] = -1 if i % 2 else 10 ** 6
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = bsa.decode_shared_prefix(q, pool.cache, _i32(bad), n, table, _i32(lens), err_flag=err, out_dtype=torch.float32)
        assert int(err) == bsa.FLAG_BAD_INDEX
        agree(out[some], lse[some], expect(pool, f64(q[some]), G,
                                           lambda b, h: [(bad, range(n)), (ht[some[b]], range(lens[some[b]]))], 1 / math.sqrt(128), coarse))


@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
@pytest.mark.parametrize("scale", [2.0 ** -126, 0.0])           # as rows of zeros are appended, as a new cache holds them
@pytest.mark.parametrize("B,G,H,n", OWN_KERNEL + [(2, 20, 2, 1)])
def test_zero_keys_in_the_last_tile_of_a_long_prefix(B, G, H, n, scale, dtype):
    n = (n - 1) // 128 * 128 + 1
    pool, hp = _own_kernel(174, B, G, H, n, 128, dtype)
    for name in ("k", "v"):
        _set_row(pool, name, hp[-1], 0, scale)
    q = _q(175, B, H * G, 128)
    out, lse = bsa.decode_shared_prefix(q, pool.cache, _i32(hp), n, None, _i32([0] * B), out_dtype=torch.float32)
    some = [0, 1, B - 1]
    agree(out[some], lse[some], expect(pool, f64(q[some]), G, lambda b, h: [(hp, range(n))], 1 / math.sqrt(128),
                                       2.0 ** -10 if dtype == "int8" else 0.0))


@pytest.mark.parametrize("B,G,H,n", OWN_KERNEL)
def test_a_long_prefix_in_a_new_cache(B, G, H, n):
    """A zero-filled cache, as a warm-up call meets it: every score is 0, every value too."""
    cache = bsa.alloc_kv_cache(-(-n // 128), H, 128)
    out, lse = bsa.decode_shared_prefix(_q(176, B, H * G, 128), cache, _i32(list(range(cache.num_pages))), n, None,
                                        _i32([0] * B), out_dtype=torch.float32)
    assert not out.any() and (lse - math.log(n)).abs().max() <= math.log(n) * 2.0 ** -22 + 2.0 ** -20


@pytest.mark.parametrize("B,G,H,n", OWN_KERNEL)
@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
def test_the_smallest_scales_of_a_long_prefix(B, G, H, n, dtype):
    """Keys and values whose scales are fp32's smallest normal number, queries so large that the scores differ."""
    pool, hp = _own_kernel(177, B, G, H, n, 128, dtype)
    for name in ("k", "v"):
        pool.scales[name][:] = 2.0 ** -126
        getattr(pool.cache, name + "_scale").fill_(2.0 ** -126)
    q = _q(178, B, H * G, 128, size=2.0 ** (126 - 6))
    out, lse = bsa.decode_shared_prefix(q, pool.cache, _i32(hp), n, None, _i32([0] * B), out_dtype=torch.float32)
    some = [0, 1, B - 1]
    agree(out[some], lse[some], expect(pool, f64(q[some]), G, lambda b, h: [(hp, range(n))], 1 / math.sqrt(128)))


@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
@pytest.mark.parametrize("B,G,H,n", OWN_KERNEL + [(4, 2, 3, 300), (2, 12, 3, 300)])
def test_a_nan_key_scale_is_not_dropped(B, G, H, n, dtype):
    """A row whose key scale is NaN is NaN whatever its codes are, also where all of them and the queries have one sign
    each, so that a score of infinite size would be -inf, the score of a key that does not count."""
    pool = Pool(179, pages_for([n], 64), H, 128, 64, dtype)
    hp = pool.take(-(-n // 64))
    at = (hp[1], 1, 9)
    pool.cache.k.view(torch.uint8)[at] = 0x7E if dtype == "e4m3" else 0x7F     # the largest code
    pool.cache.k_scale[at] = float("nan")
    q = -_q(180, B, H * G, 128).abs()
    nan = torch.arange(H * G, device="cuda") // G == 1
    out, lse = bsa.decode_shared_prefix(q, pool.cache, _i32(hp), n, None, _i32([0] * B), out_dtype=torch.float32)
    assert out[:, nan].isnan().all() and lse[:, nan].isnan().all()
    assert out[:, ~nan].isfinite().all() and lse[:, ~nan].isfinite().all()
    o2, l2 = bsa.decode(q, pool.cache, _i32([hp] * B), _i32([n] * B), out_dtype=torch.float32)
    assert o2[:, nan].isnan().all() and l2[:, nan].isnan().all() and l2[:, ~nan].isfinite().all()


@pytest.mark.parametrize("B,G,H,n", OWN_KERNEL)
@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
@pytest.mark.parametrize("far", [15, 34, 80])
def test_a_huge_key_leaves_the_others_their_scores(B, G, H, n, dtype, far):
    """One key's scale is 2^far times its neighbours', and its score so low that it has no weight: the scores of the
    keys in its tile are as exact as without it."""
    pool, hp = _own_kernel(181, B, G, H, n, 128, dtype)
    pool.cache.k.view(torch.uint8)[hp[1], :, 9] = 0xFE if dtype == "e4m3" else 0x81     # -448, -127
    pool.cache.k_scale[hp[1], :, 9] = 2.0 ** (far - 8)      # the neighbours' are about 2^-8 (e4m3) and 2^-6
    q = _q(182, B, H * G, 128).abs()
    out, lse = bsa.decode_shared_prefix(q, pool.cache, _i32(hp), n, None, _i32([0] * B), out_dtype=torch.float32)
    some = [0, 1, B - 1]
    agree(out[some], lse[some], expect(pool, f64(q[some]), G, lambda b, h: [(hp, [j for j in range(n) if j != 128 + 9])],
                                       1 / math.sqrt(128), 2.0 ** -10 if dtype == "int8" else 0.0))


def _agree_far(out, lse, pool, q, G, keys, coarse):
    """Against the oracle, relative to what the keys contribute, not to the largest value.  The weights of P V carry the
    value scales where these lie far apart: a weight is rounded by 2^-11 of itself, or by 2^-25 where the largest is 2^7
    or more, and multiplies at most 2^7 largest codes, the one of the largest contribution at least 2^5 (codes and
    factors vary by 2 each): 2^-30 of the largest contribution, 2^-28 where the scales of tiles that are not far apart
    differ by 2^2 at most.  Scores: as in expect()."""
    B, Hq, D = q.shape
    scale = 1 / math.sqrt(D)
    got, gl, x = f64(out), f64(lse), f64(q)
    for h in range(Hq // G):
        k, v = pool.host("k", keys, h, range(len(keys) * pool.page)), pool.host("v", keys, h, range(len(keys) * pool.page))
        for b in range(B):
            for g in range(G):
                i = h * G + g
                o, l, spread = okv.attend(x[b, i], k, v, scale)
                s = scale * (k @ x[b, i])
                ds = (D + 8) * 2.0 ** -24 * scale * float(np.max(np.abs(k) @ np.abs(x[b, i])))
                top = float(np.max(np.exp(s - l) * np.max(np.abs(v), 1)))
                tol = spread * (2.0 ** -11 + 2 * ds + coarse + 2.0 ** -20) + len(k) * 2.0 ** -28 * top
                assert np.all(np.abs(got[b, i] - o) <= tol), (b, i, np.max(np.abs(got[b, i] - o) / tol))
                assert abs(gl[b, i] - l) <= ds + 2.0 ** -20 + abs(l) * 2.0 ** -22


def _scaled(pool, name, factor):
    """Multiplies scales (broadcast over heads) by factor [pages, rows], in the cache and in its host copy."""
    pool.scales[name] = (pool.scales[name] * factor[:, None]).astype(np.float32)
    getattr(pool.cache, name + "_scale").copy_(torch.from_numpy(pool.scales[name]))


@pytest.mark.parametrize("B,G,H,n", [(120, 1, 2, 1536), (3, 20, 3, 384), (60, 5, 2, 2688), (3, 20, 60, 1536), (75, 4, 40, 1024)])
@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
@pytest.mark.parametrize("far,first", [(13, 0), (26, 0), (26, 1), (60, 0), (60, 1), (40, 2)])
def test_value_scales_far_apart_in_a_long_prefix(B, G, H, n, dtype, far, first):
    """Half of the values are 2^far smaller than the others, and one key there has 2^far the weight of one among the
    others, so that both contribute alike, whichever half comes first (2: every other key)."""
    pool, hp = _own_kernel(183, B, G, H, n, 128, dtype, spread=0.0, more=0)
    small = np.zeros((len(hp), 128), bool).reshape(-1)
    small[::2] = first == 2
    if first < 2:
        small[:n // 2] = first == 0
        small[n // 2:] = first == 1
    _scaled(pool, "v", np.where(small, 2.0 ** -far * 1.3, 1.0).reshape(-1, 128)[np.argsort(hp)])
    pair = [int(np.flatnonzero(small)[len(small) // 4 - 3]), int(np.flatnonzero(~small)[len(small) // 4 - 3])]
    _scaled(pool, "k", np.full((len(hp), 128), 2.0 ** -10))
    q = _q(184, B, H * G, 128).abs()
    some = sorted({0, 1, B - 1})
    for j, s in zip(pair, (20 + far, 20)):               # scores of about s ln 2: q . k = 1.2 x 128 code scale
        x = s * math.log(2) * math.sqrt(128) / (1.2 * 128)
        code, value = (0x7E, 448.0) if dtype == "e4m3" else (0x7F, 127.0)
        pg, row = hp[j // 128], j % 128
        pool.codes["k"][pg, :, row] = code
        pool.cache.k.view(torch.uint8)[pg, :, row] = code
        _set_row(pool, "k", pg, row, float(np.float32(x / value)), zero=False)
    out, lse = bsa.decode_shared_prefix(q, pool.cache, _i32(hp), n, None, _i32([0] * B), out_dtype=torch.float32)
    _agree_far(out[some], lse[some], pool, q[some], G, hp, 2.0 ** -10)


@pytest.mark.parametrize("B,G,H,n", [(120, 1, 2, 1536), (3, 20, 3, 384), (60, 5, 2, 2688)])
@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
def test_value_scales_of_all_sizes_in_a_long_prefix(B, G, H, n, dtype):
    """Value scales of every size from 2^-60 to 2^60 and 0, some rows of zeros, one tile of bad pages; queries so large
    that the weights differ as much."""
    pool, hp = _own_kernel(185, B, G, H, n, 128, dtype, spread=0.0, more=0)
    rng = np.random.default_rng(186)
    _scaled(pool, "v", 2.0 ** rng.uniform(-60, 60, (len(hp), 128)))
    for row, scale in ((5, 0.0), (70, 2.0 ** -126), (127, 0.0)):
        _set_row(pool, "v", hp[2], row, scale)
    pages = list(hp)
    pages[1] = -1
    q = _q(187, B, H * G, 128, size=12.0)
    some = sorted({0, 1, B - 1})
    out, lse = bsa.decode_shared_prefix(q, pool.cache, _i32(pages), n, None, _i32([0] * B), out_dtype=torch.float32)
    _agree_far(out[some], lse[some], pool, q[some], G, pages, 2.0 ** -10)


@pytest.mark.parametrize("dtype,H,G,D,B,prefix", [
    ("e4m3", 8, 1, 128, 5, 8000),      # prefix in the streaming line
    ("int8", 2, 2, 128, 20, 8000),     # in its own kernel
    ("e4m3", 1, 20, 64, 9, 3000),      # the same, more query rows a head than a streaming warp holds
])
@pytest.mark.parametrize("kind", ["varlen", "batched"])
def test_long_prefix_with_lists_and_fused_rows(dtype, H, G, D, B, prefix, kind):
    page, lens = 64, [(137 * i) % 400 for i in range(B)]
    pool = Pool(128, pages_for(lens + [prefix], page), H, D, page, dtype)
    hp = pool.take(-(-prefix // page))
    ht, table = pool.tables(lens)
    q = _q(129, B, H * G + 3 * H, D)[:, 2 * H:2 * H + H * G]     # rows of a fused projection
    sel = lambda b, h: [t for t in range(-(-lens[b] // 128)) if (t + b + h) % 3]  # noqa: E731
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = bsa.decode_shared_prefix(q, pool.cache, _i32(hp), prefix, table, _i32(lens), err_flag=err,
                                        meta=lists(H, lens, sel, kind=kind, mask_every=2), out_dtype=torch.float32)
    assert int(err) == 0
    keys = lambda b, h: [p for t in sel(b, h) for p in range(128 * t, min(lens[b], 128 * t + 128))]  # noqa: E731
    coarse = 2.0 ** -10 if dtype == "int8" else 0.0
    agree(out, lse, expect(pool, f64(q), G, lambda b, h: [(hp, range(prefix)), (ht[b], keys(b, h))], 1 / math.sqrt(D), coarse))


@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
@pytest.mark.parametrize("B,G", [(4, 2), (20, 1), (150, 2), (3, 20)])
def test_nan_rows_of_a_prefix_reach_their_head_only(dtype, B, G):
    H, D, page, prefix = 10, 128, 128, 9000
    pool = Pool(130, pages_for([prefix], page), H, D, page, dtype)
    hp = pool.take(-(-prefix // page))
    q = _q(131, B, H * G, D)
    run = lambda: bsa.decode_shared_prefix(q, pool.cache, _i32(hp), prefix, None, _i32([0] * B), out_dtype=torch.float32)  # noqa: E731
    clean, clean_lse = run()
    at = (hp[4000 // page], 3, 4000 % page)
    heads = torch.arange(H * G, device="cuda") // G == 3
    pool.cache.v[at] = torch.zeros(D, device="cuda").to(pool.cache.v.dtype)    # as a row with NaN or infinity is kept
    pool.cache.v_scale[at] = float("nan")
    out, lse = run()
    assert out[:, heads].isnan().all() and torch.equal(out[:, ~heads], clean[:, ~heads]) and torch.equal(lse, clean_lse)
    pool.cache.k[at] = torch.zeros(D, device="cuda").to(pool.cache.k.dtype)
    pool.cache.k_scale[at] = float("nan")
    out, lse = run()
    assert out[:, heads].isnan().all() and lse[:, heads].isnan().all()
    assert torch.equal(out[:, ~heads], clean[:, ~heads]) and torch.equal(lse[:, ~heads], clean_lse[:, ~heads])


@pytest.mark.parametrize("listed", [False, True])
def test_many_sequences(listed):
    """More sequences than a block has threads, most of them short or empty; many blocks of query rows."""
    B, H, G, D, page, prefix = 3000, 2, 2, 64, 16, 500
    lens = [(7 * i) % 4 if i % 500 else 300 for i in range(B)]
    pool = Pool(136, pages_for(lens + [prefix], page), H, D, page, "e4m3")
    hp = pool.take(-(-prefix // page))
    ht, table = pool.tables(lens)
    q = _q(137, B, H * G, D)
    meta = lists(H, lens, lambda b, h: range(0, -(-lens[b] // 128), 2)) if listed else None
    keys = lambda b: [p for p in range(lens[b]) if not listed or p // 128 % 2 == 0]  # noqa: E731
    some = sorted({0, 1, 2, 3, 31, 32, 499, 500, 501, 1023, 1024, 1500, 2047, 2500, 2998, 2999})
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = bsa.decode(q, pool.cache, table, _i32(lens), meta=meta, err_flag=err, out_dtype=torch.float32)
    agree(out[some], lse[some], expect(pool, f64(q[some]), G, lambda b, h: [(ht[some[b]], keys(some[b]))], 1 / math.sqrt(D)))
    empty = torch.tensor([n == 0 for n in lens], device="cuda")
    assert not out[empty].any() and torch.isneginf(lse[empty]).all() and lse[~empty].isfinite().all()
    out, lse = bsa.decode_shared_prefix(q, pool.cache, _i32(hp), prefix, table, _i32(lens), meta=meta, err_flag=err,
                                        out_dtype=torch.float32)
    assert int(err) == 0 and lse.isfinite().all()
    agree(out[some], lse[some], expect(pool, f64(q[some]), G, lambda b, h: [(hp, range(prefix)), (ht[some[b]], keys(some[b]))],
                                       1 / math.sqrt(D)))


@pytest.mark.parametrize("G", [1, 24])
def test_one_long_sequence_among_many(G):
    """A sequence that takes most of the line, empty ones before and behind it."""
    H, D, page = 1, 64, 64
    lens = [0] * 300 + [20000] + [0, 1] * 200
    pool = Pool(138, pages_for(lens, page), H, D, page, "int8")
    ht, table = pool.tables(lens)
    q = _q(139, len(lens), H * G, D)
    out, lse = bsa.decode(q, pool.cache, table, _i32(lens), out_dtype=torch.float32)
    some = [0, 299, 300, 301, 302, 303, 699, 700]
    agree(out[some], lse[some], expect(pool, f64(q[some]), G, lambda b, h: [(ht[some[b]], range(lens[some[b]]))], 1 / math.sqrt(D)))
    assert lse[torch.tensor([n > 0 for n in lens], device="cuda")].isfinite().all()


def test_prefix_equals_private_copies():
    """A shared prefix gives what the same keys at the head of every sequence's own table give."""
    H, G, D, page, prefix, lens = 2, 4, 128, 16, 160, [37, 1, 300]
    pool = Pool(23, pages_for(lens + [prefix], page), H, D, page, "e4m3")
    hp = pool.take(prefix // page)
    ht, table = pool.tables(lens)
    q = _q(24, 3, H * G, D)
    out, lse = bsa.decode_shared_prefix(q, pool.cache, _i32(hp), prefix, table, _i32(lens), out_dtype=torch.float32)
    whole = torch.cat([_i32(hp)[None].expand(3, -1), table], 1).contiguous()
    o2, l2 = bsa.decode(q, pool.cache, whole, _i32([prefix + n for n in lens]), out_dtype=torch.float32)
    ref = expect(pool, f64(q), G, lambda b, h: [(hp, range(prefix)), (ht[b], range(lens[b]))], 1 / math.sqrt(D))
    agree(out, lse, ref)
    agree(o2, l2, ref)


def test_prefix_with_lists():
    """Lists choose among a sequence's own tiles; the prefix is attended whole."""
    H, G, D, page, prefix, lens = 2, 2, 64, 64, 200, [600, 0, 129]
    pool = Pool(25, pages_for(lens + [prefix], page), H, D, page, "int8")
    hp = pool.take(-(-prefix // page))
    ht, table = pool.tables(lens)
    q = _q(26, 3, H * G, D)
    sel = lambda b, h: [t for t in range(-(-lens[b] // 128) - 1, -1, -1) if (t + h) % 2 == 0]  # noqa: E731
    out, lse = bsa.decode_shared_prefix(q, pool.cache, _i32(hp), prefix, table, _i32(lens),
                                        meta=lists(H, lens, sel), out_dtype=torch.float32)
    keys = lambda b, h: [p for t in sel(b, h) for p in range(128 * t, min(lens[b], 128 * t + 128))]  # noqa: E731
    agree(out, lse, expect(pool, f64(q), G, lambda b, h: [(hp, range(prefix)), (ht[b], keys(b, h))], 1 / math.sqrt(D)))


def test_bad_pages_and_lengths():
    """Keys on a page outside the cache are left out and flagged; a length past the table is cut."""
    H, G, D, page, lens = 2, 2, 128, 32, [100, 90, 500, -4]
    pool = Pool(27, pages_for([100, 90, 128], page), H, D, page, "e4m3")
    ht, table = pool.tables([100, 90, 128, 0])
    ht[0, 1], ht[0, 3], ht[1, 0] = 10 ** 6, -7, pool.cache.num_pages
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = _q(28, 4, H * G, D)
    out, lse = bsa.decode(q, pool.cache, torch.from_numpy(ht).cuda(), _i32(lens), err_flag=err, out_dtype=torch.float32)
    assert int(err) == bsa.FLAG_BAD_INDEX | bsa.FLAG_BAD_SEQLENS
    ref = expect(pool, f64(q), G, lambda b, h: [(ht[b], range(min(max(lens[b], 0), 128)))], 1 / math.sqrt(D))
    agree(out, lse, ref)
    # without an error word the same results
    o2, l2 = bsa.decode(q, pool.cache, torch.from_numpy(ht).cuda(), _i32(lens), out_dtype=torch.float32)
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    # a prefix of bad pages only: nothing to attend there
    err.zero_()
    o3, l3 = bsa.decode_shared_prefix(q, pool.cache, _i32([-1, 99]), 40, torch.from_numpy(ht).cuda(), _i32(lens),
                                      err_flag=err, out_dtype=torch.float32)
    assert int(err) == bsa.FLAG_BAD_INDEX | bsa.FLAG_BAD_SEQLENS
    agree(o3, l3, ref)


@pytest.mark.parametrize("kind", ["varlen", "batched"])
def test_bad_lists(kind):
    H, G, D, page, lens = 1, 2, 64, 128, [600, 300]
    pool = Pool(29, pages_for(lens, page), H, D, page, "int8")
    ht, table = pool.tables(lens)
    q = _q(30, 2, H * G, D)
    run = lambda meta, err: bsa.decode(q, pool.cache, table, _i32(lens), meta=meta, err_flag=err, out_dtype=torch.float32)  # noqa: E731
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    meta = lists(H, lens, lambda b, h: [-(-lens[b] // 128) - 1, 0], kind=kind)
    flat = meta.full_idx.view(-1)
    flat[0] = 77                                  # sequence 0 lists tile 77 and tile 0
    out, lse = run(meta, err)
    assert int(err) == bsa.FLAG_BAD_INDEX
    keys = [list(range(128)), list(range(256, 300)) + list(range(128))]
    agree(out, lse, expect(pool, f64(q), G, lambda b, h: [(ht[b], keys[b])], 1 / math.sqrt(D)))
    err.zero_()
    meta = lists(H, lens, lambda b, h: [0], kind=kind)
    meta.full_cnt.view(-1)[0], meta.full_cnt.view(-1)[1] = 1000, -3
    out, lse = run(meta, err)                     # 1000 -> all of the row's entries, the rest of them -1
    assert int(err) == bsa.FLAG_BAD_INDEX | bsa.FLAG_BAD_COUNT
    agree(out, lse, expect(pool, f64(q), G, lambda b, h: [(ht[b], range(128 if b == 0 else 0))], 1 / math.sqrt(D)))
    if kind == "varlen":
        err.zero_()
        meta = lists(H, lens, lambda b, h: [0], kind=kind)
        meta.cu_block_idx_offsets[1] = 7          # sequence 1's row would leave the index array
        out, lse = run(meta, err)
        assert int(err) == bsa.FLAG_BAD_SEQLENS
        agree(out, lse, expect(pool, f64(q), G, lambda b, h: [(ht[b], range(128 if b == 0 else 0))], 1 / math.sqrt(D)))


@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
@pytest.mark.parametrize("G", [1, 16])
def test_what_lies_behind_the_last_key_is_not_read_into_the_result(dtype, G):
    """Codes and scales past a sequence's end, in the same page, may be anything, NaN included."""
    H, D, page, lens = 2, 128, 128, [5, 77, 128 + 3]
    pool = Pool(31, pages_for(lens, page) + 1, H, D, page, dtype)
    ht, table = pool.tables(lens)
    q = _q(32, 3, H * G, D)
    for b, n in enumerate(lens):
        last = int(ht[b, n // page])
        for t in (pool.cache.k, pool.cache.v):
            t.view(torch.uint8)[last, :, n % page:] = 0x7F
        for t in (pool.cache.k_scale, pool.cache.v_scale):
            t[last, :, n % page:] = float("nan")
    out, lse = bsa.decode(q, pool.cache, table, _i32(lens), out_dtype=torch.float32)
    agree(out, lse, expect(pool, f64(q), G, lambda b, h: [(ht[b], range(lens[b]))], 1 / math.sqrt(D)))
    o2, l2 = bsa.decode_shared_prefix(q, pool.cache, table[2].contiguous(), lens[2], table, _i32(lens), out_dtype=torch.float32)
    agree(o2, l2, expect(pool, f64(q), G, lambda b, h: [(ht[2], range(lens[2])), (ht[b], range(lens[b]))], 1 / math.sqrt(D)))


def test_nan_rows_reach_their_own_sequences_only():
    H, G, D, page, lens = 1, 2, 64, 16, [40, 40]
    pool = Pool(33, pages_for(lens, page), H, D, page, "e4m3")
    ht, table = pool.tables(lens)
    pool.cache.v_scale[int(ht[0, 1]), 0, 3] = float("nan")
    q = _q(34, 2, H * G, D)
    out, lse = bsa.decode(q, pool.cache, table, _i32(lens), out_dtype=torch.float32)
    assert out[0].isnan().all() and out[1].isfinite().all() and lse.isfinite().all()
    pool.cache.k_scale[int(ht[0, 1]), 0, 3] = float("nan")
    out, lse = bsa.decode(q, pool.cache, table, _i32(lens), out_dtype=torch.float32)
    assert out[0].isnan().all() and lse[0].isnan().all() and out[1].isfinite().all() and lse[1].isfinite().all()


@pytest.mark.parametrize("G", [1, 12])
def test_scales_of_all_sizes(G):
    """Rows whose scales differ by 2^40 and more, zero scales, large scores: the weight of a key that
    matters is never lost to the range of a 16-bit type."""
    H, D, page, lens = 1, 64, 64, [300, 200]
    pool = Pool(35, pages_for(lens, page), H, D, page, "e4m3", spread=0.0)
    ht, table = pool.tables(lens)
    rng = np.random.default_rng(36)
    for name in ("k", "v"):
        e = rng.integers(-30, 12, pool.scales[name].shape) if name == "v" else rng.integers(-6, 3, pool.scales[name].shape)
        pool.scales[name] = (pool.scales[name] * 2.0 ** e).astype(np.float32)
        pool.scales[name][..., 5] = 0.0
        getattr(pool.cache, name + "_scale").copy_(torch.from_numpy(pool.scales[name]))
    q = _q(37, 2, H * G, D, size=4.0)
    out, lse = bsa.decode(q, pool.cache, table, _i32(lens), out_dtype=torch.float32)
    agree(out, lse, expect(pool, f64(q), G, lambda b, h: [(ht[b], range(lens[b]))], 1 / math.sqrt(D)))
    # one key whose values are tiny next to its neighbours' but which takes all of the weight
    pool.scales["v"][:] = 1.0
    pool.scales["v"][ht[1, 0], 0, 7] = 2.0 ** -20
    pool.cache.v_scale.copy_(torch.from_numpy(pool.scales["v"]))
    meta_q = q.clone()
    k7 = pool.host("k", ht[1], 0, [7])[0]
    meta_q[1] = bf16((k7 / np.linalg.norm(k7) * 2000)[None].repeat(G, 0)).cuda()
    pool.scales["k"][ht[1, 0], 0, 7] = 4.0
    pool.cache.k_scale.copy_(torch.from_numpy(pool.scales["k"]))
    out, lse = bsa.decode(meta_q, pool.cache, table, _i32(lens), out_dtype=torch.float32)
    agree(out, lse, expect(pool, f64(meta_q), G, lambda b, h: [(ht[b], range(lens[b]))], 1 / math.sqrt(D)))


@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
@pytest.mark.parametrize("G,D", [(1, 128), (12, 64), (20, 128), (100, 64)])
def test_the_smallest_scales(G, D, dtype):
    """Keys and values whose scales are fp32's smallest normal number, queries so large that the scores differ."""
    H, page, lens = 2, 32, [500, 1, 70]
    pool = Pool(188, pages_for(lens, page), H, D, page, dtype)
    ht, table = pool.tables(lens)
    for name in ("k", "v"):
        pool.scales[name][:] = 2.0 ** -126
        getattr(pool.cache, name + "_scale").fill_(2.0 ** -126)
    q = _q(189, 3, H * G, D, size=2.0 ** (126 - 6))
    out, lse = bsa.decode(q, pool.cache, table, _i32(lens), out_dtype=torch.float32)
    agree(out, lse, expect(pool, f64(q), G, lambda b, h: [(ht[b], range(lens[b]))], 1 / math.sqrt(D)))


def test_queries_of_all_sizes():
    """Queries far below and above fp16's range, zeros, strided rows."""
    H, G, D, page, lens = 1, 6, 128, 128, [200]
    pool = Pool(38, 2, H, D, page, "int8")
    ht, table = pool.tables(lens)
    x = np.random.default_rng(39).standard_normal((1, 2 * G, D))
    for g, s in enumerate([1e-30, 1e-6, 0.0, 1e5, 1e20, 1.0]):
        x[:, g] *= s
    q = bf16(x).cuda()[:, :G]
    for scale in (1e-20, 0.1):
        part = q if scale < 1e-10 else torch.cat([q[:, :3], q[:, 5:]], 1)
        g = part.shape[1]
        out, lse = bsa.decode(part, pool.cache, table, _i32(lens), softmax_scale=scale, out_dtype=torch.float32)
        agree(out, lse, expect(pool, f64(part), g, lambda b, h: [(ht[b], range(lens[b]))], float(np.float32(scale))))


def test_fused_query_rows_and_given_buffers():
    H, G, D, page, lens = 2, 3, 64, 32, [70, 10, 0]
    pool = Pool(40, pages_for(lens, page), H, D, page, "e4m3")
    _, table = pool.tables(lens)
    qkv = _q(41, 3, H * G + 2 * H, D)
    want = bsa.decode(qkv[:, :H * G].contiguous(), pool.cache, table, _i32(lens))
    ws = bsa.alloc_decode_workspace(pool.cache, 3, H * G)
    out, lse = torch.full((3, H * G, D), 5.0, dtype=torch.bfloat16, device="cuda"), torch.full((3, H * G), 5.0, device="cuda")
    for _ in range(3):                                   # whatever the workspace held before
        ws.fill_(255)
        got = bsa.decode(qkv[:, :H * G], pool.cache, table, _i32(lens), out=out, lse=lse, workspace=ws)
        assert got[0] is out and torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_small_workspace_is_refused():
    pool = Pool(42, 1, 1, 64, 16, "e4m3")
    ws = torch.empty(64, dtype=torch.uint8, device="cuda")
    with pytest.raises(bsa.BsattnError):
        bsa.decode(_q(1, 1, 1, 64), pool.cache, _i32([[0]]), _i32([3]), workspace=ws)


@pytest.mark.parametrize("op", ["decode", "prefix"])
def test_repeats_are_equal_bit_for_bit(op):
    H, G, D, page, lens, prefix = 2, 4, 128, 64, [3000, 10, 777, 0], 900
    pool = Pool(43, pages_for(lens + [prefix], page), H, D, page, "int8")
    hp = pool.take(-(-prefix // page))
    _, table = pool.tables(lens)
    q = _q(44, 4, H * G, D)
    call = lambda: bsa.decode(q, pool.cache, table, _i32(lens)) if op == "decode" else \
        bsa.decode_shared_prefix(q, pool.cache, _i32(hp), prefix, table, _i32(lens))  # noqa: E731
    a = call()
    for _ in range(5):
        b = call()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_captured_steps_share_a_workspace():
    """Append and decode, captured twice over one workspace, replayed in turn with the lengths advancing on the
    device: each replay equals the eager calls."""
    H, G, D, page, B = 2, 4, 128, 16, 3
    start, steps = [5, 100, 31], 4
    pool = Pool(45, pages_for([n + steps for n in start], page), H, D, page, "e4m3")
    _, table = pool.tables([n + steps for n in start])
    twin = bsa.KVCache(*(t.clone() for t in (pool.cache.k, pool.cache.v, pool.cache.k_scale, pool.cache.v_scale)))
    n = _i32(start)
    n2 = n.clone()
    bufs = [dict(q=_q(50 + i, B, H * G, D), k=_q(60 + i, B, H, D), v=_q(70 + i, B, H, D)) for i in range(2)]
    ws = bsa.alloc_decode_workspace(pool.cache, B, H * G)

    def step(b, cache, n):
        n += 1
        bsa.kv_append(b["k"], b["v"], cache, table, n)
        return bsa.decode(b["q"], cache, table, n, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(bufs[0], pool.cache, n)                     # first calls outside the capture
    torch.cuda.current_stream().wait_stream(side)
    n.copy_(_i32(start))
    graphs = []
    for b in bufs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = step(b, pool.cache, n)
        graphs.append((g, res))
    for i in range(steps):
        g, res = graphs[i % 2]
        g.replay()
        got = [t.clone() for t in res]
        want = step(bufs[i % 2], twin, n2)
        assert torch.equal(n, n2) and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_captured_fork_and_join():
    """Appends on a side stream of a capture, joined before the decodes; both decodes depend on more than their
    stream's last kernel, one of them through the prefix's own kernel.  Replays see new inputs."""
    H, G, D, page, B, prefix = 8, 2, 128, 64, 16, 5000
    lens = [1 + 37 * i for i in range(B)]
    pool = Pool(132, pages_for(lens + [prefix], page), H, D, page, "int8")
    hp = _i32(pool.take(-(-prefix // page)))
    _, table = pool.tables(lens)
    twin = bsa.KVCache(*(t.clone() for t in (pool.cache.k, pool.cache.v, pool.cache.k_scale, pool.cache.v_scale)))
    n, q, k, v = _i32(lens), _q(133, B, H * G, D), _q(134, B, H, D), _q(135, B, H, D)
    ws = [bsa.alloc_decode_workspace(pool.cache, B, H * G, prefix_len=prefix) for _ in range(2)]

    def step(cache, side):
        main = torch.cuda.current_stream()
        if side is not None:
            side.wait_stream(main)
            with torch.cuda.stream(side):
                bsa.kv_append(k, v, cache, table, n)
            twice = q * 2
            main.wait_stream(side)
        else:
            bsa.kv_append(k, v, cache, table, n)
            twice = q * 2
        a = bsa.decode_shared_prefix(twice, cache, hp, prefix, table, n, workspace=ws[0])
        b = bsa.decode(twice, cache, table, n, workspace=ws[1])
        c = bsa.decode_shared_prefix(twice, cache, hp, prefix, table, n, workspace=ws[0])
        return a + b + c
    step(pool.cache, None)
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g):
        res = step(pool.cache, side)
    for i in range(4):
        q.copy_(_q(140 + i, B, H * G, D))
        k.copy_(_q(150 + i, B, H, D))
        v.copy_(_q(160 + i, B, H, D))
        g.replay()
        got = [t.clone() for t in res]
        for x, y in zip(got, step(twin, None)):
            assert torch.equal(x, y)


def test_other_streams_have_their_own_allocations():
    H, G, D, page, lens = 2, 4, 128, 128, [2000, 500]
    pool = Pool(46, pages_for(lens, page), H, D, page, "e4m3")
    _, table = pool.tables(lens)
    q, n = _q(47, 2, H * G, D), _i32(lens)
    want = bsa.decode(q, pool.cache, table, n)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = [bsa.decode(q, pool.cache, table, n, stream=s if i % 2 else s.cuda_stream)
           for _ in range(4) for i, s in enumerate(streams)]
    torch.cuda.synchronize()
    for o, l in got:
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])


def test_the_default_streams_handle_is_the_default_stream():
    """Its handle is 0 (what current_stream().cuda_stream gives): the calls run behind what is queued there, with
    their outputs allocated there."""
    from block_sparse_flashattention_gb300 import kv_cache
    H, G, D, page, lens = 2, 4, 128, 128, [2000, 500]
    pool = Pool(46, pages_for(lens, page), H, D, page, "e4m3")
    _, table = pool.tables(lens)
    x, n = _q(47, 2, H * G, D), _i32(lens)
    want = bsa.decode(x, pool.cache, table, n)
    seen = kv_cache._elsewhere(pool.cache, 0, torch.cuda.current_stream)
    assert seen == torch.cuda.default_stream() and seen.cuda_stream == 0
    big, q = torch.ones((8192, 8192), dtype=torch.bfloat16, device="cuda"), torch.zeros_like(x)
    torch.cuda.synchronize()
    for _ in range(30):
        big = big @ big * 2.0 ** -13
    q += x * big[0, 0]                                    # queued behind the products; 1 times x
    out, lse = bsa.decode(q, pool.cache, table, n, stream=torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("dtype,G,B", [("e4m3", 2, 3), ("int8", 20, 3), ("e4m3", 4, 40)])
def test_codes_past_32_bits_of_bytes(dtype, G, B):
    """A cache with more than 2^31 bytes of codes gives the bits of a small one with the same rows, wherever its pages
    lie: appended, read back, decoded, behind a prefix (by its own kernel: G = 20, B = 40)."""
    H, D, page, prefix = 8, 128, 128, 1200
    lens = [1 + (61 * i) % 300 for i in range(B)]
    need = pages_for(lens + [prefix], page)
    small = bsa.alloc_kv_cache(need, H, D, dtype=DT[dtype])
    large = bsa.alloc_kv_cache((5 << 29) // (H * page * D), H, D, dtype=DT[dtype])
    rng = np.random.default_rng(190)
    at = torch.from_numpy(np.concatenate([[large.num_pages - 1 - i for i in range(need // 2)],
                                          rng.permutation(large.num_pages - need)[:need - need // 2]]).astype(np.int32)).cuda()
    table, k = torch.zeros((B + 1, -(-prefix // page)), dtype=torch.int32), 0
    for b, n in enumerate(lens + [prefix]):
        table[b, :-(-n // page)] = torch.arange(k, k - (-n // page), dtype=torch.int32)
        k -= -n // page
    table = table.cuda()
    total = sum(lens) + prefix
    x, q = [_q(191 + i, total, H, D) for i in range(2)], _q(193, B, H * G, D)
    n, cu = _i32(lens + [prefix]), _i32(np.concatenate([[0], np.cumsum(lens + [prefix])]).tolist())
    got = []
    for cache, t in ((small, table), (large, at[table.long()])):
        bsa.kv_append(*x, cache, t, n, cu_seqlens=cu)
        got.append([*bsa.kv_read(cache, t, cu, total=total), *bsa.decode(q, cache, t[:B], n[:B]),
                    *bsa.decode_shared_prefix(q, cache, t[B].contiguous(), prefix, t[:B], n[:B])])
    for a, b in zip(*got):
        assert a.isfinite().all() and torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
def test_a_serving_run(dtype):
    """Prompts appended, steps of append + decode, then the cached context read back for the block-sparse forward:
    the forward's row for the newest token equals decode's, by way of the same lists."""
    H, D, page, prompts, steps = 4, 128, 64, [100, 260, 1], 3
    pool = Pool(48, pages_for([n + steps for n in prompts], page), H, D, page, dtype)
    _, table = pool.tables([n + steps for n in prompts])
    cache, B = pool.cache, len(prompts)
    rng = np.random.default_rng(49)
    x = [[bf16(rng.standard_normal((n + steps, H, D))) for n in prompts] for _ in range(3)]
    cu = _i32(np.concatenate([[0], np.cumsum(prompts)]).tolist())
    k, v = (torch.cat([x[j][b][:n] for b, n in enumerate(prompts)]).cuda() for j in (1, 2))
    bsa.kv_append(k, v, cache, table, _i32(prompts), cu_seqlens=cu)
    for s in range(steps):
        lens = [n + s + 1 for n in prompts]
        q, kn, vn = (torch.stack([x[j][b][n + s] for b, n in enumerate(prompts)]).cuda() for j in range(3))
        bsa.kv_append(kn, vn, cache, table, _i32(lens))
        out, lse = bsa.decode(q, cache, table, _i32(lens), out_dtype=torch.float32)
    # the oracle, from the rows that were appended
    qs, scale = f64(q), 1 / math.sqrt(D)
    for b, n in enumerate(lens):
        kq, vq = (c * s[..., None] for c, s in (okv.quantise(f64(x[j][b]), dtype) for j in (1, 2)))
        for h in range(H):
            o, l, spread = okv.attend(qs[b, h], kq[:, h], vq[:, h], scale)
            assert np.all(np.abs(f64(out[b, h]) - o) <= spread * 2.0 ** -10 + 1e-6)
            assert abs(float(lse[b, h]) - l) <= 1e-5
    # the whole context through the framework's forward, one query row a sequence
    total, cuk = sum(lens), _i32(np.concatenate([[0], np.cumsum(lens)]).tolist())
    kr, vr = bsa.kv_read(cache, table, cuk, total=total)
    cuq = _i32(list(range(B + 1)))
    nn = [-(-n // 128) for n in lens]
    meta = bsa.alloc_meta(B, H, varlen=True, total_m_blocks=B, total_n_blocks=sum(nn), max_num_n=max(nn))
    block_map = torch.ones((H, sum(nn)), dtype=torch.uint8, device="cuda")
    block_map[1, nn[0] + nn[1] - 1] = 0                 # head 1 of sequence 1 skips its last tile
    bsa.build_meta(block_map, meta, cu_seqlens_q=cuq, cu_seqlens_k=cuk, seqlen_q=B, seqlen_k=total)
    fo, fl = bsa.forward(q, kr, vr, meta, cu_seqlens_q=cuq, cu_seqlens_k=cuk, out_dtype=torch.float32)
    do, dl = bsa.decode(q, cache, table, _i32(lens), meta=meta, out_dtype=torch.float32)
    # the forward rounds its weights to bf16 (2^-8), and int8 rows were rounded to bf16 (2^-8 of scores and values)
    vmax = float(vr.float().abs().max())
    assert (fo - do).abs().max() <= 5e-3 + (0 if dtype == "e4m3" else 2.0 ** -7 * vmax)
    assert (fl.t() - dl).abs().max() <= (1e-4 if dtype == "e4m3" else 3e-2)
    assert not torch.equal(dl[1, 1], lse[1, 1])
    # all tiles listed: the same keys, cut over the device at other places.  Each LSE is within expect()'s
    # tolerance of the true one, ds + 2^-20 + |lse| 2^-22 with ds = (D + 8) 2^-24 scale max_j |q| . |k_j|,
    # so two of them are within twice that of each other
    kmax = float(kr.float().abs().max()) * float(q.float().abs().sum(-1).max())
    tol = 2 * ((D + 8) * 2.0 ** -24 * scale * kmax + 2.0 ** -20 + float(lse[0].abs().max()) * 2.0 ** -22)
    assert (dl[0] - lse[0]).abs().max() <= tol


def test_new_tokens_over_cached_context():
    """What kv_read's documentation says of a causal prefill over cached context: query rows for the context's positions
    too, whose Q tiles list nothing, and K and V repeated for grouped heads."""
    H, G, D, page, context, new = 2, 2, 64, 32, [300, 128], [90, 200]
    lens = [a + b for a, b in zip(context, new)]
    pool = Pool(196, pages_for(lens, page), H, D, page, "e4m3")
    ht, table = pool.tables(lens)
    cu = _i32(np.concatenate([[0], np.cumsum(lens)]).tolist())
    k, v = (x.repeat_interleave(G, 1) for x in bsa.kv_read(pool.cache, table, cu, total=sum(lens)))
    q = _q(197, sum(lens), H * G, D)
    nb = [-(-n // 128) for n in lens]
    meta = bsa.alloc_meta(2, H * G, varlen=True, total_m_blocks=sum(nb), total_n_blocks=sum(n * n for n in nb), max_num_n=max(nb))
    block_map = torch.cat([torch.ones((H * G, n, n), dtype=torch.uint8).index_fill_(1, torch.arange(c // 128), 0).flatten(1)
                           for n, c in zip(nb, context)], 1).cuda()
    args = dict(cu_seqlens_q=cu, cu_seqlens_k=cu, kind=bsa.MASK_CAUSAL)
    bsa.build_meta(block_map, meta, seqlen_q=sum(lens), seqlen_k=sum(lens), **args)
    out, lse = bsa.forward(q, k, v, meta, out_dtype=torch.float32, **args)
    x = f64(q)
    for b, n in enumerate(lens):
        at = int(cu[b])
        assert not out[at:at + context[b] // 128 * 128].any()           # the context's tiles were left out
        for i in sorted({context[b], context[b] + 1, n - 50, n - 1}):
            for h in range(H * G):
                o, l, _ = okv.attend(x[at + i, h], pool.host("k", ht[b], h // G, range(i + 1)),
                                     pool.host("v", ht[b], h // G, range(i + 1)), 1 / math.sqrt(D))
                # a weight is rounded to bf16, by at most 2^-8 of itself, and the weights sum to 1
                assert np.all(np.abs(f64(out[at + i, h]) - o) <= 2.0 ** -8 * np.max(np.abs(pool.host("v", ht[b], h // G, range(i + 1)))))
                assert abs(float(lse[h, at + i]) - l) <= 1e-4


@pytest.mark.parametrize("listed", [False, True])
def test_native_calls_equal_the_marshalled_ones(monkeypatch, listed):
    """The native form of the calls and the ctypes form give the same bits, and refuse the same arguments."""
    from block_sparse_flashattention_gb300 import kv_cache
    H, G, D, page, lens, prefix = 2, 4, 128, 64, [500, 0, 77], 130
    pool = Pool(90, pages_for(lens + [prefix], page), H, D, page, "e4m3")
    if kv_cache._calls is None:
        pytest.skip("torch_calls.cpp was not compiled for this torch")
    hp = pool.take(-(-prefix // page))
    _, table = pool.tables(lens)
    n, q = _i32(lens), _q(91, 3, H * G, D)
    k, v = _q(92, 3, H, D), _q(93, 3, H, D)
    meta = lists(H, lens, lambda b, h: [0], mask_every=2) if listed else None
    ws = bsa.alloc_decode_workspace(pool.cache, 3, H * G, prefix_len=prefix)
    cu = _i32([0, 500, 500, 577])

    def run():
        c = bsa.KVCache(*(t.clone() for t in (pool.cache.k, pool.cache.v, pool.cache.k_scale, pool.cache.v_scale)))
        bsa.kv_append(k, v, c, table, n)
        return [*(t.view(torch.uint8) for t in (c.k, c.v, c.k_scale, c.v_scale)),
                *bsa.kv_read(c, table, cu, total=577), *bsa.decode(q, c, table, n, meta=meta, workspace=ws),
                *bsa.decode_shared_prefix(q, c, _i32(hp), prefix, table, n, meta=meta, workspace=ws, softmax_scale=0.3)]
    bad = [lambda: bsa.kv_append(k.float(), v, pool.cache, table, n), lambda: bsa.kv_append(k, v[:2], pool.cache, table, n),
           lambda: bsa.kv_append(k, v, pool.cache, table.long(), n), lambda: bsa.kv_append(k, v, pool.cache, table, n[:2]),
           lambda: bsa.kv_append(k, v, pool.cache, table, n, cu_seqlens=n), lambda: bsa.kv_read(pool.cache, table, cu[:3], total=577),
           lambda: bsa.kv_read(pool.cache, table, cu), lambda: bsa.decode(q.float(), pool.cache, table, n, workspace=ws),
           lambda: bsa.decode(q, pool.cache, table[:2], n, workspace=ws), lambda: bsa.decode(q, pool.cache, table, n.cpu(), workspace=ws),
           lambda: bsa.decode(q, pool.cache, table, n, workspace=ws.cpu()), lambda: bsa.decode(q, pool.cache, None, n, workspace=ws),
           lambda: bsa.decode_shared_prefix(q, pool.cache, _i32(hp), 9999, table, n, workspace=ws)]
    status = [lambda: bsa.decode(q[:, :5], pool.cache, table, n, workspace=ws),
              lambda: bsa.decode(q, pool.cache, table, n, workspace=ws, softmax_scale=-1.0),
              lambda: bsa.decode(q, pool.cache, table, n, workspace=ws[:256])]
    got = run()
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for call in status:
        with pytest.raises(bsa.BsattnError):
            call()
    monkeypatch.setattr(kv_cache, "_calls", None)
    for a, b in zip(got, run()):
        assert a.dtype == b.dtype and a.shape == b.shape and torch.equal(a, b)
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for call in status:
        with pytest.raises(bsa.BsattnError):
            call()
