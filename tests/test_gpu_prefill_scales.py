"""prefill where the scales of cached values differ widely from key tile to key tile, or whole tiles hold no value;
tolerances as derived in chunk_case.Chunks.expect (weights and values are each rounded to 11 bits)."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import block_sparse_flashattention_gb300 as bsa  # noqa: E402
from tests.chunk_case import Chunks, i32  # noqa: E402
from tests.kv_case import agree  # noqa: E402
from tests.test_gpu_prefill import _run, _scales  # noqa: E402

pytestmark = pytest.mark.gpu

TILE = 128
COARSE = 2 * 2.0 ** -11
# New tokens: of the kernel of few query rows, of the one whose tiles are widened once.
FEW, MANY = 2, 260


def _no_values(c, keys, scale):
    """Values of the given keys become rows of zeros with the given scale, on both sides."""
    for j in keys:
        pg, row = c.host_table[0][j // c.pool.page], j % c.pool.page
        c.pool.codes["v"][pg, :, row] = 0
        c.pool.scales["v"][pg, :, row] = scale
    c.pool.cache.v.view(torch.uint8).copy_(torch.from_numpy(c.pool.codes["v"]))
    c.pool.cache.v_scale.copy_(torch.from_numpy(c.pool.scales["v"]))


COPIES = 90


def _check(c, flag=0):
    """Many sequences at once that are all the same one: pieces of work long enough to hold its tiles one after the
    other, and cut at other places for each."""
    m, n = c.news[0], c.lens[0]
    assert len(c.lens) == 1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = bsa.prefill(c.q.repeat(COPIES, 1, 1), c.pool.cache, c.table.expand(COPIES, -1).contiguous(), i32([n] * COPIES),
                           i32([m * b for b in range(COPIES + 1)]), keys=n * COPIES, out_dtype=torch.float32, err_flag=err, **c.kw)
    assert int(err) == flag
    ref = c.expect(COARSE)
    for o, l in zip(out.split(m), lse.split(m)):
        agree(o, l, ref)


# 12 tiles, of which these hold no value
RUNS = [[5], [5, 6], [5, 6, 7], list(range(1, 11)), [10, 11], [0, 1], [0, 1, 4, 5, 8, 9, 10], list(range(12))]


@pytest.mark.parametrize("tiles", RUNS)
@pytest.mark.parametrize("scale", [2.0 ** -126, 0.0])
@pytest.mark.parametrize("m", [FEW, MANY])
@pytest.mark.parametrize("dtype,D", [("e4m3", 64), ("int8", 128)])
def test_tiles_of_zero_values(dtype, D, m, scale, tiles):
    c = Chunks(81, dtype, 2, 2, D, 64, [12 * TILE], [m])
    _no_values(c, [j for t in tiles for j in range(t * TILE, (t + 1) * TILE)], scale)
    _check(c)


@pytest.mark.parametrize("mask", [dict(kind=bsa.MASK_SLIDING_WINDOW, window=150, sinks=0),
                                  dict(kind=bsa.MASK_SLIDING_WINDOW, window=700, sinks=200), dict(kind=bsa.MASK_NONE)])
@pytest.mark.parametrize("dtype,D", [("e4m3", 128), ("int8", 64)])
def test_tiles_of_zero_values_in_the_chunk(dtype, D, mask):
    """Within the new tokens themselves: rows that meet none of them visit the tiles all the same."""
    c = Chunks(82, dtype, 1, 1, D, 32, [1400], [900], **mask)
    _no_values(c, range(640, 1152), 2.0 ** -126)
    _check(c)


@pytest.mark.parametrize("tiles", [[3], [3, 4], [2, 3, 4, 5, 6], [8, 9], [0, 1, 2]])
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("m", [FEW, MANY])
@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
def test_tiles_on_pages_outside_the_cache(dtype, m, page, tiles):
    c = Chunks(83, dtype, 1, 2, 64, page, [10 * TILE], [m])
    for t in tiles:
        c.host_table[0, t * TILE // page:(t + 1) * TILE // page] = -1 if t % 2 else 10 ** 6
    c.table.copy_(torch.from_numpy(c.host_table))
    _check(c, bsa.FLAG_BAD_INDEX)


# 2^60 at first, so that what is left is still a normal number; 12 tiles
FALLS = {
    "two steps of 2^60": lambda t: 60 - 60 * min(t // 4, 2),
    "six steps of 2^20": lambda t: 60 - 20 * min(t // 2, 6),
    "2^30 a tile": lambda t: 60 - 30 * min(t, 5),
    "2^10 a tile": lambda t: 60 - 10 * t,
    "and back": lambda t: 60 - 30 * min(t, 10 - t) if t <= 10 else 60,
    "in turns": lambda t: 40 if t % 2 else -50,
    "up": lambda t: -70 + 10 * t,
    "nothing, then little": lambda t: 60 if t < 4 else -70,
}


@pytest.mark.parametrize("fall", list(FALLS))
@pytest.mark.parametrize("m", [FEW, MANY])
@pytest.mark.parametrize("dtype,D", [("e4m3", 128), ("int8", 64), ("e4m3", 64), ("int8", 128)])
def test_scales_that_fall(dtype, D, m, fall):
    c = Chunks(84, dtype, 1, 1, D, 128, [12 * TILE], [m])
    _scales(c, "v", lambda j: 2.0 ** FALLS[fall](j // TILE))
    _check(c)


@pytest.mark.parametrize("dtype", ["e4m3", "int8"])
def test_small_values_behind_large_ones_that_a_query_does_not_meet(dtype):
    """528 keys, the last 300 new, a window of 64.  Tile 1 holds 20 keys with values 2^100 times the others', which no
    query meets.  The first 256 queries visit it, but those from the 129th on meet no key of it: for them its
    values are as if they were 0."""
    c = Chunks(85, dtype, 1, 1, 64, 128, [528], [300], kind=bsa.MASK_SLIDING_WINDOW, window=64)
    _scales(c, "v", lambda j: 2.0 ** 50 if j < TILE + 20 else 2.0 ** -50)
    out, lse, err = _run(c, out_dtype=torch.float32)
    assert err == 0
    for j in range(TILE + 20):
        c.pool.scales["v"][c.host_table[0][j // c.pool.page], :, j % c.pool.page] = 0
    o, l, to, tl = c.expect(COARSE)
    assert np.all(np.abs(lse.cpu().numpy() - l) <= tl)
    got = out.cpu().numpy().astype(np.float64)
    assert np.all(np.isfinite(got)) and np.all(np.abs(got - o)[TILE:] <= to[TILE:])


def test_largest_scales():
    """Values next to fp32's largest, the others far below: finite, and the small ones within what is documented."""
    for m in (FEW, MANY):
        c = Chunks(86, "int8", 1, 1, 64, 64, [6 * TILE], [m])
        _scales(c, "v", lambda j: 2.0 ** 120 if j // TILE in (1, 4) else 2.0 ** -100)
        out, lse, err = _run(c, out_dtype=torch.float32)
        assert err == 0 and math.isfinite(float(lse.sum()))
        agree(out, lse, c.expect(COARSE))


@pytest.mark.parametrize("tiny", [list(range(12)), [3, 4, 5], [0, 1, 2, 3], [9, 10, 11], [1, 3, 5, 7, 9, 11]])
@pytest.mark.parametrize("m", [FEW, MANY])
@pytest.mark.parametrize("dtype,D", [("e4m3", 128), ("int8", 64)])
def test_smallest_scales(dtype, D, m, tiny):
    """The scale of rows of zeros, 2^-126, under codes that are not 0, alone and among ordinary tiles."""
    c = Chunks(87, dtype, 1, 1, D, 64, [12 * TILE], [m])
    for t in tiny:
        for j in range(t * TILE, (t + 1) * TILE):
            c.pool.scales["v"][c.host_table[0][j // 64], :, j % 64] = 2.0 ** -126
    c.pool.cache.v_scale.copy_(torch.from_numpy(c.pool.scales["v"]))
    _check(c)


def test_zero_scales_under_codes():
    """A scale of 0 makes a value 0 whatever its code is."""
    for dtype in ("e4m3", "int8"):
        c = Chunks(88, dtype, 1, 2, 64, 64, [12 * TILE], [MANY])
        for j in range(4 * TILE, 9 * TILE):
            c.pool.scales["v"][c.host_table[0][j // 64], :, j % 64] = 0
        c.pool.cache.v_scale.copy_(torch.from_numpy(c.pool.scales["v"]))
        _check(c)
