"""kv_weigh: a query whose lse is -inf gives no weight, whatever it or the keys hold; with as many rows as each kernel takes."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import block_sparse_flashattention_gb300 as bsa  # noqa: E402
from tests.chunk_case import Chunks  # noqa: E402
from tests.test_gpu_kv_weights import _lse, _near, _weigh  # noqa: E402

pytestmark = pytest.mark.gpu



def _finite(w, ref):
    assert torch.isfinite(w).all()
    _near(w, ref)


# query heads of a KV head, new tokens: rows of up to 32 columns, up to 64, 128 and several blocks
ROWS = [(1, 4), (4, 7), (1, 40), (3, 20), (1, 64), (2, 64), (1, 200), (7, 50)]


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("G,m", ROWS)
@pytest.mark.parametrize("dtype,D", [("e4m3", 64), ("int8", 128), ("e4m3", 128)])
def test_keys_that_are_no_numbers(dtype, D, G, m, accumulate):
    """The last key, met by the last token alone, is NaN (by its scale, by a code); the last token is switched off."""
    c = Chunks(101, dtype, 2, G, D, 32, [300 + m], [m])
    lse = _lse(c)
    lse[-1] = -math.inf
    ref = c.expect_weights(lse)
    n = 300 + m
    pg, row = int(c.host_table[0][(n - 1) // 32]), (n - 1) % 32
    c.pool.cache.k_scale[pg, 0, row] = math.nan
    if dtype == "e4m3":
        c.pool.cache.k.view(torch.uint8)[pg, 1, row, 3] = 0x7f
    w, err = _weigh(c, lse, accumulate=accumulate)
    assert err == 0
    _finite(w, ref)


@pytest.mark.parametrize("G,m", ROWS)
@pytest.mark.parametrize("dtype,D", [("e4m3", 128), ("int8", 64)])
def test_queries_that_are_no_numbers(dtype, D, G, m):
    """Queries of NaN and of infinities that are switched off leave every weight as it is without them."""
    c = Chunks(102, dtype, 1, G, D, 16, [250 + m], [m])
    lse = _lse(c)
    off = np.random.default_rng(103).random(lse.shape) < 0.3
    off[0, 0] = True
    lse[torch.from_numpy(off).cuda()] = -math.inf
    ref = c.expect_weights(lse)
    at = torch.from_numpy(np.argwhere(off)).cuda()
    c.q[at[:, 0], at[:, 1], 5] = math.nan
    c.q[at[::2, 0], at[::2, 1], 7] = math.inf
    w, err = _weigh(c, lse, accumulate=False)
    assert err == 0
    _finite(w, ref)


@pytest.mark.parametrize("G,m", ROWS)
def test_all_switched_off(G, m):
    c = Chunks(104, "e4m3", 1, G, 64, 64, [100 + m, 70 + m], [m, m])
    c.pool.cache.k_scale[int(c.host_table[0][0])] = math.nan
    lse = torch.full((2 * m, G), -math.inf, device="cuda")
    w, err = _weigh(c, lse, torch.full_like(c.pool.cache.k_scale, 3.0))
    assert err == 0 and (w == 3.0).all()
    w, err = _weigh(c, lse, w, accumulate=False)
    want = c.expect_weights(lse)[0]
    assert err == 0 and np.array_equal(w.cpu().numpy(), np.where(np.isnan(want), 3.0, 0.0))
