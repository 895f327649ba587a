"""kv_weigh without query rows: nothing is done; with an error word the sequences' numbers are checked all the same."""
import pytest

torch = pytest.importorskip("torch")

import block_sparse_flashattention_gb300 as bsa  # noqa: E402
from block_sparse_flashattention_gb300 import _build  # noqa: E402
from tests.test_chunk_abi import _weigh  # noqa: E402
from tests.test_kv_cache_abi import FAKE, INV  # noqa: E402


def test_no_rows_and_no_error_word():
    """Returns before any CUDA call, as prefill does (no GPU needed)."""
    _build.build()
    for Hq in (4, 2 * 40, 2 * 128):
        kw = dict(total=0, Hq=Hq, q_stride=Hq * 128)
        assert _weigh(**kw, q=None, lse=None) == bsa.BSATTN_OK
        assert _weigh(**kw) == bsa.BSATTN_OK
        assert _weigh(**kw, B=0) == INV and _weigh(**kw, weights=None) == INV and _weigh(**kw, cu_seqlens=None) == INV
        assert _weigh(**kw, q=FAKE + 2) == INV


@pytest.mark.gpu
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("G", [1, 16, 33, 40, 128])
def test_no_rows(G, accumulate):
    from tests.chunk_case import Chunks, i32
    c = Chunks(111, "int8", 1, G, 64, 16, [40, 70], [0, 0])
    for cu, lens, flag in (([0, 0, 0], [40, 70], 0), ([0, 1, 0], [40, 70], bsa.FLAG_BAD_SEQLENS),
                           ([0, 0, 0], [40, 10 ** 6], bsa.FLAG_BAD_SEQLENS)):
        w, err = torch.full_like(c.pool.cache.k_scale, 3.0), i32([0])
        bsa.kv_weigh(c.q, torch.zeros(0, G, device="cuda"), c.pool.cache, w, c.table, i32(lens), cu_seqlens=i32(cu),
                     accumulate=accumulate, err_flag=err)
        assert int(err) == flag and (w == 3.0).all()
        bsa.kv_weigh(c.q, torch.zeros(0, G, device="cuda"), c.pool.cache, w, c.table, i32(lens), cu_seqlens=i32(cu),
                     accumulate=accumulate)
        assert (w == 3.0).all()
