"""kv_evict with numbers next to the largest that it takes."""
import pytest

torch = pytest.importorskip("torch")

import block_sparse_flashattention_gb300 as bsa  # noqa: E402
from tests.chunk_case import i32  # noqa: E402
from tests.test_gpu_kv_weights import _evict_case, _state  # noqa: E402

pytestmark = pytest.mark.gpu

MOST = 2 ** 31 - 1 - 128


@pytest.mark.parametrize("keep", [MOST, 2 ** 31 - 4096, 2 ** 31 - 4097])
@pytest.mark.parametrize("in_place", [True, False])
def test_keep_next_to_the_largest(keep, in_place):
    """Entries of `kept` behind the last key are counted past 2^31 by those that write them; nothing around it is written."""
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB")
    pool, ht, table, w = _evict_case(95, "int8", 1, 64, 16, [20], 20)
    out = None if in_place else pool.tables([20])[1]
    guard = 1 << 20
    buf = torch.full((keep + 2 * guard,), 7, dtype=torch.int32, device="cuda")
    lens = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    before = _state(pool, w)
    n = table.shape[1]
    status = bsa.bsattn_kv_evict(pool.cache.ref, w, table, n, n, i32([20]), 1, keep, 0, 0, out, n if out is not None else 0,
                                 n if out is not None else 0, buf.data_ptr() + 4 * guard, lens)
    torch.cuda.synchronize()
    assert status == bsa.BSATTN_OK and lens.tolist() == [20]
    assert (buf[:guard] == 7).all() and (buf[guard + keep:] == 7).all()
    kept = buf[guard:guard + keep]
    assert kept[:20].tolist() == list(range(20))
    for piece in kept[20:].split(1 << 28):
        assert (piece == -1).all()
    if in_place:
        for x, y in zip(before, _state(pool, w)):
            assert (x == y).all()
    del buf, kept, piece
    torch.cuda.empty_cache()
