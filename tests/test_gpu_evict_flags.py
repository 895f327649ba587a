"""kv_evict flags every page outside the cache that a key which stays lies on or goes to, whether its row moves or not."""
import pytest

torch = pytest.importorskip("torch")

import block_sparse_flashattention_gb300 as bsa  # noqa: E402
from tests.chunk_case import i32  # noqa: E402
from tests.test_gpu_kv_weights import _err, _evict_case, _evict_check, _state  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,keep,sinks,bad", [
    ([40, 90], 64, 0, (0, 1)),          # all of a short sequence's keys stay where they are
    ([200, 90], 64, 20, (1, 0)),        # the first ones of a long one stay
    ([64, 200], 64, 0, (0, 3)),         # as many keys as are kept
])
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("dtype,D", [("e4m3", 128), ("int8", 64)])
def test_keys_that_stay_on_a_page_outside(dtype, D, in_place, lens, keep, sinks, bad):
    pool, ht, table, w = _evict_case(91, dtype, 2, D, 16, lens, keep)
    out_host, out = (None, None) if in_place else pool.tables([min(n, keep) for n in lens])
    for flag, page in ((0, None), (bsa.FLAG_BAD_INDEX, -1), (bsa.FLAG_BAD_INDEX, 10 ** 6)):
        if page is not None:
            ht[bad] = page
            table.copy_(torch.from_numpy(ht))
        before, err = _state(pool, w), _err()
        kept, new = bsa.kv_evict(pool.cache, w, table, i32(lens), keep, sinks=sinks, out_table=out, err_flag=err)
        assert int(err) == flag
        _evict_check(pool, ht, lens, w, before, keep, 0, sinks, out_host, kept, new)


def test_pages_of_keys_that_go_raise_no_flag():
    """Entries behind a sequence's keys, and pages of keys that do not stay, say nothing."""
    lens, keep = [200, 17], 64
    pool, ht, table, w = _evict_case(92, "int8", 1, 64, 16, lens, keep)
    ht[0, 9] = -1                        # keys 144 .. 159: of less weight than any
    table.copy_(torch.from_numpy(ht))
    before, err = _state(pool, w), _err()
    kept, new = bsa.kv_evict(pool.cache, w, table, i32(lens), keep, recent=4, err_flag=err)
    assert int(err) == 0
    _evict_check(pool, ht, lens, w, before, keep, 4, 0, None, kept, new)
