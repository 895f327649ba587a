"""prefill's workspace for a number of keys: a sequence whose keys have no room in it is left, and nothing behind it is
written."""
import pytest

torch = pytest.importorskip("torch")

import block_sparse_flashattention_gb300 as bsa  # noqa: E402
from tests.chunk_case import Chunks, i32  # noqa: E402
from tests.kv_case import agree  # noqa: E402

pytestmark = pytest.mark.gpu

GUARD = 1 << 20


# lens, new tokens, keys -> the sequences that have room.  keys / 128 + B tiles (rounded down), those of a sequence
# side by side; one that has no room still takes its place.
CASES = [
    ([2000, 3000], [600, 700], 2000, [True, False]),         # 17 tiles, of which 16 and 24
    ([2000, 3000], [600, 700], 5000, [True, True]),
    ([2000, 3000], [600, 700], 0, [False, False]),
    ([1, 129, 4000], [1, 129, 900], 130, [True, True, False]),
    ([4000, 1, 129], [900, 1, 129], 130, [False, False, False]),
]


@pytest.mark.parametrize("lens,news,keys,room", CASES)
@pytest.mark.parametrize("dtype,D", [("e4m3", 128), ("int8", 64)])
def test_sequences_without_room(dtype, D, lens, news, keys, room):
    G = 4
    c = Chunks(121, dtype, 1, G, D, 128, lens, news)
    total, B = sum(news), len(lens)
    n = bsa.bsattn_prefill_workspace_size(c.pool.cache.ref, total, B, G, keys)
    ws = torch.full((n + GUARD,), 77, dtype=torch.uint8, device="cuda")
    out, lse = torch.full((total, G, D), 7.0, device="cuda"), torch.full((total, G), 7.0, device="cuda")
    err = i32([0])
    bsa.prefill(c.q, c.pool.cache, c.table, c.seqlens, c.cu, keys=keys, out=out, lse=lse, workspace=ws[:n], err_flag=err, **c.kw)
    torch.cuda.synchronize()
    assert (ws[n:] == 77).all()
    assert int(err) == (0 if all(room) else bsa.FLAG_BAD_SEQLENS)
    ref = c.expect()
    for b in range(B):
        r = slice(c.first[b], c.first[b + 1])
        if room[b]:
            agree(out[r], lse[r], tuple(x[r] for x in ref))
        else:
            assert (out[r] == 7).all() and (lse[r] == 7).all()
