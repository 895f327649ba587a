"""A sequence of the most keys that a page table's row may have: positions next to 2^31, on few pages that it names over
and over."""
import math

import pytest

torch = pytest.importorskip("torch")

import block_sparse_flashattention_gb300 as bsa  # noqa: E402
from tests.chunk_case import i32  # noqa: E402

pytestmark = pytest.mark.gpu

PAGE, PAGES, D = 16, 4096, 64
COLS = (2 ** 31 - 1 - 128) // PAGE                           # 134217719 pages, 2147483504 keys


@pytest.fixture(scope="module")
def long():
    g = torch.Generator(device="cuda").manual_seed(5)

    def rand(*s):
        return torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)

    cache = bsa.alloc_kv_cache(PAGES, 1, D, page_size=PAGE, dtype=torch.int8)
    short = torch.arange(PAGES, dtype=torch.int32, device="cuda")[None]
    n = PAGES * PAGE
    bsa.kv_append(rand(n, 1, D), rand(n, 1, D), cache, short, i32([n]), cu_seqlens=i32([0, n]))
    table = short.repeat(1, COLS // PAGES + 1)[:, :COLS].contiguous()
    yield cache, short, table, rand
    torch.cuda.empty_cache()


@pytest.mark.parametrize("G", [1, 40])
def test_weights(long, G):
    """Each key's weight is that which it has in a short sequence, whichever of its places wrote it; some place of every
    page does, also where the last pages alone are looked at."""
    cache, short, table, rand = long
    q, lse = rand(1, G, D), torch.zeros(1, G, device="cuda")
    want = bsa.kv_weigh(q, lse, cache, bsa.alloc_kv_weights(cache), short, i32([PAGES * PAGE]), accumulate=False)
    assert (want > 0).all()
    for window in (0, 5000):
        kw = dict(kind=bsa.MASK_SLIDING_WINDOW, mask_params=bsa.MaskParams(window_left=window)) if window else {}
        w, err = torch.full_like(want, -1.0), i32([0])
        bsa.kv_weigh(q, lse, cache, w, table, i32([COLS * PAGE]), accumulate=bool(window), err_flag=err, **kw)
        torch.cuda.synchronize()
        assert int(err) == 0
        if not window:
            assert torch.equal(w, want)
            continue
        met = torch.zeros(PAGES * PAGE, dtype=torch.bool, device="cuda")
        at = torch.arange(COLS * PAGE - window, COLS * PAGE, device="cuda")
        met[table[0, at // PAGE].long() * PAGE + at % PAGE] = True
        w, want = w.view(-1), want.view(-1)
        assert (w[~met] == -1).all()
        assert ((w[met] + 1 - want[met]).abs() <= 2.0 ** -23 * (1 + want[met])).all()


def test_attention(long):
    """A key that is named c times weighs c times as much.  A CTA's sums go over up to 2^31 / 128 / 152 / 2 tiles, each of
    which may leave 2^-23 of them behind: 2^16 2^-23 for the weights' sum, as much for the values'."""
    cache, short, table, rand = long
    q = rand(1, 1, D)
    out, lse = bsa.prefill(q, cache, table, i32([COLS * PAGE]), i32([0, 1]), keys=COLS * PAGE, out_dtype=torch.float32,
                           workspace=bsa.alloc_prefill_workspace(cache, 1, 1, 1, COLS * PAGE))
    k, v = (c.double() * s.double()[..., None] for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
    k, v = k.view(-1, D), v.view(-1, D)
    times = torch.bincount(table[0].long(), minlength=PAGES).double().repeat_interleave(PAGE)
    s = k @ q[0, 0].double() / math.sqrt(D) + times.log()
    p = torch.softmax(s, 0)
    rel = 2 * 2.0 ** -7
    assert abs(float(lse) - float(torch.logsumexp(s, 0))) <= rel
    assert ((out[0, 0].double() - p @ v).abs() <= (rel + 2.0 ** -10) * (p @ v.abs())).all()
