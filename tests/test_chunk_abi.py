"""Refusals of prefill, kv_weigh and kv_evict: every case fails validation on the host, before any CUDA call
(no GPU needed)."""
import pytest

torch = pytest.importorskip("torch")

import block_sparse_flashattention_gb300 as bsa  # noqa: E402
from block_sparse_flashattention_gb300 import _build  # noqa: E402
from tests.test_kv_cache_abi import BAD_CACHES, FAKE, INV, UNS, _cache  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


def _prefill(cache=None, **kw):
    a = dict(q=FAKE, q_stride=512, total=9, B=3, Hq=4, cu_seqlens=FAKE, cache=_cache(**(cache or {})), page_table=FAKE,
             table_stride=2, table_cols=2, seqlens=FAKE, keys=600, kind=bsa.MASK_CAUSAL, mask_params=None,
             softmax_scale=0.1, out=FAKE, out_dtype=bsa.OUT_BF16, lse=FAKE, workspace=FAKE, workspace_bytes=1 << 40,
             stream=0)
    a.update(kw)
    return bsa.bsattn_prefill(**a)


def _weigh(cache=None, **kw):
    a = dict(q=FAKE, q_stride=512, lse=FAKE, total=9, B=3, Hq=4, cu_seqlens=FAKE, cache=_cache(**(cache or {})),
             weights=FAKE, accumulate=1, page_table=FAKE, table_stride=2, table_cols=2, seqlens=FAKE,
             kind=bsa.MASK_CAUSAL, mask_params=None, softmax_scale=0.1, stream=0)
    a.update(kw)
    return bsa.bsattn_kv_weigh(**a)


def _evict(cache=None, **kw):
    a = dict(cache=_cache(**(cache or {})), weights=FAKE, page_table=FAKE, table_stride=2, table_cols=2, seqlens=FAKE,
             B=3, keep=100, recent=10, sinks=4, out_table=None, out_stride=0, out_cols=0, kept=FAKE, lens=FAKE, stream=0)
    a.update(kw)
    return bsa.bsattn_kv_evict(**a)


@pytest.mark.parametrize("cache,expect", BAD_CACHES)
def test_bad_caches(cache, expect):
    for f in (_prefill, _weigh, _evict):
        assert f(cache=cache) == expect


MP = bsa.MaskParams


@pytest.mark.parametrize("kw,expect", [
    (dict(B=0), INV), (dict(total=-1), INV), (dict(Hq=3), INV), (dict(Hq=0), INV), (dict(q=None), INV),
    (dict(q=FAKE + 2), INV), (dict(q_stride=504), INV), (dict(q_stride=516), INV), (dict(seqlens=None), INV),
    (dict(page_table=None), INV), (dict(table_cols=0), INV), (dict(table_stride=1), INV),
    (dict(table_cols=1 << 24, table_stride=1 << 24), INV), (dict(softmax_scale=0.0), INV), (dict(lse=None), INV),
    (dict(softmax_scale=float("nan")), INV), (dict(softmax_scale=float("inf")), INV), (dict(kind=9), INV),
    (dict(kind=bsa.MASK_DOCUMENT, mask_params=MP(doc_id_q=FAKE, doc_id_k=FAKE)), UNS),
    (dict(kind=bsa.MASK_SLIDING_WINDOW), INV), (dict(kind=bsa.MASK_PREFIX), INV),
    (dict(kind=bsa.MASK_SLIDING_WINDOW, mask_params=MP(window_left=-1)), INV),
    (dict(kind=bsa.MASK_SLIDING_WINDOW, mask_params=MP(window_left=1, sink_tokens=-1)), INV),
    (dict(kind=bsa.MASK_PREFIX, mask_params=MP(prefix_len=-1)), INV),
    (dict(Hq=2 * 129, q_stride=2 * 129 * 128), UNS), (dict(total=1 << 30), INV), (dict(B=1 << 30), INV),
])
def test_chunk_calls_refuse(kw, expect):
    assert _prefill(**kw) == expect
    assert _weigh(**kw) == expect


@pytest.mark.parametrize("kw", [
    dict(cu_seqlens=None), dict(out=None), dict(out=FAKE + 4), dict(out_dtype=3), dict(workspace=None),
    dict(workspace=FAKE + 16), dict(workspace_bytes=16), dict(keys=-1), dict(keys=1 << 62)])
def test_prefill_refuses(kw):
    assert _prefill(**kw) == INV


@pytest.mark.parametrize("kw", [dict(cu_seqlens=None), dict(weights=None), dict(weights=FAKE + 4)])
def test_weigh_refuses(kw):
    assert _weigh(**kw) == INV


@pytest.mark.parametrize("kw", [
    dict(B=0), dict(keep=0), dict(keep=-1), dict(recent=-1), dict(sinks=-1), dict(recent=97), dict(sinks=101),
    dict(recent=2 ** 31 - 1, sinks=2 ** 31 - 1), dict(keep=2 ** 31 - 1), dict(weights=None), dict(weights=FAKE + 4),
    dict(seqlens=None), dict(kept=None), dict(lens=None), dict(page_table=None), dict(table_cols=0), dict(table_stride=1),
    dict(out_table=FAKE), dict(out_table=FAKE, out_cols=1, out_stride=0), dict(out_table=FAKE, out_cols=1, out_stride=1, keep=129),
    dict(B=1 << 30)])
def test_evict_refuses(kw):
    assert _evict(**kw) == INV


def test_nothing():
    assert _prefill(total=0, q=None, out=None, lse=None) == bsa.BSATTN_OK
    assert _prefill(total=0, q=None, out=None, lse=None, B=0) == INV


def test_workspace_size():
    n = bsa.bsattn_prefill_workspace_size(_cache(k=None, v=None), 9, 3, 4, 600)
    assert n > 0 and bsa.bsattn_prefill_workspace_size(_cache(), 9, 3, 4, 60000) >= n
    for kw in (dict(B=0), dict(Hq=3), dict(total=-1), dict(keys=-1), dict(B=1 << 30), dict(Hq=2 * 129), dict(keys=1 << 62)):
        with pytest.raises(bsa.BsattnError):
            bsa.bsattn_prefill_workspace_size(_cache(), **{**dict(total=9, B=3, Hq=4, keys=600), **kw})


# ------------------------------------------------------ the torch wrappers --

I32 = dict(dtype=torch.int32)


def _args():
    c = bsa.alloc_kv_cache(4, 2, 64, page_size=16, device="cpu")
    return dict(q=torch.zeros(5, 4, 64, dtype=torch.bfloat16), cache=c, page_table=torch.zeros(3, 2, **I32),
                seqlens=torch.zeros(3, **I32), cu_seqlens=torch.zeros(4, **I32))


COMMON = [
    dict(q=torch.zeros(5, 4, 64)), dict(q=torch.zeros(5, 4, 32, dtype=torch.bfloat16)),
    dict(q=torch.zeros(5, 256, dtype=torch.bfloat16)), dict(q=torch.zeros(5, 64, 4, dtype=torch.bfloat16).transpose(1, 2)),
    dict(seqlens=torch.zeros(2, **I32)), dict(seqlens=torch.zeros(3)), dict(page_table=torch.zeros(3, 2)),
    dict(page_table=torch.zeros(1, 2, **I32).expand(3, 2)), dict(cu_seqlens=torch.zeros(3, **I32)), dict(cu_seqlens=None),
    dict(lse=torch.zeros(4, 5)), dict(lse=torch.zeros(5, 8)[:, ::2]), dict(err_flag=torch.zeros(1)), {}]


@pytest.mark.parametrize("kw", COMMON + [
    dict(out=torch.zeros(5, 4, 128)[..., ::2]), dict(out=torch.zeros(5, 4, 64), out_dtype=torch.bfloat16),
    dict(out_dtype=torch.float16), dict(workspace=torch.zeros(64, 2, dtype=torch.uint8)[:, 0])])
def test_prefill_checks_tensors(kw):
    with pytest.raises(ValueError):                 # the last, the arguments as they are: not on a GPU
        bsa.prefill(**{**_args(), **kw})


@pytest.mark.parametrize("kw", COMMON + [dict(weights=torch.zeros(4, 2, 8)), dict(weights=torch.zeros(4, 2, 16).double()),
                                         dict(weights=torch.zeros(4, 16, 2).transpose(1, 2))])
def test_weigh_checks_tensors(kw):
    a = {**_args(), "lse": torch.zeros(5, 4), "weights": torch.zeros(4, 2, 16), **kw}
    with pytest.raises(ValueError):
        bsa.kv_weigh(**a)


@pytest.mark.parametrize("kw", [
    dict(weights=torch.zeros(4, 2, 8)), dict(seqlens=torch.zeros(2, **I32)), dict(page_table=torch.zeros(3, 2)),
    dict(out_table=torch.zeros(2, 2, **I32)), dict(out_table=torch.zeros(3, 2)), dict(keep=0), dict(recent=-1),
    dict(recent=5, sinks=6), dict(err_flag=torch.zeros(1)), {}])
def test_evict_checks_tensors(kw):
    a = _args()
    a.pop("q"), a.pop("cu_seqlens")
    with pytest.raises(ValueError):
        bsa.kv_evict(**{**a, "weights": torch.zeros(4, 2, 16), "keep": 10, **kw})


@pytest.mark.parametrize("H,G,D,B", [(1, 1, 64, 1), (8, 4, 128, 8), (32, 1, 64, 300), (2, 64, 128, 5), (4, 7, 64, 64), (8, 128, 128, 3)])
def test_a_workspace_serves_fewer_tokens_and_keys(H, G, D, B):
    """Bytes never fall with the tokens or keys of a call."""
    cache = _cache(H=H, D=D)
    last = 0
    for total in sorted({*range(0, 70), *(B * k + d for k in (1, 2, 4, 8, 16, 32, 64, 128) for d in (-1, 0, 1)),
                         *(B * k // G + d for k in (16, 32, 64, 128) for d in (0, 1)), 1000, 5000, 20000}):
        n = [bsa.bsattn_prefill_workspace_size(cache, total, B, H * G, keys) for keys in (0, 300, 40000)]
        assert n == sorted(n) and n[1] >= last
        last = n[1]


def test_evict_the_same_table_by_other_strides():
    assert _evict(out_table=FAKE, out_stride=3, out_cols=2) == INV
