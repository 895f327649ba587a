"""Refusals of the cache calls: every case fails validation on the host, before any
CUDA call (no GPU needed)."""
import pytest

torch = pytest.importorskip("torch")

import block_sparse_flashattention_gb300 as bsa  # noqa: E402
from block_sparse_flashattention_gb300 import _build  # noqa: E402

FAKE = 0x10000
INV, UNS = bsa.BSATTN_ERR_INVALID_ARG, bsa.BSATTN_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


def _cache(**kw):
    a = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, num_pages=8, page_size=128, H=2, D=128, dtype=bsa.KV_E4M3)
    a.update(kw)
    return bsa.bsattn_kv_cache(*(a[n] for n, _ in bsa.bsattn_kv_cache._fields_))


def _append(cache=None, **kw):
    a = dict(k=FAKE, v=FAKE, k_stride=256, v_stride=256, total=3, B=3, cu_seqlens=None, page_table=FAKE,
             table_stride=2, table_cols=2, seqlens=FAKE, cache=_cache(**(cache or {})), stream=0)
    a.update(kw)
    return bsa.bsattn_kv_append(**a)


def _read(cache=None, **kw):
    a = dict(cache=_cache(**(cache or {})), page_table=FAKE, table_stride=2, table_cols=2, B=3, cu_seqlens=FAKE,
             total=9, k=FAKE, v=FAKE, stream=0)
    a.update(kw)
    return bsa.bsattn_kv_read(**a)


def _decode(cache=None, **kw):
    a = dict(q=FAKE, q_stride=512, B=3, Hq=4, cache=_cache(**(cache or {})), page_table=FAKE, table_stride=2,
             table_cols=2, seqlens=FAKE, meta=None, kv_valid_len=None, softmax_scale=0.1, out=FAKE,
             out_dtype=bsa.OUT_BF16, lse=FAKE, workspace=FAKE, workspace_bytes=1 << 40, stream=0)
    a.update(kw)
    return bsa.bsattn_decode(**a)


def _prefix(cache=None, **kw):
    a = dict(q=FAKE, q_stride=512, B=3, Hq=4, cache=_cache(**(cache or {})), prefix_table=FAKE, prefix_len=200,
             page_table=FAKE, table_stride=2, table_cols=2, seqlens=FAKE, meta=None, kv_valid_len=None,
             softmax_scale=0.1, out=FAKE, out_dtype=bsa.OUT_BF16, lse=FAKE, workspace=FAKE,
             workspace_bytes=1 << 40, stream=0)
    a.update(kw)
    return bsa.bsattn_decode_shared_prefix(**a)


BAD_CACHES = [
    (dict(D=96), UNS), (dict(page_size=8), UNS), (dict(page_size=256), UNS), (dict(page_size=48), UNS),
    (dict(dtype=7), INV), (dict(H=0), INV), (dict(num_pages=-1), INV), (dict(k=None), INV), (dict(v=None), INV),
    (dict(k_scale=None), INV), (dict(v_scale=None), INV), (dict(k=FAKE + 8), INV), (dict(v=FAKE + 4), INV),
    (dict(k_scale=FAKE + 4), INV), (dict(num_pages=1 << 23, H=2), INV),
]


@pytest.mark.parametrize("cache,expect", BAD_CACHES)
def test_bad_caches(cache, expect):
    for f in (_append, _read, _decode, _prefix):
        assert f(cache=cache) == expect


@pytest.mark.parametrize("kw", [
    dict(B=0), dict(total=-1), dict(total=4), dict(k=None), dict(v=None), dict(k=FAKE + 2), dict(k_stride=255),
    dict(k_stride=260), dict(v_stride=128), dict(seqlens=None), dict(page_table=None), dict(table_cols=0),
    dict(table_stride=1), dict(table_cols=1 << 24, table_stride=1 << 24)])
def test_append_refuses(kw):
    assert _append(**kw) == INV


def test_append_of_nothing():
    assert _append(total=0, cu_seqlens=FAKE) == bsa.BSATTN_OK


def test_nothing_has_no_address():
    """An empty tensor's address is null; the other arguments are checked all the same."""
    none = dict(total=0, k=None, v=None)
    assert _append(cu_seqlens=FAKE, **none) == bsa.BSATTN_OK and _read(**none) == bsa.BSATTN_OK
    for bad in (dict(B=0), dict(seqlens=None), dict(table_cols=0), dict(k_stride=255)):
        assert _append(**{**none, "cu_seqlens": FAKE, **bad}) == INV
    for bad in (dict(B=0), dict(cu_seqlens=None), dict(page_table=None)):
        assert _read(**{**none, **bad}) == INV
    assert _append(**none) == INV                  # B rows are due without offsets


@pytest.mark.parametrize("kw", [
    dict(B=0), dict(total=-1), dict(cu_seqlens=None), dict(k=None), dict(v=None), dict(k=FAKE + 8), dict(v=FAKE + 2),
    dict(page_table=None), dict(table_cols=0), dict(table_stride=0)])
def test_read_refuses(kw):
    assert _read(**kw) == INV


def test_read_of_nothing():
    assert _read(total=0) == bsa.BSATTN_OK


def _meta(**kw):
    a = dict(full_cnt=FAKE, full_idx=FAKE, mask_cnt=FAKE, mask_idx=FAKE, varlen=0, B=3, H=2, num_m=1, num_n=2)
    a.update(kw)
    return bsa.Meta(**a)


VARLEN = dict(varlen=1, num_m=0, total_m_blocks=3, total_n_blocks=6, cu_total_m_blocks=FAKE, cu_block_idx_offsets=FAKE)


@pytest.mark.parametrize("kw,expect", [
    (dict(B=0), INV), (dict(Hq=3), INV), (dict(Hq=0), INV), (dict(q=None), INV), (dict(q=FAKE + 2), INV),
    (dict(q_stride=504), INV), (dict(q_stride=516), INV), (dict(out=None), INV), (dict(out=FAKE + 4), INV),
    (dict(lse=None), INV), (dict(seqlens=None), INV), (dict(softmax_scale=0.0), INV),
    (dict(softmax_scale=float("nan")), INV), (dict(softmax_scale=float("inf")), INV), (dict(out_dtype=3), INV),
    (dict(workspace=None), INV), (dict(workspace=FAKE + 16), INV), (dict(workspace_bytes=16), INV),
    (dict(Hq=2 * 129, q_stride=2 * 129 * 128), UNS), (dict(kv_valid_len=FAKE), INV),
    (dict(meta=_meta(num_m=2)), INV), (dict(meta=_meta(H=4)), INV), (dict(meta=_meta(B=2)), INV),
    (dict(meta=_meta(tile_m=256)), UNS), (dict(meta=_meta(full_cnt=None)), INV),
    (dict(meta=_meta(**{**VARLEN, "total_m_blocks": 4})), INV),
    (dict(meta=_meta(**{**VARLEN, "cu_block_idx_offsets": None})), INV),
    (dict(meta=_meta(**{**VARLEN, "num_n": 0}), kv_valid_len=FAKE), INV),
])
def test_decode_refuses(kw, expect):
    assert _decode(**kw) == expect
    assert _prefix(**kw) == expect


@pytest.mark.parametrize("kw", [dict(table_cols=0), dict(page_table=None), dict(table_stride=1)])
def test_decode_refuses_tables(kw):
    assert _decode(**kw) == INV


@pytest.mark.parametrize("kw", [dict(prefix_len=-1), dict(prefix_table=None), dict(prefix_len=(1 << 31) - 1),
                                dict(prefix_len=0, table_cols=0)])
def test_prefix_refuses(kw):
    assert _prefix(**kw) == INV


def test_workspace_size():
    n = bsa.bsattn_decode_workspace_size(_cache(k=None, v=None), 3, 4)
    assert n > 0 and bsa.bsattn_decode_workspace_size(_cache(), 3, 4, 1000) >= n
    for kw in (dict(B=0), dict(Hq=3), dict(prefix_len=-1), dict(B=1 << 24), dict(Hq=2 * 129)):
        with pytest.raises(bsa.BsattnError):
            bsa.bsattn_decode_workspace_size(_cache(), **{**dict(B=3, Hq=4, prefix_len=0), **kw})


# -------------------------------------------------------- the native calls --

def test_native_calls_are_compiled_anew_for_another_torch(monkeypatch, tmp_path):
    if not _build.build_calls():
        pytest.skip("torch_calls.cpp does not compile here")
    assert _build.calls_up_to_date(torch.__version__) and not _build.calls_up_to_date("0.1")
    stamp = tmp_path / "version"
    stamp.write_text("0.1")
    monkeypatch.setattr(_build, "CALLS_TORCH", str(stamp))
    ran = []

    class Failed:
        returncode, stderr = 1, "not run"
    monkeypatch.setattr(_build.subprocess, "run", lambda cmd, **kw: ran.append(cmd) or Failed)
    assert not _build.build_calls() and len(ran) == 1 and ran[0][0] == "g++"
    stamp.write_text(torch.__version__)
    assert _build.build_calls() and len(ran) == 1


def test_native_calls_of_another_torch_are_left_with_a_warning(monkeypatch):
    import sys
    import types
    from block_sparse_flashattention_gb300 import kv_cache
    other = types.ModuleType("other")
    other.torch_version = lambda: "0.1"
    monkeypatch.setitem(sys.modules, "block_sparse_flashattention_gb300._torch_calls", other)
    monkeypatch.setattr(bsa, "_torch_calls", other, raising=False)
    for name in ("_calls", "torch"):                # as they were when this is over: bound later, or bound already
        monkeypatch.setattr(kv_cache, name, None if name == "_calls" else kv_cache.torch)
    with pytest.warns(UserWarning, match="compiled for torch 0.1"):
        kv_cache._bind()
    assert kv_cache._calls is None


# ------------------------------------------------------ the torch wrappers --

def _cpu_cache(**kw):
    return bsa.alloc_kv_cache(4, 2, 64, page_size=16, device="cpu", **kw)


def test_cache_object():
    c = _cpu_cache()
    assert c.k.dtype == torch.float8_e4m3fn and tuple(c.k.shape) == (4, 2, 16, 64) and not c.k.view(torch.uint8).any()
    assert _cpu_cache(dtype=torch.int8).v.dtype == torch.int8
    with pytest.raises(ValueError):
        _cpu_cache(dtype=torch.bfloat16)
    for bad in ((c.k, c.v.view(torch.int8), c.k_scale, c.v_scale), (c.k, c.v[:3], c.k_scale, c.v_scale),
                (c.k, c.v, c.k_scale.double(), c.v_scale), (c.k, c.v, c.k_scale[..., :8], c.v_scale),
                (c.k, c.v.transpose(1, 2), c.k_scale, c.v_scale)):
        with pytest.raises(ValueError):
            bsa.KVCache(*bad)


def _args(B=3):
    i32 = dict(dtype=torch.int32)
    return dict(k=torch.zeros(B, 2, 64, dtype=torch.bfloat16), v=torch.zeros(B, 2, 64, dtype=torch.bfloat16),
                cache=_cpu_cache(), page_table=torch.zeros(B, 1, **i32), seqlens=torch.zeros(B, **i32))


@pytest.mark.parametrize("change", [
    lambda a: a.update(k=a["k"].float()), lambda a: a.update(k=a["k"][:, :1]), lambda a: a.update(v=a["v"][:2]),
    lambda a: a.update(k=a["k"].transpose(1, 2).contiguous().transpose(1, 2)),
    lambda a: a.update(page_table=a["page_table"].long()), lambda a: a.update(seqlens=a["seqlens"][:2]),
    lambda a: a.update(seqlens=a["seqlens"].float()), lambda a: a.update(page_table=a["page_table"][:, 0]),
    lambda a: a.update(page_table=torch.zeros(1, 4, dtype=torch.int32).expand(3, 4)),
    lambda a: a.update(cu_seqlens=torch.zeros(3, dtype=torch.int32)),
    lambda a: a.update(err_flag=torch.zeros(1))])
def test_append_checks_tensors(change):
    a = _args()
    change(a)
    with pytest.raises(ValueError):
        bsa.kv_append(**a)


def test_read_checks_tensors():
    a, cu = _args(), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        bsa.kv_read(a["cache"], a["page_table"], cu)
    with pytest.raises(ValueError):
        bsa.kv_read(a["cache"], a["page_table"], cu[:3], total=3)
    with pytest.raises(ValueError):
        bsa.kv_read(a["cache"], a["page_table"], cu, k=a["k"])
    with pytest.raises(ValueError):
        bsa.kv_read(a["cache"], a["page_table"], cu, k=a["k"], v=a["v"], total=5)


@pytest.mark.parametrize("kw", [
    dict(q=torch.zeros(3, 4, 64)), dict(q=torch.zeros(3, 4, 32, dtype=torch.bfloat16)),
    dict(seqlens=torch.zeros(2, dtype=torch.int32)), dict(out=torch.zeros(3, 4, 64)[..., ::2]),
    dict(out=torch.zeros(3, 4, 64), out_dtype=torch.bfloat16), dict(out_dtype=torch.float16),
    dict(lse=torch.zeros(4, 3)), dict(kv_valid_len=torch.zeros(3, 1, dtype=torch.int32)),
    dict(workspace=torch.zeros(64, 2, dtype=torch.uint8)[:, 0])])
def test_decode_checks_tensors(kw):
    a = _args()
    b = dict(q=torch.zeros(3, 4, 64, dtype=torch.bfloat16), cache=a["cache"], page_table=a["page_table"],
             seqlens=a["seqlens"])
    b.update(kw)
    with pytest.raises(ValueError):
        bsa.decode(**b)
    with pytest.raises(ValueError):
        bsa.decode_shared_prefix(prefix_table=torch.zeros(1, dtype=torch.int32), prefix_len=3, **b)


def test_prefix_checks_tensors():
    a = _args()
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    for table, n in ((None, 3), (torch.zeros(1, dtype=torch.int32), 17), (torch.zeros(1), 3),
                     (torch.zeros(1, dtype=torch.int32), -1)):
        with pytest.raises(ValueError):
            bsa.decode_shared_prefix(q, a["cache"], table, n, a["page_table"], a["seqlens"])
