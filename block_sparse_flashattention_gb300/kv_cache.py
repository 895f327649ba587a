"""The paged 8-bit K/V cache and the attention of single query tokens over it.

``kv_append`` quantises new K and V rows into a cache's pages, ``kv_read`` reads
them back as packed bf16 rows (what ``forward`` takes), ``decode`` attends one query token per sequence over them, and
``decode_shared_prefix`` does so for a batch behind one common prefix.  These are
calls of the C functions of the same names (bsattn_*, include/bsattn.h, where the
formats and faults are described) with torch checks and allocations around them.

    cache = bsa.alloc_kv_cache(num_pages, H, D)                 # e4m3, pages of 128
    bsa.kv_append(k, v, cache, page_table, seqlens)             # k, v [B, H, D]: a token each
    out, lse = bsa.decode(q, cache, page_table, seqlens)        # q [B, Hq, D]

Work is queued on ``stream`` (a torch stream or its handle; the current stream of the
cache's device when None); outputs and workspaces that a call allocates belong to that
stream, and tensors that come from another one are the caller's to keep until the work is
done.  Device faults
(a page outside the cache, lengths that do not fit) set FLAG_* bits in ``err_flag``.
"""
from __future__ import annotations

import ctypes
import math
import warnings

from ._binding import (BSATTN_OK, KV_E4M3, KV_INT8, OUT_BF16, OUT_F32, BsattnError, bsattn_decode_workspace_size,
                       bsattn_kv_cache, library)


def _check(status: int, where: str) -> None:
    if status != BSATTN_OK:
        raise BsattnError(status, where)


# Bound by the first KVCache, so that importing the package does not import torch.
torch = BF16 = F32 = I32 = _lib = _raw_stream = _current_device = _calls = None


def _bind() -> None:
    global torch, BF16, F32, I32, _lib, _raw_stream, _current_device, _calls
    import torch as t
    BF16, F32, I32 = t.bfloat16, t.float32, t.int32
    # The current stream's handle: the raw form saves the stream object that the public
    # call makes (2.9 us of a decode call's host time).
    _raw_stream = getattr(t._C, "_cuda_getCurrentRawStream", None) or (lambda i: t.cuda.current_stream(i).cuda_stream)
    _current_device = getattr(t._C, "_cuda_getDevice", None) or t.cuda.current_device
    _lib = library()
    # The ordinary calls in native code (csrc/torch_calls.cpp), where it was compiled for
    # this torch: 8 us of host time for a decode call, against 17 here.
    try:
        from . import _torch_calls as calls
        if calls.torch_version() == t.__version__.split("+")[0]:
            calls.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
                _lib.bsattn_kv_append, _lib.bsattn_kv_read, _lib.bsattn_decode, _lib.bsattn_decode_shared_prefix)))
            _calls = calls
        else:
            warnings.warn(f"the native cache calls were compiled for torch {calls.torch_version()}, not {t.__version__}: "
                          "they are marshalled through ctypes until the package is built again", stacklevel=3)
    except ImportError:
        pass
    torch = t


class KVCache:
    """A paged cache over caller-owned tensors (kept, not copied).

    k, v: torch.float8_e4m3fn or torch.int8 [num_pages, H, page_size, D];
    k_scale, v_scale: float32 [num_pages, H, page_size]; contiguous, one device."""

    __slots__ = ("k", "v", "k_scale", "v_scale", "num_pages", "H", "page_size", "D", "dtype", "device", "index", "c", "ref",
                 "scale", "at")

    def __init__(self, k, v, k_scale, v_scale):
        if torch is None:
            _bind()
        if k.dtype not in (torch.float8_e4m3fn, torch.int8) or v.dtype != k.dtype:
            raise ValueError("k and v must both be torch.float8_e4m3fn or torch.int8")
        if k_scale.dtype != torch.float32 or v_scale.dtype != torch.float32:
            raise ValueError("k_scale and v_scale must be torch.float32")
        if k.dim() != 4 or v.shape != k.shape or k_scale.shape != k.shape[:3] or v_scale.shape != k.shape[:3]:
            raise ValueError("k, v must be [num_pages, H, page_size, D] and the scales [num_pages, H, page_size]")
        for t in (k, v, k_scale, v_scale):
            if t.device != k.device:
                raise ValueError("the cache's tensors must be on one device")
            if not t.is_contiguous():
                raise ValueError("the cache's tensors must be contiguous")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.num_pages, self.H, self.page_size, self.D = k.shape
        self.dtype, self.device, self.index = k.dtype, k.device, k.get_device()   # -1: not on a GPU
        self.scale = 1.0 / math.sqrt(max(self.D, 1))
        self.c = bsattn_kv_cache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                 self.num_pages, self.page_size, self.H, self.D,
                                 KV_INT8 if k.dtype == torch.int8 else KV_E4M3)
        self.ref, self.at = ctypes.pointer(self.c), ctypes.addressof(self.c)


def alloc_kv_cache(num_pages: int, H: int, D: int, *, page_size: int = 128, dtype=None, device="cuda") -> KVCache:
    """A cache of num_pages pages, zero-filled; dtype torch.float8_e4m3fn (default) or torch.int8."""
    if torch is None:
        _bind()
    dtype = torch.float8_e4m3fn if dtype is None else dtype
    if dtype not in (torch.float8_e4m3fn, torch.int8):
        raise ValueError("dtype must be torch.float8_e4m3fn or torch.int8")
    codes = [torch.zeros((num_pages, H, page_size, D), dtype=torch.uint8, device=device).view(dtype) for _ in range(2)]
    scales = [torch.zeros((num_pages, H, page_size), dtype=torch.float32, device=device) for _ in range(2)]
    return KVCache(codes[0], codes[1], scales[0], scales[1])


def _elsewhere(cache, stream, call):
    """Runs call() with the cache's device current and, if a stream is given, that
    stream current, so that allocations and launches inside belong to them."""
    if cache.index < 0:
        return call()
    with torch.cuda.device(cache.device):
        if stream is None:
            return call()
        if isinstance(stream, int):
            # the default stream's handle is 0, which ExternalStream takes for a stream of torch's pool
            stream = torch.cuda.ExternalStream(stream, device=cache.device) if stream else \
                torch.cuda.default_stream(cache.device)
        elif stream.device != cache.device:
            raise ValueError("stream must be of the cache's device")
        with torch.cuda.stream(stream):
            return call()


def _on_gpu(cache):
    if cache.index < 0:
        raise ValueError("the cache is not on a CUDA device")


# Full checks, with the reason in the error.  The calls below first test in one
# expression what an ordinary call satisfies and come here only if that fails.

def _ints(t, name, dim, device):
    if t.dtype != torch.int32 or t.dim() != dim or t.device != device:
        raise ValueError(f"{name} must be a {dim}-D torch.int32 tensor on the cache's device")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must be contiguous along its last dimension")


def _err(t, device):
    if t is not None:
        _ints(t, "err_flag", 1, device)
        if t.numel() < 1:
            raise ValueError("err_flag must hold one element")


def _table(t, name, B, device):
    """(row stride, columns) of a page table of B rows."""
    _ints(t, name, 2, device)
    rows, cols = t.shape
    if rows != B:
        raise ValueError(f"{name} must have one row per sequence")
    stride = t.stride(0) if rows > 1 else cols
    if stride < cols:
        raise ValueError(f"{name}'s rows must not overlap")
    return stride, cols


def _rows(t, name, H, D, device):
    """Elements from token to token of bf16 rows [tokens, H, D] whose [H, D] part is contiguous."""
    if t.dtype != torch.bfloat16 or t.dim() != 3 or t.shape[1] != H or t.shape[2] != D or t.device != device:
        raise ValueError(f"{name} must be a torch.bfloat16 tensor [tokens, {H}, {D}] on the cache's device")
    s0, s1, s2 = t.stride()
    if s2 != 1 or (s1 != D and H > 1):
        raise ValueError(f"{name}'s heads and elements must be contiguous")
    return s0 if t.shape[0] > 1 else H * D


def kv_append(k, v, cache: KVCache, page_table, seqlens, *, cu_seqlens=None, err_flag=None, stream=None) -> KVCache:
    """Quantises k, v (bf16 [total, H, D]; tokens may be any multiple of 8 elements
    apart) into the cache and returns it.

    cu_seqlens None: one new token per sequence; else int32 [B+1], the rows of each
    sequence's new tokens.  seqlens int32 [B]: the lengths after the append (0: a
    padding row); page_table int32 [B, pages]."""
    if _calls is not None and stream is None and err_flag is None:
        status = _calls.kv_append(cache.at, cache.index, k, v, page_table, seqlens, cu_seqlens)
        if status is not None:
            if status:
                raise BsattnError(status, "bsattn_kv_append")
            return cache
    if stream is not None or (cache.index >= 0 and cache.index != _current_device()):
        return _elsewhere(cache, stream, lambda: kv_append(k, v, cache, page_table, seqlens, cu_seqlens=cu_seqlens,
                                                           err_flag=err_flag))
    dev, B = cache.device, page_table.shape[0]
    ks, vs = _rows(k, "k", cache.H, cache.D, dev), _rows(v, "v", cache.H, cache.D, dev)
    total = k.shape[0]
    if v.shape[0] != total:
        raise ValueError("k and v must hold the same tokens")
    stride, cols = _table(page_table, "page_table", B, dev)
    _ints(seqlens, "seqlens", 1, dev)
    if seqlens.shape[0] != B:
        raise ValueError("seqlens must have one entry per sequence")
    if cu_seqlens is not None:
        _ints(cu_seqlens, "cu_seqlens", 1, dev)
        if cu_seqlens.shape[0] != B + 1:
            raise ValueError("cu_seqlens must have B + 1 entries")
    _err(err_flag, dev)
    _on_gpu(cache)
    _check(_lib.bsattn_kv_append(k.data_ptr(), v.data_ptr(), ks, vs, total, B,
                                 None if cu_seqlens is None else cu_seqlens.data_ptr(), page_table.data_ptr(),
                                 stride, cols, seqlens.data_ptr(), cache.ref,
                                 None if err_flag is None else err_flag.data_ptr(), _raw_stream(cache.index)),
           "bsattn_kv_append")
    return cache


def kv_read(cache: KVCache, page_table, cu_seqlens, *, total=None, k=None, v=None, err_flag=None, stream=None):
    """The cached rows of every sequence, packed: (k, v) bf16 [total, H, D], sequence
    b's positions 0, 1, ... in rows cu_seqlens[b] .. cu_seqlens[b+1] (int32 [B+1]).

    total: rows to allocate when k and v are not given (cu_seqlens[-1], which lives on
    the device); rows outside every sequence are not written.

    A causal prefill of new tokens over cached context: ``forward`` counts query positions
    from 0 in every sequence, so give it query rows for the context's positions too (of any
    content) and list nothing for their Q tiles; repeat k and v along their heads
    (repeat_interleave) where query heads are grouped."""
    if _calls is not None and stream is None and err_flag is None and k is None and v is None:
        got = _calls.kv_read(cache.at, cache.index, page_table, cu_seqlens, total)
        if got is not None:
            if got.__class__ is tuple:
                return got
            raise BsattnError(got, "bsattn_kv_read")
    if stream is not None or (cache.index >= 0 and cache.index != _current_device()):
        return _elsewhere(cache, stream, lambda: kv_read(cache, page_table, cu_seqlens, total=total, k=k, v=v,
                                                         err_flag=err_flag))
    dev, B = cache.device, page_table.shape[0]
    stride, cols = _table(page_table, "page_table", B, dev)
    _ints(cu_seqlens, "cu_seqlens", 1, dev)
    if cu_seqlens.shape[0] != B + 1:
        raise ValueError("cu_seqlens must have B + 1 entries")
    _err(err_flag, dev)
    if (k is None) != (v is None):
        raise ValueError("give both k and v, or neither")
    if k is None:
        if total is None:
            raise ValueError("total is needed to allocate k and v")
        shape = (total, cache.H, cache.D)
        k, v = torch.empty(shape, dtype=BF16, device=dev), torch.empty(shape, dtype=BF16, device=dev)
    else:
        for t, name in ((k, "k"), (v, "v")):
            _rows(t, name, cache.H, cache.D, dev)
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
        if v.shape[0] != k.shape[0] or (total is not None and total != k.shape[0]):
            raise ValueError("k, v and total disagree")
    _on_gpu(cache)
    _check(_lib.bsattn_kv_read(cache.ref, page_table.data_ptr(), stride, cols, B, cu_seqlens.data_ptr(), k.shape[0],
                               k.data_ptr(), v.data_ptr(), None if err_flag is None else err_flag.data_ptr(),
                               _raw_stream(cache.index)), "bsattn_kv_read")
    return k, v


def alloc_decode_workspace(cache: KVCache, B: int, Hq: int, *, prefix_len: int = 0):
    """Workspace of a decode call for B sequences and Hq query heads (prefix_len as in
    ``decode_shared_prefix``).  It can be kept from call to call; two calls that may
    run at the same time need one each."""
    return torch.empty(bsattn_decode_workspace_size(cache.ref, B, Hq, prefix_len), dtype=torch.uint8,
                       device=cache.device)


def _meta_fits(meta, index):
    """Whether a Meta's tensors are contiguous int32 tensors of device `index` (addresses are taken as given)."""
    for t in (meta.full_cnt, meta.full_idx, meta.mask_cnt, meta.mask_idx, meta.cu_block_idx_offsets):
        if t is not None and not isinstance(t, int) and not (t.dtype is I32 and t.get_device() == index and
                                                             t.is_contiguous()):
            return False
    return True


def _decode_checks(q, cache, prefix_table, prefix_len, page_table, seqlens, meta, kv_valid_len, out, out_dtype, lse,
                   workspace, err_flag):
    dev = cache.device
    if q.dim() != 3:
        raise ValueError("q must be [B, Hq, D]")
    B, Hq = q.shape[0], q.shape[1]
    _rows(q, "q", Hq, cache.D, dev)
    if page_table is not None:
        _table(page_table, "page_table", B, dev)
    elif prefix_table is None:
        raise ValueError("page_table is needed")
    _ints(seqlens, "seqlens", 1, dev)
    if seqlens.shape[0] != B:
        raise ValueError("seqlens must have one entry per sequence")
    if meta is not None and not _meta_fits(meta, cache.index):
        raise ValueError("meta's tensors must be contiguous torch.int32 tensors on the cache's device")
    if kv_valid_len is not None:
        if meta is None:
            raise ValueError("kv_valid_len belongs to the listed tiles of meta")
        _ints(kv_valid_len, "kv_valid_len", 2, dev)
        if tuple(kv_valid_len.shape) != (B, meta.num_n) or not kv_valid_len.is_contiguous():
            raise ValueError("kv_valid_len must be a contiguous [B, meta.num_n] tensor")
    if prefix_table is not None:
        _ints(prefix_table, "prefix_table", 1, dev)
        if prefix_len < 0 or prefix_table.shape[0] * cache.page_size < prefix_len:
            raise ValueError("prefix_table does not hold prefix_len tokens")
    _err(err_flag, dev)
    if out_dtype not in (None, BF16, F32):
        raise ValueError("out_dtype must be torch.bfloat16 or torch.float32")
    if out is not None and (out.dtype not in (BF16, F32) or (out_dtype is not None and out.dtype != out_dtype) or
                            out.shape != q.shape or out.device != dev or not out.is_contiguous()):
        raise ValueError("out must be a contiguous [B, Hq, D] tensor of out_dtype on the cache's device")
    if lse is not None and (lse.dtype != F32 or tuple(lse.shape) != (B, Hq) or lse.device != dev or
                            not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 [B, Hq] tensor on the cache's device")
    if workspace is not None and (workspace.device != dev or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous tensor on the cache's device")
    _on_gpu(cache)


def _decode(q, cache, prefix_table, prefix_len, page_table, seqlens, meta, kv_valid_len, softmax_scale, out,
            out_dtype, lse, workspace, err_flag, stream):
    if stream is not None or (cache.index >= 0 and cache.index != _current_device()):
        return _elsewhere(cache, stream, lambda: _decode(q, cache, prefix_table, prefix_len, page_table, seqlens,
                                                         meta, kv_valid_len, softmax_scale, out, out_dtype, lse,
                                                         workspace, err_flag, None))
    index, shape = cache.index, q.shape
    # what a step of a serving loop passes: contiguous tensors of one device, no error word,
    # outputs allocated here; anything else takes the full checks
    if not (len(shape) == 3 and q.dtype is BF16 and shape[2] == cache.D and q.is_contiguous() and
            q.get_device() == index >= 0 and seqlens.dtype is I32 and seqlens.is_contiguous() and
            seqlens.shape == shape[:1] and seqlens.get_device() == index and page_table is not None and
            page_table.dtype is I32 and page_table.is_contiguous() and page_table.dim() == 2 and
            page_table.shape[0] == shape[0] and page_table.get_device() == index and
            (meta is None or _meta_fits(meta, index)) and kv_valid_len is None and out is None and lse is None and err_flag is None and out_dtype is None and
            (workspace is None or (workspace.get_device() == index and workspace.is_contiguous())) and
            (prefix_table is None or (prefix_table.dtype is I32 and prefix_table.dim() == 1 and
                                      prefix_table.is_contiguous() and prefix_table.get_device() == index and
                                      0 <= prefix_len <= prefix_table.shape[0] * cache.page_size))):
        _decode_checks(q, cache, prefix_table, prefix_len, page_table, seqlens, meta, kv_valid_len, out, out_dtype,
                       lse, workspace, err_flag)
    B, Hq, D = shape
    qs = q.stride(0) if B > 1 else Hq * D
    if page_table is not None:
        cols = page_table.shape[1]
        table, stride = page_table.data_ptr(), page_table.stride(0) if B > 1 else cols
    else:
        table = None
        stride = cols = 0
    if out is None:
        out = torch.empty(shape, dtype=out_dtype or BF16, device=cache.device)
    if lse is None:
        lse = torch.empty((B, Hq), dtype=F32, device=cache.device)
    if workspace is None:
        workspace = alloc_decode_workspace(cache, B, Hq, prefix_len=prefix_len)
    rest = (table, stride, cols, seqlens.data_ptr(), None if meta is None else ctypes.byref(meta.to_c()),
            None if kv_valid_len is None else kv_valid_len.data_ptr(),
            cache.scale if softmax_scale is None else softmax_scale, out.data_ptr(),
            OUT_BF16 if out.dtype is BF16 else OUT_F32, lse.data_ptr(), workspace.data_ptr(), workspace.nbytes,
            None if err_flag is None else err_flag.data_ptr(), _raw_stream(index))
    if prefix_table is None:
        _check(_lib.bsattn_decode(q.data_ptr(), qs, B, Hq, cache.ref, *rest), "bsattn_decode")
    else:
        _check(_lib.bsattn_decode_shared_prefix(q.data_ptr(), qs, B, Hq, cache.ref, prefix_table.data_ptr(),
                                                prefix_len, *rest), "bsattn_decode_shared_prefix")
    return out, lse


def decode(q, cache: KVCache, page_table, seqlens, *, meta=None, kv_valid_len=None, softmax_scale=None, out=None,
           out_dtype=None, lse=None, workspace=None, err_flag=None, stream=None):
    """Attention of one query token per sequence, q bf16 [B, Hq, D] (Hq a multiple of
    the cache's heads; tokens may be any multiple of 8 elements apart), over the
    seqlens[b] cached keys of each sequence.

    meta: lists of KV tiles to attend instead of all (a Meta with one query row per
    sequence and H = cache.H: batched with num_m = 1, or varlen with total_m_blocks =
    B); kv_valid_len int32 [B, meta.num_n] as for ``forward``.  Returns (out [B, Hq, D]
    bf16 or out_dtype, lse fp32 [B, Hq]); a sequence without keys gets 0 and -inf.
    workspace: see alloc_decode_workspace; None allocates one for this call."""
    if _calls is not None and workspace is not None and stream is None and out is None and lse is None and \
            out_dtype is None and err_flag is None and kv_valid_len is None:
        got = _calls.decode(cache.at, cache.index, q, page_table, seqlens,
                            cache.scale if softmax_scale is None else softmax_scale, workspace, meta, None, 0)
        if got is not None:
            if got.__class__ is tuple:
                return got
            raise BsattnError(got, "bsattn_decode")
    return _decode(q, cache, None, 0, page_table, seqlens, meta, kv_valid_len, softmax_scale, out, out_dtype, lse,
                   workspace, err_flag, stream)


def decode_shared_prefix(q, cache: KVCache, prefix_table, prefix_len: int, page_table, seqlens, *, meta=None,
                         kv_valid_len=None, softmax_scale=None, out=None, out_dtype=None, lse=None, workspace=None,
                         err_flag=None, stream=None):
    """``decode`` for a batch whose sequences all begin with one prefix of prefix_len
    cached tokens, in the pages prefix_table (int32 [pages]); page_table and seqlens
    (and meta, kv_valid_len) describe what each sequence has after it.  page_table may
    be None when no sequence has keys of its own.  The prefix is read from HBM once for all;
    a long one is also worked on once for all."""
    if prefix_table is None:
        raise ValueError("prefix_table is needed (decode attends sequences without a prefix)")
    if _calls is not None and workspace is not None and stream is None and out is None and lse is None and \
            out_dtype is None and err_flag is None and kv_valid_len is None:
        got = _calls.decode(cache.at, cache.index, q, page_table, seqlens,
                            cache.scale if softmax_scale is None else softmax_scale, workspace, meta, prefix_table, prefix_len)
        if got is not None:
            if got.__class__ is tuple:
                return got
            raise BsattnError(got, "bsattn_decode_shared_prefix")
    return _decode(q, cache, prefix_table, prefix_len, page_table, seqlens, meta, kv_valid_len, softmax_scale, out,
                   out_dtype, lse, workspace, err_flag, stream)
