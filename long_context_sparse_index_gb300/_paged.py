"""Serving a DSA layer from a paged cache (argument marshalling only).

``PagedCache`` holds one layer's pages, ``PagedBatch`` the sequences of a call
and ``PageTable`` the page bookkeeping; each checks its tensors once and keeps
them, so that the calls themselves stay short.  As in ``_binding``, all
arithmetic runs in libdsa's CUDA kernels on the current CUDA stream (or the
one given), and outputs and workspaces that the caller does not pass are
allocated with torch, on the stream that the call runs on.
"""
from __future__ import annotations

import ctypes

import torch

from ._binding import _check, _need, _out, _shape, load

_vp, _i64, _i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int


class _CacheStruct(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("k_idx", _vp), ("khat", _vp), ("k_stride", _i64), ("v_stride", _i64),
                ("k_idx_stride", _i64), ("khat_stride", _i64), ("num_pages", _i64), ("page_size", _i32), ("D", _i32),
                ("Di", _i32)]


class _BatchStruct(ctypes.Structure):
    _fields_ = [("block_table", _vp), ("table_stride", _i64), ("seq_lens", _vp), ("cu_q", _vp), ("rows", _i64),
                ("max_pages", _i32), ("batch", _i32)]


class _TableStruct(ctypes.Structure):
    _fields_ = [("block_table", _vp), ("table_stride", _i64), ("seq_lens", _vp), ("page_count", _vp),
                ("num_pages", _i64), ("max_pages", _i32), ("max_seqs", _i32), ("page_size", _i32)]


_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch.cuda.current_device


def _full(t, name: str, dtype, ndim: int, device: int):
    """_need for a call whose current device is known: the checks that pass
    cost a decoding step less than a microsecond, one that fails is repeated
    there for its message."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.dim() == ndim and t.get_device() == device
            and t.is_contiguous()):
        _need(t, name, dtype, ndim)


def _on_device(t, name: str, dtype, ndim: int):
    """_need without contiguity: a CUDA tensor on the current device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor (got {t.device})")
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, but the kernels run on the current device "
                         f"cuda:{torch.cuda.current_device()}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions (got shape {tuple(t.shape)})")


def _rows_strided(t, name: str, dtype, row: int, device: int) -> int:
    """[rows, row] whose rows are contiguous; returns the distance between rows, which is free."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.dim() == 2 and t.get_device() == device):
        _on_device(t, name, dtype, 2)
    n, d = t.shape
    apart, step = t.stride()
    if d != row or (n > 0 and step != 1):
        raise ValueError(f"{name} must have contiguous rows of {row} elements (got shape {tuple(t.shape)}, "
                         f"strides {t.stride()})")
    return apart if n > 1 else row


def _table(t, name: str):
    _on_device(t, name, torch.int32, 2)
    if t.numel() == 0 or t.stride(1) != 1 or (t.shape[0] > 1 and t.stride(0) < t.shape[1]):
        raise ValueError(f"{name} must be int32 with contiguous rows (got shape {tuple(t.shape)}, "
                         f"strides {t.stride()})")


def _device_of(*owners) -> int:
    """The current device, which every handle must be on."""
    now = _current_device()
    for x in owners:
        if x.device_index != now:
            raise ValueError(f"the {type(x).__name__} is on cuda:{x.device_index}, but the kernels run on the current "
                             f"device cuda:{now}")
    return now


class PagedCache:
    """One layer's cache in pages of ``page_size`` tokens (a power of two, 16..1024).

    k, v [pages, page_size, 128], k_idx [pages, page_size, 64] and khat
    [pages, page_size / 4, 128] (pooled indexer keys: hi in columns 0..63, lo
    in 64..127), all bf16.  Within a page everything is contiguous; the
    distance between pages is free (a multiple of 8 elements)."""

    def __init__(self, k, v, k_idx, khat):
        for t, n, d in ((k, "k", 128), (v, "v", 128), (k_idx, "k_idx", 64), (khat, "khat", 128)):
            _on_device(t, n, torch.bfloat16, 3)
            if t.shape[2] != d or t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != d):
                raise ValueError(f"{n} must be [pages, tokens, {d}] with contiguous pages (got shape "
                                 f"{tuple(t.shape)}, strides {t.stride()})")
        pages, page_size = k.shape[0], k.shape[1]
        _shape(v, "v", (pages, page_size, 128))
        _shape(k_idx, "k_idx", (pages, page_size, 64))
        _shape(khat, "khat", (pages, page_size // 4, 128))
        self.k, self.v, self.k_idx, self.khat = k, v, k_idx, khat
        self.num_pages, self.page_size = pages, page_size
        self.device = k.device
        self.device_index = k.device.index

        def stride(t):
            return t.stride(0) if pages > 1 else t.shape[1] * t.shape[2]

        self._struct = _CacheStruct(k.data_ptr(), v.data_ptr(), k_idx.data_ptr(), khat.data_ptr(), stride(k),
                                    stride(v), stride(k_idx), stride(khat), pages, page_size, 128, 64)
        self._ref = ctypes.byref(self._struct)

    @classmethod
    def empty(cls, num_pages: int, page_size: int, device="cuda"):
        """A cache of uninitialised pages."""
        def new(tokens, d):
            return torch.empty(num_pages, tokens, d, dtype=torch.bfloat16, device=device)
        return cls(new(page_size, 128), new(page_size, 128), new(page_size, 64), new(page_size // 4, 128))


class PagedBatch:
    """The sequences of a call and their new tokens, as int32 device tensors:
    block_table [batch, max_pages], seq_lens [batch] (new tokens included) and
    cu_q [batch + 1] (rows cu_q[s] .. cu_q[s+1]-1 of the call's tensors are
    sequence s's new tokens).  The contents are read when the kernels run."""

    def __init__(self, block_table, seq_lens, cu_q):
        _table(block_table, "block_table")
        _need(seq_lens, "seq_lens", torch.int32, 1)
        _need(cu_q, "cu_q", torch.int32, 1)
        self.batch, self.max_pages = cu_q.shape[0] - 1, block_table.shape[1]
        if self.batch < 1 or block_table.shape[0] < self.batch or seq_lens.shape[0] < self.batch:
            raise ValueError("cu_q must have batch + 1 entries, block_table and seq_lens at least batch rows")
        self.block_table, self.seq_lens, self.cu_q = block_table, seq_lens, cu_q
        self.device_index = block_table.device.index
        self._fields = (block_table.data_ptr(), block_table.stride(0) if block_table.shape[0] > 1 else self.max_pages,
                        seq_lens.data_ptr(), cu_q.data_ptr())
        self._last = (-1, None)
        self._index_ws = (None, 0)

    def _index_workspace(self, rows: int, page_size: int) -> int:
        last = self._index_ws
        if last[0] != (rows, page_size):
            last = self._index_ws = ((rows, page_size),
                                     load().dsa_paged_index_topk_workspace(rows, self.max_pages, page_size))
        return last[1]

    def _with_rows(self, rows: int):
        # the struct of the last number of rows is kept; it is never written
        # again, so threads may share a batch
        last = self._last
        if last[0] != rows:
            last = self._last = (rows, ctypes.byref(_BatchStruct(*self._fields, rows, self.max_pages, self.batch)))
        return last[1]


class PageTable:
    """The page bookkeeping of a cache, as int32 device tensors that the page
    operators write: block_table [max_seqs, max_pages], seq_lens [max_seqs] (0:
    the row is free) and page_count [num_pages] (sequences holding the page, 0:
    free)."""

    def __init__(self, block_table, seq_lens, page_count):
        _table(block_table, "block_table")
        _need(seq_lens, "seq_lens", torch.int32, 1)
        _need(page_count, "page_count", torch.int32, 1)
        self.max_seqs, self.max_pages = block_table.shape
        _shape(seq_lens, "seq_lens", (self.max_seqs,))
        if page_count.shape[0] < 1:
            raise ValueError("page_count must have an entry per page")
        self.block_table, self.seq_lens, self.page_count = block_table, seq_lens, page_count
        self.num_pages = page_count.shape[0]
        self.device, self.device_index = block_table.device, block_table.device.index
        self._fields = (block_table.data_ptr(), block_table.stride(0) if self.max_seqs > 1 else self.max_pages,
                        seq_lens.data_ptr(), page_count.data_ptr(), self.num_pages, self.max_pages, self.max_seqs)
        self._last = (-1, None)

    @classmethod
    def empty(cls, cache: PagedCache, max_seqs: int, max_pages: int):
        """The table of a cache in which every page is free."""
        dev = cache.device
        return cls(torch.full((max_seqs, max_pages), -1, dtype=torch.int32, device=dev),
                   torch.zeros(max_seqs, dtype=torch.int32, device=dev),
                   torch.zeros(cache.num_pages, dtype=torch.int32, device=dev))

    def _with_page(self, page_size: int):
        last = self._last
        if last[0] != page_size:
            last = self._last = (page_size, ctypes.byref(_TableStruct(*self._fields, page_size)))
        return last[1]


def _configure_paged(lib):
    f32, sz, i64, i32, vp = ctypes.c_float, ctypes.c_size_t, _i64, _i32, _vp
    lib.dsa_cache_append.argtypes = [vp, vp, vp, i64, vp, i64, vp, i64, vp]
    lib.dsa_cache_append_reserved.argtypes = [vp, vp, vp, i64, vp, i64, vp, i64, vp, vp]
    lib.dsa_cache_copy_pages.argtypes = [vp, i32, vp, vp, i64, vp]
    lib.dsa_cache_workspace.argtypes = [i64, i32, i64]
    lib.dsa_cache_workspace.restype = sz
    lib.dsa_cache_reserve.argtypes = [vp, vp, vp, vp, sz, vp]
    lib.dsa_cache_fork.argtypes = [vp, i32, vp, vp, vp, i64, vp, vp, sz, vp]
    lib.dsa_cache_free.argtypes = [vp, vp, i64, vp]
    lib.dsa_cache_compact.argtypes = [vp, i32, vp, vp, vp, sz, vp]
    lib.dsa_paged_index_topk_workspace.argtypes = [i64, i32, i32]
    lib.dsa_paged_index_topk_workspace.restype = sz
    lib.dsa_paged_index_topk.argtypes = [vp, vp, vp, vp, i32, i32, i32, vp, vp, sz, vp]
    lib.dsa_paged_sparse_attn_fwd.argtypes = [vp, vp, vp, vp, i32, i32, i32, f32, vp, vp, vp]
    for f in (lib.dsa_cache_append, lib.dsa_cache_append_reserved, lib.dsa_cache_copy_pages, lib.dsa_cache_reserve,
              lib.dsa_cache_fork, lib.dsa_cache_free, lib.dsa_cache_compact, lib.dsa_paged_index_topk,
              lib.dsa_paged_sparse_attn_fwd):
        f.restype = ctypes.c_int


def _handle(stream, device: int) -> int:
    return _raw_stream(device) if stream is None else stream.cuda_stream


def _new(shape, dtype, device, stream):
    """An allocation that belongs to the call's stream.  (`device` is a
    torch.device: an ordinal costs torch.empty three microseconds more.)"""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _result(given, name, shape, dtype, device, stream):
    return _new(shape, dtype, device, stream) if given is None else _out(given, name, shape, dtype, device)


def _scratch(nbytes: int, given, device, stream):
    if given is None:
        return _new(max(nbytes, 256), torch.uint8, device, stream)
    _need(given, "workspace", given.dtype, given.dim())
    return given


def _ids(t, name: str, device: int) -> int:
    _full(t, name, torch.int32, 1, device)
    return t.shape[0]


def dsa_cache_append(cache: PagedCache, batch: PagedBatch, k, v, k_idx, stream=None, reserved=None):
    """Writes the new tokens' k, v [rows, 128] and k_idx [rows, 64] (bf16, rows
    any multiple of 8 elements apart) into their pages, and the pooled key of
    every pool that they complete.

    reserved: the word that dsa_cache_reserve returned for these tokens.  When
    it is negative the sequences have their old lengths and the rows would
    overwrite their last tokens; given it, the append then writes nothing and
    dsa_sync_status reports DSA_ERR_INTERNAL.  Without it, look at the word
    before appending."""
    dev = _device_of(cache, batch)
    ks = _rows_strided(k, "k", torch.bfloat16, 128, dev)
    vs = _rows_strided(v, "v", torch.bfloat16, 128, dev)
    kis = _rows_strided(k_idx, "k_idx", torch.bfloat16, 64, dev)
    rows = k.shape[0]
    if v.shape[0] != rows or k_idx.shape[0] != rows:
        raise ValueError(f"k, v and k_idx must have the same rows (got {rows}, {v.shape[0]} and {k_idx.shape[0]})")
    args = (cache._ref, batch._with_rows(rows), k.data_ptr(), ks, v.data_ptr(), vs, k_idx.data_ptr(), kis)
    if reserved is None:
        _check(load().dsa_cache_append(*args, _handle(stream, dev)))
        return
    _full(reserved, "reserved", torch.int32, 1, dev)
    _shape(reserved, "reserved", (1,))
    _check(load().dsa_cache_append_reserved(*args, reserved.data_ptr(), _handle(stream, dev)))


def _layers(cache):
    """(first cache, struct array, count) of one cache or of a sequence of the layers' caches."""
    if isinstance(cache, PagedCache):
        return cache, cache._ref, 1
    caches = list(cache)
    if not caches or not all(isinstance(c, PagedCache) for c in caches):
        raise TypeError("cache must be a PagedCache or a sequence of the layers' PagedCaches")
    first = caches[0]
    for c in caches:
        if c.device_index != first.device_index:
            raise ValueError("the layers' caches must be on one device")
    return first, (_CacheStruct * len(caches))(*[c._struct for c in caches]), len(caches)


def dsa_cache_copy_pages(cache, src, dst, stream=None):
    """Copies page src[j] onto page dst[j] (int32 tensors), all four buffers,
    of a cache or of every layer's (a sequence of caches)."""
    first, ref, layers = _layers(cache)
    dev = _device_of(first)
    n = _ids(src, "src", dev)
    _ids(dst, "dst", dev)
    _shape(dst, "dst", (n,))
    _check(load().dsa_cache_copy_pages(ref, layers, src.data_ptr(), dst.data_ptr(), n, _handle(stream, dev)))


def cache_workspace_size(num_pages: int, max_seqs: int, n: int = 0) -> int:
    """Bytes of workspace of the page operators (n: children of a fork)."""
    return int(load().dsa_cache_workspace(num_pages, max_seqs, n))


def _of_cache(cache, pages: PageTable) -> int:
    dev = _device_of(cache, pages)
    if pages.num_pages != cache.num_pages:
        raise ValueError(f"the page table counts {pages.num_pages} pages, the cache has {cache.num_pages}")
    return dev


def dsa_cache_reserve(cache, pages: PageTable, add, result=None, workspace=None, stream=None):
    """Changes the length of every sequence s by add[s] tokens (int32
    [max_seqs]): longer ones take the lowest free pages, shorter ones give
    theirs back; returns a device word: pages taken, or minus the number
    lacking (then nothing changed).  cache: the one, or the layers'."""
    cache = _layers(cache)[0]
    dev, lib = _of_cache(cache, pages), load()
    _ids(add, "add", dev)
    _shape(add, "add", (pages.max_seqs,))
    result = _result(result, "result", (1,), torch.int32, cache.device, stream)
    ws = _scratch(lib.dsa_cache_workspace(pages.num_pages, pages.max_seqs, 0), workspace, cache.device, stream)
    _check(lib.dsa_cache_reserve(pages._with_page(cache.page_size), add.data_ptr(), result.data_ptr(), ws.data_ptr(),
                                 ws.numel() * ws.element_size(), _handle(stream, dev)))
    return result


def dsa_cache_fork(cache, pages: PageTable, src, dst, result=None, workspace=None, stream=None):
    """Row dst[j] becomes a copy of sequence src[j] (int32 tensors): full pages
    shared, a partly filled last page copied, in a cache or in every layer's (a
    sequence of caches); returns a device word: pages taken, or minus the
    number lacking (then nothing changed)."""
    cache, ref, layers = _layers(cache)
    dev, lib = _of_cache(cache, pages), load()
    n = _ids(src, "src", dev)
    _ids(dst, "dst", dev)
    _shape(dst, "dst", (n,))
    result = _result(result, "result", (1,), torch.int32, cache.device, stream)
    ws = _scratch(lib.dsa_cache_workspace(pages.num_pages, pages.max_seqs, n), workspace, cache.device, stream)
    _check(lib.dsa_cache_fork(ref, layers, pages._with_page(cache.page_size), src.data_ptr(), dst.data_ptr(), n,
                              result.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size(), _handle(stream, dev)))
    return result


def dsa_cache_free(cache, pages: PageTable, seqs, stream=None):
    """Frees the sequences named in seqs (int32 tensor).  cache: the one, or
    the layers'."""
    cache = _layers(cache)[0]
    dev = _of_cache(cache, pages)
    n = _ids(seqs, "seqs", dev)
    _check(load().dsa_cache_free(pages._with_page(cache.page_size), seqs.data_ptr(), n, _handle(stream, dev)))


def dsa_cache_compact(cache, pages: PageTable, result=None, workspace=None, stream=None):
    """Moves the used pages down over the free ones, in a cache or in every
    layer's (a sequence of caches); returns device words [pages in use, pages
    moved]."""
    cache, ref, layers = _layers(cache)
    dev, lib = _of_cache(cache, pages), load()
    result = _result(result, "result", (2,), torch.int32, cache.device, stream)
    ws = _scratch(lib.dsa_cache_workspace(pages.num_pages, pages.max_seqs, 0), workspace, cache.device, stream)
    _check(lib.dsa_cache_compact(ref, layers, pages._with_page(cache.page_size), result.data_ptr(), ws.data_ptr(),
                                 ws.numel() * ws.element_size(), _handle(stream, dev)))
    return result


def paged_index_topk_workspace_size(rows: int, max_pages: int, page_size: int) -> int:
    return int(load().dsa_paged_index_topk_workspace(rows, max_pages, page_size))


def dsa_paged_index_topk(cache: PagedCache, batch: PagedBatch, q_idx, w, topk: int, pool_idx=None, workspace=None,
                         stream=None):
    """pool_idx [rows, topk] int32 of the new tokens' selected pools (ascending,
    -1 padded), for q_idx [rows, Hi, 64] bf16 and w [rows, Hi] fp32."""
    dev, lib = _device_of(cache, batch), load()
    _full(q_idx, "q_idx", torch.bfloat16, 3, dev)
    _full(w, "w", torch.float32, 2, dev)
    rows, Hi, Di = q_idx.shape
    if w.shape[0] != rows or w.shape[1] != Hi:
        _shape(w, "w", (rows, Hi))
    pool_idx = _result(pool_idx, "pool_idx", (rows, max(topk, 0)), torch.int32, cache.device, stream)
    ws = _scratch(batch._index_workspace(rows, cache.page_size), workspace, cache.device, stream)
    _check(lib.dsa_paged_index_topk(cache._ref, batch._with_rows(rows), q_idx.data_ptr(), w.data_ptr(), Hi, Di, topk,
                                    pool_idx.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size(),
                                    _handle(stream, dev)))
    return pool_idx


def dsa_paged_sparse_attn_fwd(cache: PagedCache, batch: PagedBatch, q, pool_idx, scale: float = 0.0, o=None, lse=None,
                              stream=None):
    """(o [rows, 16, 128] bf16, lse [rows, 16] fp32) of the new tokens' attention
    over their selected pools and their own partial pool."""
    dev = _device_of(cache, batch)
    _full(q, "q", torch.bfloat16, 3, dev)
    _full(pool_idx, "pool_idx", torch.int32, 2, dev)
    rows, Hq, D = q.shape
    sel_rows, topk = pool_idx.shape
    if sel_rows != rows:
        raise ValueError(f"pool_idx must have {rows} rows (got {sel_rows})")
    o = _result(o, "o", (rows, Hq, D), torch.bfloat16, cache.device, stream)
    lse = _result(lse, "lse", (rows, Hq), torch.float32, cache.device, stream)
    _check(load().dsa_paged_sparse_attn_fwd(cache._ref, batch._with_rows(rows), q.data_ptr(), pool_idx.data_ptr(), Hq,
                                            D, topk, scale, o.data_ptr(), lse.data_ptr(), _handle(stream, dev)))
    return o, lse
