"""Key/value cache in pages: bf16 rows in a pool shared by all sequences, block tables
and slot maps kept on the GPU, and attention of new tokens, a chunk of a prompt or one
at a time, over a sequence's pages (include/attn.h has the layouts and rules).

    cache = cca.paged_cache(pages, Hkv, page, D)
    tables = cca.paged_tables(B, max_pages, pages, page)       # every page free, every sequence empty
    ws = cca.paged_workspace(cache, q, B, tables)
    cu, slots = cca.paged_reserve(tables, add, T, ws=ws)       # add: new tokens of each sequence, -1: it ends
    cca.paged_store(cache, k, v, slots, ws=ws)                 # k, v: the step's rows, packed [T, Hkv, D]
    o, lse = cca.paged_attention(q, cache, tables.table, tables.lens, cu, ws=ws)

All integers are int32 tensors on the GPU, so that a step can be captured into a graph
and replayed. Torch provides memory and streams only.
"""
from __future__ import annotations

import ctypes
from typing import Optional

from . import _lib
from ._lib import ATTN_E_INVAL, AttnError


class _Calls:
    """What the calls on a handle's device ask for every time, looked up once: a decode step is
    bound by the host's time, of which these lookups are the larger part."""

    def __init__(self, device):
        import torch
        self.int32, self.bf16, self.fp32 = torch.int32, torch.bfloat16, torch.float32
        self.empty, self.empty_like, self.empty_strided = torch.empty, torch.empty_like, torch.empty_strided
        self.device = device
        self.gpu = (device.index or 0) if device.type == "cuda" else -2      # no tensor's get_device()
        self.raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        self.current = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)

    def stream(self, stream, t):
        """The given stream, or the current one of the device."""
        if stream is None and self.raw_stream is not None:
            return self.raw_stream(self.gpu)
        return _lib._stream_of(stream, t)

    def run(self, name: str, t, *args) -> None:
        """The library's entry point of that name, on the device (t's)."""
        fn = getattr(_lib._lib or _lib.lib(), name)
        if self.current() == self.gpu:
            st = fn(*args)
        else:
            with _lib._on(t):
                st = fn(*args)
        if st:
            raise AttnError(name, st)

    def ints(self, t, numel: int) -> bool:
        """A contiguous int32 tensor of numel elements on the device."""
        return t.dtype is self.int32 and t.get_device() == self.gpu and t.numel() == numel and t.is_contiguous()

    def table(self, t) -> bool:
        """An int32 matrix on the device whose rows are contiguous."""
        return (t.dtype is self.int32 and t.get_device() == self.gpu and t.dim() == 2
                and (t.stride(1) == 1 or t.shape[1] == 1))


class PagedCache:
    """A pool: k and v, bf16 [pages, Hkv, page, D] of the same strides, D contiguous. Other
    orders in memory are views: for [pages, page, Hkv, D] pass its transpose(1, 2)."""

    def __init__(self, k, v):
        import torch
        if not (k.dim() == 4 and k.dtype == torch.bfloat16 and v.dtype == torch.bfloat16 and k.shape == v.shape
                and k.device == v.device and (k.shape[3] == 1 or k.stride(3) == v.stride(3) == 1)
                and _lib._same_rows(k, v)):
            raise AttnError("PagedCache", ATTN_E_INVAL)
        self.k, self.v = k, v
        self.pages, self.Hkv, self.page, self.D = k.shape
        self.device = k.device
        # strides of dims of size 1 are free: what a contiguous tensor would have
        st = k.stride(2) if self.page > 1 else self.D
        sh = k.stride(1) if self.Hkv > 1 else self.page * st
        sp = k.stride(0) if self.pages > 1 else self.Hkv * sh
        self.desc = _lib.attn_paged_cache(self.pages, self.Hkv, self.page, self.D, sp, sh, st, k.data_ptr(), v.data_ptr())
        _lib.attn_paged_workspace_size(self.desc, None, 1, _lib.PAGED_STORE)       # the library's own checks
        self._ref = ctypes.byref(self.desc)
        self._calls = _Calls(self.device)
        self._shapes = {}

    def _shape(self, x, scale: Optional[float]):
        """A reference to the attn_shape of a packed tensor, kept by sizes, strides and scale: a
        decode loop asks for the same one at every step."""
        scale = None if scale is None else float(scale)      # a tensor's value, which may change, not the tensor
        key = (x.shape, x.stride(), scale)
        got = self._shapes.get(key)
        if got is None:
            if x.dim() != 3 or x.shape[-1] != self.D or x.stride(-1) != 1:
                raise AttnError("attn_shape", ATTN_E_INVAL)
            if len(self._shapes) >= 64:
                self._shapes.clear()
            got = self._shapes[key] = ctypes.byref(_lib.shape_of(x, scale, True))
        return got


class PagedTables:
    """Block tables int32 [B, max_pages] (rows contiguous), slots in use int32 [B], and the
    stack of free pages: int32 [pages], of which the first n_free (int32 [1]) are free."""

    def __init__(self, table, lens, free, n_free, page: int):
        fn = "PagedTables"
        self.ld = _lib._table_ld(fn, table)
        self.B, self.max_pages = table.shape
        self.table, self.lens, self.free, self.n_free, self.page = table, lens, free, n_free, int(page)
        self.device = table.device
        for t in (lens, free, n_free):
            if t.device != table.device:
                raise AttnError(fn, ATTN_E_INVAL)
        _lib._expect_flat(fn, "int32", self.B, lens)
        _lib._expect_flat(fn, "int32", free.numel(), free)
        _lib._expect_flat(fn, "int32", 1, n_free)
        if self.page < 16 or self.page > 1024 or self.page & (self.page - 1):
            raise AttnError(fn, ATTN_E_INVAL)
        self._calls = _Calls(self.device)


def paged_cache(pages: int, Hkv: int, page: int, D: int, device="cuda") -> PagedCache:
    """An empty pool; page: slots of a page, a power of two from 16 to 1024."""
    import torch
    return PagedCache(*(torch.zeros((pages, Hkv, page, D), dtype=torch.bfloat16, device=device) for _ in range(2)))


def paged_tables(B: int, max_pages: int, pages: int, page: int, device="cuda") -> PagedTables:
    """Tables of B empty sequences of up to max_pages pages each, every page of the pool free
    (page 0 is taken first)."""
    import torch
    i32 = dict(dtype=torch.int32, device=device)
    return PagedTables(torch.full((B, max_pages), -1, **i32), torch.zeros(B, **i32),
                       torch.arange(pages - 1, -1, -1, **i32), torch.full((1,), pages, **i32), page)


def paged_workspace(cache: Optional[PagedCache] = None, q=None, B: int = 1, tables: Optional[PagedTables] = None):
    """A workspace, status header zeroed: for storing in this cache, with q (packed [T, H, D])
    also for attention of queries of its shape of B sequences, and with tables for reserving.
    _lib.attn_status reads its errors."""
    import torch
    n = 256
    if cache is not None:
        n = max(n, _lib.attn_paged_workspace_size(cache.desc, None, 1, _lib.PAGED_STORE))
        if q is not None:
            n = max(n, _lib.attn_paged_workspace_size(cache.desc, _lib.shape_of(q, None, True), B, _lib.PAGED_ATTEND))
    if tables is not None:
        n = max(n, _lib.attn_paged_workspace_size(None, None, tables.B, _lib.PAGED_RESERVE))
    ws = torch.empty(n, dtype=torch.uint8, device=(cache if cache is not None else tables).device)
    ws[:256].zero_()
    return ws


def paged_reserve(tables: PagedTables, add, T: int, lens_out=None, n_free_out=None, cu_seqlens=None, slots=None, ws=None,
                  stream=None):
    """Slots for the next tokens: add int32 [B], new tokens of each sequence (negative: it ends
    and its pages become free). Extends the table in place, and the lengths and the number of
    free pages too, unless lens_out or n_free_out take them. A page that is in use has to be in one
    sequence's row only: the ends of two would put it on the stack twice (attn.h has what to do
    where sequences share pages). Returns (cu_seqlens, slots): int32
    [B + 1] offsets of the packed tokens and int32 [T] slots, -1 for padding and for sequences
    that found no pages (attn_status tells: ATTN_E_CAPACITY)."""
    fn = "paged_reserve"
    c, B, table = tables._calls, tables.B, tables.table
    if ws is None or cu_seqlens is None or slots is None:
        with _lib._alloc_on(stream, c.device):
            if ws is None:
                ws = paged_workspace(tables=tables)
            if cu_seqlens is None:
                cu_seqlens = c.empty(B + 1, dtype=c.int32, device=c.device)
            if slots is None:
                slots = c.empty(T, dtype=c.int32, device=c.device)
    lens_out = tables.lens if lens_out is None else lens_out
    n_free_out = tables.n_free if n_free_out is None else n_free_out
    if not (c.ints(add, B) and c.ints(lens_out, B) and c.ints(n_free_out, 1) and c.ints(cu_seqlens, B + 1)
            and c.ints(slots, T) and ws.get_device() == c.gpu):
        raise AttnError(fn, ATTN_E_INVAL)
    c.run("attn_paged_reserve", table, add.data_ptr(), tables.lens.data_ptr(), B, tables.page, tables.free.numel(),
          tables.n_free.data_ptr(), tables.free.data_ptr(), table.data_ptr(), tables.ld, tables.max_pages,
          lens_out.data_ptr(), n_free_out.data_ptr(), cu_seqlens.data_ptr(), slots.data_ptr(), T, ws.data_ptr(),
          ws.nbytes, c.stream(stream, table))
    return cu_seqlens, slots


def paged_store(cache: PagedCache, k, v, slots, ws=None, stream=None) -> None:
    """Store the rows of k and v, bf16 packed [T, Hkv, D], in the slots (int32 [T]) that
    paged_reserve named; rows with slot -1 are skipped. k and v may be views of the pool, of a
    page that is copied, as long as no slot is both read and written."""
    fn = "paged_store"
    c = cache._calls
    if ws is None:
        with _lib._alloc_on(stream, c.device):
            ws = paged_workspace(cache)
    ref = cache._shape(k, 1.0)
    if not (c.ints(slots, k.shape[0]) and k.dtype is c.bf16 and v.dtype is c.bf16 and k.get_device() == c.gpu
            and v.get_device() == c.gpu and ws.get_device() == c.gpu and k.shape == v.shape
            and (k.stride() == v.stride() or _lib._same_rows(k, v))):
        raise AttnError(fn, ATTN_E_INVAL)
    c.run("attn_paged_store", k, k.data_ptr(), v.data_ptr(), ref, cache._ref, slots.data_ptr(), ws.data_ptr(), ws.nbytes,
          c.stream(stream, k))


def paged_attention(q, cache: PagedCache, table, lens, cu_seqlens=None, scale: Optional[float] = None, o=None, lse=None,
                    ws=None, stream=None):
    """(o, lse) of the newest tokens of each sequence, q bf16 packed [T, H, D], over its lens[b]
    slots (their own included): token i of n_q sees the slots up to lens[b] - n_q + i. Without
    cu_seqlens (int32 [B + 1]) every sequence has T / B tokens. lse: fp32 [1, H, T]. o and lse
    may be given (o with q's strides); rows of padding stay as they were. o has q's strides,
    gaps included: for a slice of a wide tensor pass a contiguous copy."""
    fn = "paged_attention"
    c = cache._calls
    ref = cache._shape(q, scale)
    T, H, _ = q.shape
    if not c.table(table):
        raise AttnError(fn, ATTN_E_INVAL)
    B, most = table.shape
    if not (q.dtype is c.bf16 and q.get_device() == c.gpu and c.ints(lens, B)
            and (cu_seqlens is None or c.ints(cu_seqlens, B + 1))
            and (o is None or o.dtype is c.bf16 and o.get_device() == c.gpu and o.shape == q.shape
                 and (o.stride() == q.stride() or _lib._same_rows(o, q)))
            and (lse is None or lse.dtype is c.fp32 and lse.get_device() == c.gpu and lse.numel() == H * T
                 and lse.is_contiguous())
            and (ws is None or ws.get_device() == c.gpu)):
        raise AttnError(fn, ATTN_E_INVAL)
    with _lib._alloc_on(stream, c.device):
        if ws is None:
            ws = paged_workspace(cache, q, B)
        if o is None:
            o = c.empty_like(q) if q.is_contiguous() else \
                c.empty_strided(q.shape, q.stride(), dtype=c.bf16, device=c.device)
        if lse is None:
            lse = c.empty((1, H, T), dtype=c.fp32, device=c.device)
    c.run("attn_paged_attend", q, q.data_ptr(), ref, cache._ref, table.data_ptr(), table.stride(0) if B > 1 else most, most,
          lens.data_ptr(), None if cu_seqlens is None else cu_seqlens.data_ptr(), B, o.data_ptr(), lse.data_ptr(),
          ws.data_ptr(), ws.nbytes, c.stream(stream, q))
    return o, lse
