"""Key/value cache held in 4 bits: what a program does with the resident K and V
once a prompt's chunks have run. Rows are stored as e2m1 codes with one e4m3
scale for 16 dims (include/attn.h has the format), new tokens attend to them,
and a cache is cut to a budget by the attention weight that its slots received.

    cache = cca.kv4_cache(B, Hkv, cap, D)
    cca.kv4_store(cache, k, v, pos)                      # a prompt's rows, or one row a sequence
    o, lse = cca.kv4_attention(q, cache, lens, mass_in=mass, mass_out=mass)
    lens2, slots = cca.kv4_evict(cache, lens, mass, keep, recent, smaller, mass2.zero_())

pos and lens are int32 tensors on the GPU, so the calls can be captured into a
graph and replayed. Torch provides memory and streams only.
"""
from __future__ import annotations

import ctypes
from typing import Optional

from . import _lib
from ._lib import ATTN_E_INVAL, AttnError


class KV4Cache:
    """A 4-bit cache in four uint8 tensors: codes [B, Hkv, cap, D / 2] and scales
    [B, Hkv, cap, ceil(D / 16)] of the keys and of the values, possibly views of
    larger ones (some sequences, heads or slots) as long as rows are contiguous.
    k_scale and v_scale are powers of two that every value is multiplied by;
    choose them so that the largest magnitude is below 2688 times the scale."""

    def __init__(self, k_codes, k_scales, v_codes, v_scales, D: int, k_scale: float = 1.0, v_scale: float = 1.0):
        import torch
        arrays = (k_codes, k_scales, v_codes, v_scales)
        if k_codes.dim() != 4 or D < 8 or D % 8:
            raise AttnError("KV4Cache", ATTN_E_INVAL)
        B, Hkv, cap, _ = k_codes.shape
        strides = set()
        for t, n in zip(arrays, (D // 2, -(-D // 16)) * 2):
            if (t.dtype != torch.uint8 or tuple(t.shape) != (B, Hkv, cap, n) or t.device != k_codes.device
                    or (n > 1 and t.stride(3) != 1) or (cap > 1 and t.stride(2) != n)):
                raise AttnError("KV4Cache", ATTN_E_INVAL)
            sh = t.stride(1) if Hkv > 1 else cap * n
            sb = t.stride(0) if B > 1 else Hkv * sh
            if sh % n or sb % n:
                raise AttnError("KV4Cache", ATTN_E_INVAL)
            strides.add((sb // n, sh // n))
        if len(strides) != 1:
            raise AttnError("KV4Cache", ATTN_E_INVAL)
        (sb, sh), = strides
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = arrays
        self.B, self.Hkv, self.cap, self.D = B, Hkv, cap, D
        self.k_scale, self.v_scale = float(k_scale), float(v_scale)
        self.device = k_codes.device
        self.desc = _lib.attn_kv4_cache(B, Hkv, cap, D, sb, sh, *(t.data_ptr() for t in arrays), self.k_scale,
                                        self.v_scale)
        _lib.attn_kv4_workspace_size(self.desc, None, _lib.KV4_ROWS)      # the library's own checks
        self._ref = ctypes.byref(self.desc)
        self._shapes = {}

    def _shape(self, x, scale: Optional[float], packed: bool):
        """The attn_shape of a tensor and a reference to it, kept by sizes, strides and scale: a
        decode loop asks for the same one at every step."""
        key = (x.shape, x.stride(), scale, packed)
        got = self._shapes.get(key)
        if got is None:
            if x.dim() != (3 if packed else 4) or x.shape[-1] != self.D or x.stride(-1) != 1:
                raise AttnError("attn_shape", ATTN_E_INVAL)
            shape = _lib.shape_of(x, scale, packed)
            if len(self._shapes) >= 64:
                self._shapes.clear()
            got = self._shapes[key] = (shape, ctypes.byref(shape))
        return got

    def _check(self, fn: str, ints, numel: int, *others) -> None:
        """An int32 tensor of numel elements, and others, on the cache's device (a GPU)."""
        import torch
        dev = self.device
        ok = (dev.type == "cuda" and ints.dtype is torch.int32 and ints.device == dev and ints.numel() == numel
              and ints.is_contiguous())
        for t in others:
            ok = ok and (t is None or t.device == dev)
        if not ok:
            raise AttnError(fn, ATTN_E_INVAL)


def kv4_cache(B: int, Hkv: int, cap: int, D: int, device="cuda", k_scale: float = 1.0, v_scale: float = 1.0) -> KV4Cache:
    """An empty cache of cap slots (a multiple of 16)."""
    import torch
    codes = [torch.zeros((B, Hkv, cap, n), dtype=torch.uint8, device=device) for n in (D // 2, -(-D // 16)) * 2]
    return KV4Cache(*codes, D=D, k_scale=k_scale, v_scale=v_scale)


def kv4_workspace(cache: KV4Cache, q=None, mass: bool = False):
    """A workspace for the calls on this cache, status header zeroed: for storing,
    loading and evicting, and with q also for attention of queries of its shape
    (with mass: accumulating weights). _lib.attn_status reads its errors."""
    import torch
    n = _lib.attn_kv4_workspace_size(cache.desc, None, _lib.KV4_ROWS) if q is None else \
        _lib.attn_kv4_workspace_size(cache.desc, _lib.shape_of(q), _lib.KV4_ATTEND_MASS if mass else _lib.KV4_ATTEND)
    ws = torch.empty(n, dtype=torch.uint8, device=cache.device)
    ws[:256].zero_()
    return ws


def kv4_store(cache: KV4Cache, k, v, pos, cu_seqlens=None, ws=None, stream=None) -> None:
    """Store rows: k, v bf16 [B, Hkv, T, D], row t of sequence b in slot pos[b] + t;
    with cu_seqlens (int32 [B + 1]) packed [T, Hkv, D], each sequence's tokens from pos[b] on."""
    if ws is None:
        with _lib._alloc_on(stream, cache.device):
            ws = kv4_workspace(cache)
    _, ref = cache._shape(k, 1.0, cu_seqlens is not None)
    _rows_checks("kv4_store", cache, k, v, pos, cu_seqlens, ws)
    with _lib._on(k):
        _lib._check("attn_kv4_store", _lib.lib().attn_kv4_store(
            k.data_ptr(), v.data_ptr(), ref, cache._ref, pos.data_ptr(), _lib._ptr(cu_seqlens), ws.data_ptr(),
            ws.numel() * ws.element_size(), _lib._stream_of(stream, k)))


def _rows_checks(fn: str, cache: KV4Cache, k, v, pos, cu_seqlens, ws) -> None:
    import torch
    cache._check(fn, pos, cache.B, k, v, ws)
    if cu_seqlens is not None:
        cache._check(fn, cu_seqlens, cache.B + 1)
    if not (k.dtype is torch.bfloat16 and v.dtype is torch.bfloat16 and k.shape == v.shape
            and (k.stride() == v.stride() or _lib._same_rows(k, v))):
        raise AttnError(fn, ATTN_E_INVAL)


def kv4_load(cache: KV4Cache, pos, T: int, cu_seqlens=None, k=None, v=None, ws=None, stream=None):
    """The values of T rows from slot pos[b] on, bf16 [B, Hkv, T, D]; with cu_seqlens
    packed [T, Hkv, D]. k and v may be given (rows outside the cache stay as they were), views
    of wider tensors too; one that is not given has the other's strides."""
    import torch
    shape = (T, cache.Hkv, cache.D) if cu_seqlens is not None else (cache.B, cache.Hkv, T, cache.D)
    with _lib._alloc_on(stream, cache.device):
        given = v if k is None else k
        if given is None:
            k, v = (torch.empty(shape, dtype=torch.bfloat16, device=cache.device) for _ in range(2))
        elif k is None or v is None:
            # one shape describes both, so the other has the strides of the one that is given
            other = torch.empty_strided(given.shape, given.stride(), dtype=torch.bfloat16, device=cache.device)
            k, v = (other, v) if k is None else (k, other)
        if ws is None:
            ws = kv4_workspace(cache)
    _, ref = cache._shape(k, 1.0, cu_seqlens is not None)
    _rows_checks("kv4_load", cache, k, v, pos, cu_seqlens, ws)
    if k.shape != shape:
        raise AttnError("kv4_load", ATTN_E_INVAL)
    with _lib._on(k):
        _lib._check("attn_kv4_load", _lib.lib().attn_kv4_load(
            cache._ref, pos.data_ptr(), _lib._ptr(cu_seqlens), ref, k.data_ptr(), v.data_ptr(), ws.data_ptr(),
            ws.numel() * ws.element_size(), _lib._stream_of(stream, k)))
    return k, v


def kv4_attention(q, cache: KV4Cache, lens, scale: Optional[float] = None, mass_in=None, mass_out=None, ws=None,
                  stream=None):
    """(o, lse) of the newest T tokens of each sequence, q bf16 [B, H, T, D], over the
    lens[b] slots in use (their own included). mass_out fp32 [B, Hkv, n]: each slot's
    weight over the call's rows is added to mass_in (None: zeros; may be mass_out). The
    entry of a slot that was appended since has to be 0 in mass_in. o has q's strides, gaps
    included: for a few rows of a long tensor pass a contiguous copy."""
    import torch
    shape, ref = cache._shape(q, scale, False)
    if ws is None:
        with _lib._alloc_on(stream, cache.device):
            ws = kv4_workspace(cache, q, mass_out is not None)
    cache._check("kv4_attention", lens, cache.B, q, ws, mass_in, mass_out)
    if q.dtype is not torch.bfloat16:
        raise AttnError("kv4_attention", ATTN_E_INVAL)
    ld = 0
    if mass_in is not None or mass_out is not None:
        ld = _lib._mass_ld("kv4_attention", cache.desc, mass_in, mass_out)
    with _lib._alloc_on(stream, q.device):
        o = torch.empty_like(q) if q.is_contiguous() else \
            torch.empty_strided(q.shape, q.stride(), dtype=q.dtype, device=q.device)
        lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
    with _lib._on(q):
        _lib._check("attn_kv4_attend", _lib.lib().attn_kv4_attend(
            q.data_ptr(), ref, cache._ref, lens.data_ptr(), o.data_ptr(), lse.data_ptr(), _lib._ptr(mass_in),
            _lib._ptr(mass_out), ld, ws.data_ptr(), ws.numel() * ws.element_size(), _lib._stream_of(stream, q)))
    return o, lse


def kv4_evict(cache: KV4Cache, lens, mass, keep: int, recent: int, out: KV4Cache, mass_out=None, lens_out=None,
              ws=None, stream=None):
    """Cut each sequence to at most keep slots, per key/value head: its last `recent`
    and those with the highest mass, moved to the front of `out` in their order, their
    masses to the front of mass_out. What lies behind them stays as it was: zero a
    mass_out that was in use before, or the slots appended later start from its weights.
    Returns (lens_out, slots): int32 [B] and the source slots int32 [B, Hkv, keep]."""
    import torch
    fn = "kv4_evict"
    if out.device != cache.device or not 0 < keep <= out.cap or recent < 0:
        raise AttnError(fn, ATTN_E_INVAL)
    if ws is None:
        with _lib._alloc_on(stream, cache.device):
            ws = kv4_workspace(cache)
    cache._check(fn, lens, cache.B, mass, mass_out, lens_out, ws)
    if lens_out is not None:
        cache._check(fn, lens_out, cache.B)
    with _lib._alloc_on(stream, lens.device):
        slots = torch.empty((cache.B, cache.Hkv, int(keep)), dtype=torch.int32, device=lens.device)
        if lens_out is None:
            lens_out = torch.empty_like(lens)
    ld = _lib._mass_ld(fn, cache.desc, mass)
    ld_out = 0 if mass_out is None else _lib._mass_ld(fn, cache.desc, mass_out)
    with _lib._on(lens):
        _lib._check("attn_kv4_evict", _lib.lib().attn_kv4_evict(
            cache._ref, lens.data_ptr(), mass.data_ptr(), ld, keep, min(int(recent), int(keep)), out._ref,
            lens_out.data_ptr(), _lib._ptr(mass_out), ld_out, slots.data_ptr(), ws.data_ptr(),
            ws.numel() * ws.element_size(), _lib._stream_of(stream, lens)))
    return lens_out, slots
