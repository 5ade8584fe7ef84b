"""A paged key/value cache held in 4 bits, and alpha-entmax attention of the newest tokens against it
(wrappers of the ``ent_attn_kv4_*`` calls of include/entattn.h, which states the format).

A step of a decoder layer, B sequences with up to L new tokens each::

    cache = kv4_alloc(pages, heads, page, d, device)              # once
    kv4_write(cache, k, v, block_table, start, new_lens)          # k, v [B, Hkv, L, d]
    o = entmax_attn_kv4(q, cache, block_table, start, alpha, new_lens=new_lens)   # q [B, Hq, L, d]

``block_table`` int32 [B, max_pages] names the pages of each sequence in order, ``start`` int32 [B] the
position of row 0 (the tokens cached before), ``new_lens`` int32 [B] the rows that are real (None: all L).
"""
from __future__ import annotations

import functools
from typing import NamedTuple

import torch

from . import capi
from .attention import _DTYPES, _on, _raise, _stream_handle

_GROUP = 32


class KV4Cache(NamedTuple):
    """The pool's arrays: codes uint8 [pages, heads, page, d/2], meta bfloat16 [pages, heads, page,
    d/32, 2].  Every function here takes a plain tuple of the four as well."""
    k_codes: torch.Tensor
    k_meta: torch.Tensor
    v_codes: torch.Tensor
    v_meta: torch.Tensor


def kv4_alloc(pages: int, heads: int, page: int, d: int, device="cuda") -> KV4Cache:
    """A pool of ``pages`` pages of ``page`` tokens (a power of two, at least 16), all zeros."""
    if d not in (32, 64, 128):
        raise ValueError(f"head dim {d} not supported (32, 64 or 128)")
    if page < 16 or page & (page - 1):
        raise ValueError(f"page must be a power of two of at least 16, not {page}")
    shape = (pages, heads, page)
    return KV4Cache(*(torch.zeros(shape + tail, dtype=t, device=device)
                      for _ in "kv" for tail, t in (((d // 2,), torch.uint8),
                                                    ((d // _GROUP, 2), torch.bfloat16))))


def _place(device):
    """What get_device() gives of a tensor there (the CPU: -1)."""
    return -1 if device.index is None else device.index


def _check_cache(cache, device):
    """(pages, heads, page, d) of the pool.  (These checks are a third of a small call's host time: each
    attribute is asked for once.)"""
    kc, km, vc, vm = cache
    shape = kc.shape
    if len(shape) != 4:
        raise ValueError(f"expected codes [pages, heads, page, d/2], got shape {tuple(shape)}")
    pages, heads, page, half = shape
    meta = (pages, heads, page, half // 16, 2)
    if not (vc.shape == shape and km.shape == meta and vm.shape == meta and kc.dtype is torch.uint8
            and vc.dtype is torch.uint8 and km.dtype is torch.bfloat16 and vm.dtype is torch.bfloat16):
        raise ValueError("the cache must be codes uint8 [pages, heads, page, d/2] and meta bfloat16 "
                         "[pages, heads, page, d/32, 2], keys and values alike")
    where = _place(device)
    if not (where == kc.get_device() == km.get_device() == vc.get_device() == vm.get_device()):
        raise ValueError("the cache must be on the device of the other tensors")
    if not (kc.is_contiguous() and km.is_contiguous() and vc.is_contiguous() and vm.is_contiguous()):
        raise ValueError("the cache's arrays must be contiguous")
    return pages, heads, page, 2 * half


def _pointer(t, n, where):
    """Device pointer of an int32 tensor of n values (None: none)."""
    if t is None:
        return None
    if not (t.dtype is torch.int32 and t.shape == (n,) and t.get_device() == where
            and t.is_contiguous()):
        raise ValueError("start, new_lens and bad must be contiguous int32 tensors of shapes [B], [B] and [1] "
                         "on the device of the others")
    return t.data_ptr()


def _check_seqs(block_table, start, new_lens, bad, B, device):
    """Device pointers (table, start, new_lens or None, bad or None) and the table's columns."""
    shape, where = block_table.shape, _place(device)
    if len(shape) != 2 or shape[0] != B:
        raise ValueError(f"expected block_table [{B}, max_pages], got shape {tuple(shape)}")
    if not (block_table.dtype is torch.int32 and block_table.get_device() == where
            and block_table.is_contiguous()):
        raise ValueError("block_table must be a contiguous int32 tensor on the device of the others")
    if start is None:
        raise ValueError("start is needed")
    return (block_table.data_ptr(), _pointer(start, B, where), _pointer(new_lens, B, where),
            _pointer(bad, 1, where), shape[1])


# sizes alone go in: a decoder asks with the same ones at every step
_workspace_size = functools.lru_cache(maxsize=256)(lambda *sizes: capi.ent_attn_kv4_workspace_size(*sizes))


def _check_rows4(*ts):
    t0 = ts[0]
    if t0.dim() != 4:
        raise ValueError(f"expected [B, H, L, d] tensors, got shape {tuple(t0.shape)}")
    if t0.dtype not in _DTYPES:
        raise ValueError(f"dtype {t0.dtype} not supported (float32 or bfloat16)")
    for t in ts:
        if t.shape != t0.shape or t.dtype != t0.dtype or t.device != t0.device:
            raise ValueError("tensors must share shape, dtype and device")
    for t in ts:
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("tensors must be contiguous CUDA tensors")


def _call(fn, device, *args):
    """fn(*args, stream) with the tensors' device current."""
    with _on(device):
        st = fn(*args, _stream_handle(device))
    _raise(st, fn.__name__)


def kv4_write(cache, k, v, block_table, start, new_lens=None, *, bad=None) -> None:
    """Quantise k, v [B, Hkv, L, d] into the cache at positions start .. start + new_lens - 1.

    ``bad`` (int32 [1], zeroed by the caller) gets bit 0 set where a page number lies outside the pool,
    bit 1 where a start or length lies outside the table; the rows concerned are not written (and in the
    attention bit 2 if a bounded device wait gave up).  Pages
    being written must belong to one sequence."""
    _check_rows4(k, v)
    B, H, L, d = k.shape
    pages, heads, page, dc = _check_cache(cache, k.device)
    if (heads, dc) != (H, d):
        raise ValueError(f"the cache holds {heads} heads of {dc}, not {H} of {d}")
    table, st, nl, bp, max_pages = _check_seqs(block_table, start, new_lens, bad, B, k.device)
    _call(capi.ent_attn_kv4_write, k.device, k.data_ptr(), v.data_ptr(), B, H, L, d, _DTYPES[k.dtype],
          table, max_pages, st, nl, *(t.data_ptr() for t in cache), pages, page, bp)


def kv4_read(cache, block_table, start, n: int, new_lens=None, *, dtype=torch.bfloat16, out=None, bad=None):
    """The cached values of positions start .. start + n - 1 (``new_lens``: of its first rows only, the
    rest zeros): (k, v) [B, Hkv, n, d] in ``dtype`` (float32 or bfloat16), or in ``out``."""
    device = block_table.device
    pages, heads, page, d = _check_cache(cache, device)
    B = block_table.shape[0]
    if out is None:
        if dtype not in _DTYPES:
            raise ValueError(f"dtype {dtype} not supported (float32 or bfloat16)")
        if n < 0:
            raise ValueError(f"negative n={n}")
        k = torch.empty((B, heads, n, d), dtype=dtype, device=device)
        v = torch.empty_like(k)
    else:
        k, v = out
        if k.shape != (B, heads, n, d):
            raise ValueError(f"out must be of shape {(B, heads, n, d)}, not {tuple(k.shape)}")
    _check_rows4(k, v)
    if k.device != device:
        raise ValueError("out must be on the device of the other tensors")
    table, st, nl, bp, max_pages = _check_seqs(block_table, start, new_lens, bad, B, device)
    _call(capi.ent_attn_kv4_read, device, *(t.data_ptr() for t in cache), pages, page, table, max_pages,
          st, nl, B, heads, n, d, _DTYPES[k.dtype], k.data_ptr(), v.data_ptr(), bp)
    return k, v


def _cover(window, sinks, max_len, cap):
    """(window, sinks, max_len) as the library takes them: window 0 for none, all within 31 bits."""
    if window is None:
        if sinks:
            raise ValueError("sinks need a window")
        window = 0
    elif window < 1 or sinks < 0:
        raise ValueError(f"window must be at least 1 and sinks at least 0, not {window} and {sinks}")
    if max_len is None:
        max_len = cap
    elif not 0 <= max_len <= cap:
        raise ValueError(f"max_len must lie in 0 .. {cap} (what the block table covers), not {max_len}")
    big = 2 ** 31 - 1
    return min(window, big), min(sinks, big), max_len


def kv4_workspace(q, cache, block_table, *, window: int | None = None, sinks: int = 0,
                  max_len: int | None = None) -> torch.Tensor:
    """A workspace for ``entmax_attn_kv4`` of these arguments; it serves one call at a time."""
    B, Hq, L, d = q.shape
    window, sinks, max_len = _cover(window, sinks, max_len, block_table.shape[1] * cache[0].shape[2])
    n = _workspace_size(B, Hq, cache[0].shape[1], L, d, _DTYPES[q.dtype], max_len, window, sinks)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=q.device)


def entmax_attn_kv4(q, cache, block_table, start, alpha: float = 1.5, *, new_lens=None,
                    window: int | None = None, sinks: int = 0, max_len: int | None = None, out=None,
                    tau=None, ws: torch.Tensor | None = None, bad=None):
    """O [B, Hq, L, d] of the newest tokens' queries against the cache (their keys are in it already).

    Row l of sequence b, at position i = start[b] + l, sees key j when j <= i and, with a ``window``,
    i - j < window or j < sinks; rows from new_lens[b] on give zeros.  Query head h reads key head
    h // (Hq // Hkv).  ``max_len`` bounds start + new_lens (default: what the table covers) and sizes
    the workspace, 8 bytes for each query row and token of that cover (of window + sinks + L under a
    window): give it where the table covers much more than the sequences hold, and few rows a call
    where they are long; ``tau`` (float32 [B, Hq, L]) also takes the rows' thresholds; ``bad`` as in
    ``kv4_write``.  No gradient."""
    _check_rows4(q)
    B, Hq, L, d = q.shape
    device = q.device
    pages, heads, page, dc = _check_cache(cache, device)
    if dc != d or Hq % heads:
        raise ValueError(f"the cache holds {heads} heads of {dc}; q has {Hq} of {d}")
    window, sinks, max_len = _cover(window, sinks, max_len, block_table.shape[-1] * page)
    table, st, nl, bp, max_pages = _check_seqs(block_table, start, new_lens, bad, B, device)
    dt = _DTYPES[q.dtype]
    if out is None:
        out = torch.empty_like(q)
    else:
        _check_rows4(q, out)
    if tau is not None and (tau.dtype != torch.float32 or tau.shape != (B, Hq, L) or tau.device != device
                            or not tau.is_contiguous()):
        raise ValueError("tau must be a contiguous float32 tensor [B, Hq, L] on the device of q")
    need = _workspace_size(B, Hq, heads, L, d, dt, max_len, window, sinks)
    if ws is None or ws.numel() < need:
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=device)
    elif ws.dtype != torch.uint8 or ws.device != device or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous uint8 tensor on the device of q")
    _call(capi.ent_attn_kv4_fwd, device, q.data_ptr(), B, Hq, heads, L, d, dt, alpha, window, sinks,
          *(t.data_ptr() for t in cache), pages, page, table, max_pages, st, nl, max_len, out.data_ptr(),
          tau.data_ptr() if tau is not None else None, bp, ws.data_ptr(), ws.numel())
    return out
