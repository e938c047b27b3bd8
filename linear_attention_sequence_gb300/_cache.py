"""Binding of the calls on the pages of a cache (see ``include/kda.h``).  As in the rest of
the package: pointers, sizes and checks, no arithmetic of the method and no fallback.

The state of a cache is three int32 tensors on the device, kept by the caller and written
in place: ``page_refs`` [P] (0: free), ``page_table`` [N, max_pages] (-1: none) and ``kv_lens``
[N].  An empty cache is zeros, -1 and zeros.  No call waits for the host."""
from __future__ import annotations

import ctypes

import torch

import linear_attention_sequence_gb300 as _kda

from ._attn import _CACHE, _TYPES, _heads, _pages, _place, _workspace
from ._ssm import _is, _run, _sequences

_vp, _i32, _i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
_I32 = torch.int32


def declare(L):
    """Argument types of the C entry points (structures go in as bytes)."""
    for name, args in (("kda_cache_reserve", [_vp, _i32] + [_vp] * 8 + [_i64, _vp]),
                       ("kda_cache_reserve_granted", [_vp, _i32] + [_vp] * 9 + [_i64, _vp]),
                       ("kda_cache_append", [_vp] + [_i32] * 4 + [_vp] * 8),
                       ("kda_cache_append_granted", [_vp] + [_i32] * 4 + [_vp] * 9),
                       ("kda_cache_free", [_vp, _i32] + [_vp] * 3 + [_i32] + [_vp] * 3),
                       ("kda_cache_fork", [_vp, _i32] + [_vp] * 3 + [_i32] + [_vp] * 6 + [_i64, _vp]),
                       ("kda_cache_compact", [_vp, _i32] + [_vp] * 8 + [_i64, _vp]),
                       ("kda_cache_copy", [_vp] + [_i32] * 2 + [_vp] * 2 + [_i32] + [_vp] * 3)):
        getattr(L, name).argtypes = args
        getattr(L, name).restype = ctypes.c_int
    L.kda_cache_workspace.argtypes = [_vp]
    L.kda_cache_workspace.restype = _i64


def _int(t, name, dev, shape):
    """The address of a contiguous int32 tensor of this shape on this device (_is, for the usual case
    in fewer steps)."""
    if t is not None and t.dtype is _I32 and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    return _is(t, name, dev, _I32, shape)


def _state(page_refs, page_table, kv_lens, page_size):
    """(device, N, cache dims, addresses of refs, table and lens) of a cache's state."""
    if page_refs is None or page_refs.dim() != 1 or page_refs.get_device() < 0:
        raise ValueError("page_refs must be a CUDA tensor [P]")
    if page_table is None or page_table.dim() != 2:
        raise ValueError("page_table must be [N, max_pages]")
    dev = page_refs.get_device()
    shape, own = page_table.shape, page_refs.shape
    N = shape[0]
    return (dev, N, _CACHE.pack(own[0], page_size, shape[1]), _int(page_refs, "page_refs", dev, own),
            _int(page_table, "page_table", dev, shape), _int(kv_lens, "kv_lens", dev, (N,)))


def _scratch(cache, device):
    return _workspace("kda_cache_workspace", cache, device)


def _layer(k_pages, v_pages):
    """(device, P, page size, H, d, bytes of both) of one layer's pages."""
    if k_pages.dim() != 4 or not k_pages.is_cuda:
        raise ValueError("k_pages must be a CUDA tensor [P, page_size, H, d]")
    if k_pages.dtype not in _TYPES:
        raise ValueError("k_pages must be bf16 or fp16")
    dev, shape = k_pages.get_device(), k_pages.shape
    return (dev, *shape, _pages(k_pages, "k_pages", dev, k_pages.dtype, shape),
            _pages(v_pages, "v_pages", dev, k_pages.dtype, shape))


def kda_cache_reserve(page_refs, page_table, kv_lens, new_lens, page_size, *, src=None, dst=None,
                      return_copies=False, missing=None, granted=None, return_granted=False, stream=None):
    """Pages for ``new_lens`` (int32 [N]) more tokens of each sequence, in place (C entry point
    ``kda_cache_reserve``): kv_lens grows and the table gets the lowest free pages, for the
    sequences in their order; one that cannot have all of its pages keeps its length.
    ``missing`` (int32 [1] or None) gets the number of pages that were lacking.

    A sequence that was shortened into a page that others share (kda_cache_free with ``keep``
    after kda_cache_fork) gets a page of its own when it grows again: with ``return_copies``
    (or buffers given) returns ``(src, dst)``, int32 [N], the pages to copy with kda_cache_copy in
    every layer (-1: none); without, such a sequence keeps its length and the device status
    says so.

    Where pages or rows may run out: with ``return_granted`` (or a buffer given) also returns
    ``granted``, int32 [N], the new tokens of each sequence that have a place (0 for one that keeps
    its length).  Hand it to kda_cache_append and kda_attn_paged, or the tokens of a refused sequence are
    written over the last ones that it has.  Without ``missing`` and ``granted`` the device status
    tells of a refusal."""
    dev, N, cache, refs, table, lens = _state(page_refs, page_table, kv_lens, page_size)
    new = _int(new_lens, "new_lens", dev, (N,))
    lacking = _int(missing, "missing", dev, (1,))
    with _place(dev, stream):
        if return_copies and src is None:
            src = torch.empty((N,), dtype=_I32, device=page_refs.device)
        if return_copies and dst is None:
            dst = torch.empty((N,), dtype=_I32, device=page_refs.device)
        if return_granted and granted is None:
            granted = torch.empty((N,), dtype=_I32, device=page_refs.device)
        ws, n = _scratch(cache, page_refs.device)
        _run("kda_cache_reserve_granted", dev, cache, N, refs, table, lens, new, _int(src, "src", dev, (N,)),
             _int(dst, "dst", dev, (N,)), lacking, _int(granted, "granted", dev, (N,)), ws.data_ptr(), n)
    if granted is None:
        return None if src is None else (src, dst)
    return granted if src is None else (src, dst, granted)


def kda_cache_append(k, v, k_pages, v_pages, page_table, kv_lens, cu_seqlens=None, *, granted=None, stream=None):
    """Writes the new tokens' k and v [T, H, d] into one layer's pages [P, page_size, H, d] (C
    entry point ``kda_cache_append``): of the n new tokens of a sequence, token i goes to place
    kv_lens - n + i, so that kda_cache_reserve comes first.  cu_seqlens int32 [N+1] of the new
    tokens, or None: T / N each.  granted int32 [N] is what kda_cache_reserve granted: sequences that
    were refused are passed by; without it every sequence must have been served."""
    dev, P, page, H, d, kp, vp = _layer(k_pages, v_pages)
    if page_table.dim() != 2 or k.dim() != 3:
        raise ValueError("page_table must be [N, max_pages] and k [T, H, d]")
    N, wide = page_table.shape
    if cu_seqlens is not None and _sequences(cu_seqlens, None, dev) != N:
        raise ValueError("cu_seqlens must hold N + 1 entries")
    T = k.shape[0]
    rk, rv = (_heads(x, name, dev, k_pages.dtype, (T, H, d)) for x, name in ((k, "k"), (v, "v")))
    table = _int(page_table, "page_table", dev, (N, wide))
    lens = _int(kv_lens, "kv_lens", dev, (N,))
    with _place(dev, stream):
        _run("kda_cache_append_granted", dev, _CACHE.pack(P, page, wide), N, T, H, d, rk, rv, kp, vp, table, lens,
             0 if cu_seqlens is None else cu_seqlens.data_ptr(), _int(granted, "granted", dev, (N,)))


def kda_cache_free(page_refs, page_table, kv_lens, seqs, page_size, *, keep=None, stream=None):
    """Gives pages back, in place (C entry point ``kda_cache_free``): of each sequence in ``seqs``
    (int32 [M]) the first ``keep`` tokens stay (int32 [M]; None: none of them); the pages
    behind are free unless another sequence shares them."""
    dev, N, cache, refs, table, lens = _state(page_refs, page_table, kv_lens, page_size)
    if seqs is None or seqs.dim() != 1:
        raise ValueError("seqs must be [M]")
    M = seqs.shape[0]
    with _place(dev, stream):
        _run("kda_cache_free", dev, cache, N, refs, table, lens, M, _int(seqs, "seqs", dev, (M,)),
             _int(keep, "keep", dev, (M,)))


def kda_cache_fork(page_refs, page_table, kv_lens, parents, children, page_size, *, src=None, dst=None,
                   missing=None, stream=None):
    """children[i] (an empty row) becomes a continuation of parents[i] (both int32 [M]), in place
    (C entry point ``kda_cache_fork``): it shares the parent's full pages and has one of its
    own where the last is not full; a row that has pages is passed by.  Returns ``(src, dst)``, int32 [M]: the pages to copy with
    kda_cache_copy in every layer (-1: none)."""
    dev, N, cache, refs, table, lens = _state(page_refs, page_table, kv_lens, page_size)
    if parents is None or parents.dim() != 1:
        raise ValueError("parents must be [M]")
    M = parents.shape[0]
    p, c = _int(parents, "parents", dev, (M,)), _int(children, "children", dev, (M,))
    lacking = _int(missing, "missing", dev, (1,))
    with _place(dev, stream):
        if src is None:
            src = torch.empty((M,), dtype=_I32, device=page_refs.device)
        if dst is None:
            dst = torch.empty((M,), dtype=_I32, device=page_refs.device)
        ws, n = _scratch(cache, page_refs.device)
        _run("kda_cache_fork", dev, cache, N, refs, table, lens, M, p, c, _int(src, "src", dev, (M,)),
             _int(dst, "dst", dev, (M,)), lacking, ws.data_ptr(), n)
    return src, dst


def kda_cache_compact(page_refs, page_table, kv_lens, page_size, *, refs_out=None, table_out=None, src=None,
                      dst=None, stream=None):
    """Renumbers the pages so that those in use come first (C entry point ``kda_cache_compact``).
    Returns ``(refs_out, table_out, src, dst)``: the new counts and table (new tensors unless
    given; page_refs and page_table themselves may be given), and int32 [P] lists of the pages to
    copy with kda_cache_copy in every layer (-1: none)."""
    dev, N, cache, refs, table, lens = _state(page_refs, page_table, kv_lens, page_size)
    P, shape = page_refs.shape[0], tuple(page_table.shape)
    with _place(dev, stream):
        def new(given, shape):
            return torch.empty(shape, dtype=_I32, device=page_refs.device) if given is None else given

        refs_out, table_out = new(refs_out, (P,)), new(table_out, shape)
        src, dst = new(src, (P,)), new(dst, (P,))
        ws, n = _scratch(cache, page_refs.device)
        _run("kda_cache_compact", dev, cache, N, refs, table, lens, _int(refs_out, "refs_out", dev, (P,)),
             _int(table_out, "table_out", dev, shape), _int(src, "src", dev, (P,)),
             _int(dst, "dst", dev, (P,)), ws.data_ptr(), n)
    return refs_out, table_out, src, dst


def kda_cache_copy(k_pages, v_pages, src, dst, *, stream=None):
    """Page dst[i] of one layer's keys and values becomes a copy of page src[i] (int32 [M]; -1: no
    copy) (C entry point ``kda_cache_copy``)."""
    dev, P, page, H, d, kp, vp = _layer(k_pages, v_pages)
    if src is None or src.dim() != 1:
        raise ValueError("src must be [M]")
    M = src.shape[0]
    with _place(dev, stream):
        _run("kda_cache_copy", dev, _CACHE.pack(P, page, 1), H, d, kp, vp, M, _int(src, "src", dev, (M,)),
             _int(dst, "dst", dev, (M,)))
