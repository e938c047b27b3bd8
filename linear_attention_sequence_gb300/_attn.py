"""Binding of the softmax attention calls (see ``include/kda.h``).  As in the rest of the
package: pointers, sizes and checks, no arithmetic of the method and no fallback.

In a packed batch with ``cu_seqlens``, rows that belong to no sequence (before its first
entry, from its last one on) are not written: outputs allocated here hold whatever the
memory held there."""
from __future__ import annotations

import ctypes
import struct

import torch

import linear_attention_sequence_gb300 as _kda

from ._ssm import _is, _on, _run, _sequences

_vp, _i32, _i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
_F32, _I32 = torch.float32, torch.int32
_TYPES = {torch.bfloat16: 1, torch.float16: 2}     # KDA_DTYPE_*
_OUT_TYPES = {torch.float32: 0, **_TYPES}

# The structures of include/kda.h as bytes (see _ssm.py).
_HEADS = struct.Struct("Pqq")                      # data, token stride, head stride
_PAGES = struct.Struct("Pqqq")                     # data, page, token, head stride
_DIMS = struct.Struct("7if")                       # N, T, H_q, H_kv, d, in, out, scale
_CACHE = struct.Struct("3i")                       # P, page_size, max_pages


# What a small call costs the host is mostly checks, so that they ask each tensor for as little as
# they can.  The current device, without making sure of the runtime first (a CUDA tensor has).
_current = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


class _Here:
    """Nothing to change: the call's device is current, and its stream the current one."""

    __slots__ = ()

    def __enter__(self):
        pass

    def __exit__(self, *exc):
        pass


_HERE = _Here()


def _place(dev, stream):
    return _HERE if stream is None and _current() == dev else _on(dev, stream)


_sizes = {}   # bytes of a workspace, by the query and the dims it was asked for


def _workspace(query, dims, device, *more):
    n = _sizes.get((query, dims, *more))
    if n is None:
        n = getattr(_kda.lib(), query)(dims, *more)
        if n < 0:
            raise _kda.KdaError(2, query)
        if len(_sizes) > 4096:
            _sizes.clear()
        _sizes[(query, dims, *more)] = n
    return torch.empty((n,), dtype=torch.uint8, device=device), n


def declare(L):
    """Argument types of the C entry points (structures go in as bytes)."""
    for name, args in (("kda_attn_prefill", [_vp] * 8),
                       ("kda_attn_backward", [_vp] * 12 + [_i64, _vp]),
                       ("kda_attn_paged", [_vp] * 11 + [_i64, _vp]),
                       ("kda_attn_paged_granted", [_vp] * 12 + [_i64, _vp])):
        getattr(L, name).argtypes = args
        getattr(L, name).restype = ctypes.c_int
    L.kda_attn_paged_workspace.argtypes = [_vp] * 3
    L.kda_attn_paged_workspace.restype = _i64
    L.kda_attn_backward_workspace.argtypes = [_vp]
    L.kda_attn_backward_workspace.restype = _i64


def _heads(t, name, dev, dtype, shape):
    """The bytes of a [T, H, d] activation whose tokens and heads may lie strides apart."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        if t.get_device() != dev:
            raise ValueError(f"{name} must be a CUDA tensor on device {dev}")
        raise ValueError(f"{name} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    a, b, c = t.stride()
    T, H, d = shape
    if c != 1 and d > 1:
        raise ValueError(f"{name}'s channels must be contiguous")
    if T <= 1:
        a = H * d
    if H == 1:
        b = d
    at = t.data_ptr()
    if (a | b) & 7 or at & 15:
        raise ValueError(f"{name} must be 16-byte aligned, in its strides too")
    return _HEADS.pack(at, a, b)


def _pages(t, name, dev, dtype, shape):
    """The bytes of a cache [P, page, H, d] with strides."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        if t.get_device() != dev:
            raise ValueError(f"{name} must be a CUDA tensor on device {dev}")
        raise ValueError(f"{name} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    p, s, h, c = t.stride()
    P, page, H, d = shape
    if c != 1 and d > 1:
        raise ValueError(f"{name}'s channels must be contiguous")
    # (the stride of a dimension of one is any)
    if H == 1:
        h = d
    if page == 1:
        s = h * H
    if P == 1:
        p = max(s * page, h * H)
    at = t.data_ptr()
    if (p | s | h) & 7 or at & 15:
        raise ValueError(f"{name} must be 16-byte aligned, in its strides too")
    return _PAGES.pack(at, p, s, h)


def _query(q, kv_heads, N, scale, out_dtype):
    """(device, T, H_q, d, type, dims) of a call with queries q [T, H_q, d]."""
    if q.dim() != 3 or not q.is_cuda:
        raise ValueError("q must be a CUDA tensor [T, H, d]")
    code = _TYPES.get(q.dtype)
    if code is None:
        raise ValueError("q must be bf16 or fp16")
    T, H, d = q.shape
    out_code = _OUT_TYPES.get(out_dtype)
    if out_code is None:
        raise ValueError("out_dtype must be q's dtype or fp32")
    if scale is None:
        scale = d ** -0.5 if d else 1.0
    return _DIMS.pack(N, T, H, kv_heads, d, code, out_code, scale)


def kda_attn_prefill(q, k, v, cu_seqlens=None, *, num_seqs=None, scale=None, out=None, out_dtype=None,
                     lse=None, return_lse=False, stream=None):
    """Causal softmax attention over the whole prompts of a packed batch (C entry point
    ``kda_attn_prefill``).

    q [T, H, d], k and v [T, H_kv, d] in bf16 or fp16, d 64 or 128, H a multiple of H_kv;
    tokens and heads may lie strides apart (multiples of 8 elements).  scale defaults
    to d^-1/2.  Returns ``out`` [T, H, d] (``out_dtype``, default q's), and with
    ``return_lse`` (or a buffer given) ``(out, lse)``, lse fp32 [T, H], which the gradients need."""
    if k.dim() != 3:
        raise ValueError("k must be [T, H, d]")
    odt = out_dtype or q.dtype
    dev = q.get_device()
    N = _sequences(cu_seqlens, num_seqs, dev)
    dims = _query(q, k.shape[1], N, scale, odt)
    T, H, d = q.shape
    kv = (T, k.shape[1], d)
    rq, rk, rv = (_heads(q, "q", dev, q.dtype, (T, H, d)), _heads(k, "k", dev, q.dtype, kv),
                  _heads(v, "v", dev, q.dtype, kv))
    o, s = _is(out, "out", dev, odt, (T, H, d)), _is(lse, "lse", dev, _F32, (T, H))
    with _place(dev, stream):
        if out is None:
            out = torch.empty((T, H, d), dtype=odt, device=q.device)
            o = out.data_ptr()
        if lse is None and return_lse:
            lse = torch.empty((T, H), dtype=_F32, device=q.device)
            s = lse.data_ptr()
        _run("kda_attn_prefill", dev, dims, rq, rk, rv, 0 if cu_seqlens is None else cu_seqlens.data_ptr(), o, s)
    return out if lse is None else (out, lse)


def kda_attn_backward(q, k, v, out, lse, d_out, cu_seqlens=None, *, num_seqs=None, scale=None,
                      grad_dtype=None, dq=None, dk=None, dv=None, stream=None):
    """Gradients of kda_attn_prefill (C entry point ``kda_attn_backward``) for d_out [T, H, d].

    q, k, v, cu_seqlens and scale as in the forward call, out (in q's dtype) and lse its results;
    all activations may have strides.  Returns a dict with dq, dk and dv (``grad_dtype``,
    default q's dtype)."""
    if k.dim() != 3 or out is None or lse is None or d_out is None:
        raise ValueError("k must be [T, H, d]; out, lse and d_out are needed")
    gdt = grad_dtype or q.dtype
    dev = q.get_device()
    N = _sequences(cu_seqlens, num_seqs, dev)
    dims = _query(q, k.shape[1], N, scale, gdt)
    T, H, d = q.shape
    own, kv = (T, H, d), (T, k.shape[1], d)
    rq, ro, ry = (_heads(x, n, dev, q.dtype, own) for x, n in ((q, "q"), (out, "out"), (d_out, "d_out")))
    rk, rv = (_heads(x, n, dev, q.dtype, kv) for x, n in ((k, "k"), (v, "v")))
    sums = _is(lse, "lse", dev, _F32, (T, H))
    for x, n, shape in ((dq, "dq", own), (dk, "dk", kv), (dv, "dv", kv)):
        _is(x, n, dev, gdt, shape)
    with _place(dev, stream):
        def new(given, shape):
            return torch.empty(shape, dtype=gdt, device=q.device) if given is None else given

        dq, dk, dv = new(dq, own), new(dk, kv), new(dv, kv)
        ws, n = _workspace("kda_attn_backward_workspace", dims, q.device)
        _run("kda_attn_backward", dev, dims, rq, rk, rv, ro, sums, ry,
             0 if cu_seqlens is None else cu_seqlens.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), ws.data_ptr(), n)
    return dict(dq=dq, dk=dk, dv=dv)


def kda_attn_paged(q, k_pages, v_pages, page_table, kv_lens, cu_seqlens=None, *, granted=None, scale=None, out=None,
                   out_dtype=None, lse=None, return_lse=False, stream=None):
    """Attention of each sequence's new tokens over its pages of a cache, which holds their
    keys and values already (C entry point ``kda_attn_paged``).

    q [T, H, d] of the new tokens (bf16 or fp16, d 64 or 128); k_pages and v_pages
    [P, page_size, H_kv, d] with strides (multiples of 8 elements), page_size a power of two
    from 8 to 1024; page_table int32 [N, max_pages]; kv_lens int32 [N], the tokens in the
    cache with the new ones; cu_seqlens int32 [N+1] of the new tokens, or None: T / N each
    (T == N is the decode step).  Returns ``out`` [T, H, d], and with ``return_lse`` (or
    a buffer given) ``(out, lse)``.  A token that sees no key has out 0 and lse -inf; so has, with
    granted (int32 [N], what kda_cache_reserve granted), every token of a sequence that was refused."""
    if k_pages.dim() != 4 or page_table.dim() != 2:
        raise ValueError("k_pages must be [P, page_size, H, d] and page_table [N, max_pages]")
    odt = out_dtype or q.dtype
    dev = q.get_device()
    N, wide = page_table.shape
    if cu_seqlens is not None and _sequences(cu_seqlens, None, dev) != N:
        raise ValueError("cu_seqlens must hold N + 1 entries")
    P, page, Hkv, _ = k_pages.shape
    dims, cache = _query(q, Hkv, N, scale, odt), _CACHE.pack(P, page, wide)
    T, H, d = q.shape
    kv = (P, page, Hkv, d)
    rq, rk, rv = (_heads(q, "q", dev, q.dtype, (T, H, d)), _pages(k_pages, "k_pages", dev, q.dtype, kv),
                  _pages(v_pages, "v_pages", dev, q.dtype, kv))
    table = _is(page_table, "page_table", dev, _I32, (N, wide))
    lens = _is(kv_lens, "kv_lens", dev, _I32, (N,))
    cu = 0 if cu_seqlens is None else cu_seqlens.data_ptr()
    got = _is(granted, "granted", dev, _I32, (N,))
    o, s = _is(out, "out", dev, odt, (T, H, d)), _is(lse, "lse", dev, _F32, (T, H))
    with _place(dev, stream):
        if out is None:
            out = torch.empty((T, H, d), dtype=odt, device=q.device)
            o = out.data_ptr()
        if lse is None and return_lse:
            lse = torch.empty((T, H), dtype=_F32, device=q.device)
            s = lse.data_ptr()
        # (of cu_seqlens it matters only whether there are any; any address stands for them)
        ws, n = _workspace("kda_attn_paged_workspace", dims, q.device, cache, 16 if cu else 0)
        _run("kda_attn_paged_granted", dev, dims, cache, rq, rk, rv, table, lens, cu, got, o, s, ws.data_ptr(), n)
    return out if lse is None else (out, lse)
