"""Binding of the state space layer calls and the 8-bit packing (see
``include/kda.h``).  As in the rest of the package: pointers, sizes and checks,
no arithmetic of the method and no fallback.

In a packed batch with ``cu_seqlens``, rows that belong to no sequence (before its
first entry, from its last one on) are not written: outputs allocated here hold
whatever the memory held there."""
from __future__ import annotations

import ctypes
import struct

import torch

import linear_attention_sequence_gb300 as _kda

PACK_GROUP = 32   # channels that share a scale (KDA_PACK_GROUP)

_vp, _i32, _i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
_F32, _I32, _I8 = torch.float32, torch.int32, torch.int8

# The structures of include/kda.h as bytes: a call packs its arguments once instead of
# filling ctypes objects field by field, which would cost more than a small kernel.
_ROWS = struct.Struct("PqP")                     # data, stride, scales
_DIMS = struct.Struct("6i")                      # num_seqs, total_tokens, channels, state_size, in, out
_INPUTS = struct.Struct("PqP" * 5 + "PPPPi4x")   # u, dt, B, C, z; A, D, dt_bias, cu_seqlens, delta_softplus
_GRADS = struct.Struct("9P")                     # du, ddt, dB, dC, dz, dA, dD, ddt_bias, d_init_state
_GRAD_NAMES = ("du", "ddt", "dB", "dC", "dz", "dA", "dD", "ddt_bias", "d_init_state")


def declare(L):
    """Argument types of the C entry points (structures go in as bytes)."""
    for name, args in (("kda_act_pack8", [_i32, _i32, _i32] + [_vp] * 4),
                       ("kda_ssm_conv", [_vp] * 6 + [_i32] + [_vp] * 3),
                       ("kda_ssm_conv_backward", [_vp] * 6 + [_i32] + [_vp] * 7 + [_i64, _vp]),
                       ("kda_ssm_scan", [_vp] * 6 + [_i64, _vp, _i64, _vp]),
                       ("kda_ssm_step", [_vp] * 5),
                       ("kda_ssm_scan_backward", [_vp] * 4 + [_i64] + [_vp] * 4 + [_i64, _vp])):
        getattr(L, name).argtypes = args
        getattr(L, name).restype = ctypes.c_int
    for name in ("kda_ssm_conv_backward_workspace", "kda_ssm_scan_workspace",
                 "kda_ssm_scan_backward_workspace"):
        getattr(L, name).argtypes = [_vp]
        getattr(L, name).restype = _i64


def _p(t):
    return 0 if t is None else t.data_ptr()


def _device(t, name):
    """Index of the device of a [tokens, channels] activation."""
    if t is None or t.dim() != 2 or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor [tokens, channels]")
    return t.get_device()


def _is(t, name, dev, dtype, shape):
    """The address of a contiguous tensor of this type and shape on this device (None: 0)."""
    if t is None:
        return 0
    if (t.dtype == dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous()):
        return t.data_ptr()
    _kda._require(t, name, dtype, len(shape))
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on device {dev}")
    raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _rows(t, name, dev, dtype, shape, scales=None):
    """(address, stride, address of scales) of a [tokens, channels] activation whose rows
    may lie a stride apart, or of its int8 codes and scales."""
    if t is None:
        return 0, 0, 0
    if t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor on device {dev}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if scales is not None:
        if t.dtype != _I8 or not t.is_contiguous():
            raise ValueError(f"{name} with scales must be contiguous int8 codes")
        return t.data_ptr(), shape[1], _is(scales, f"scales of {name}", dev, _F32,
                                           (shape[0], -(-shape[1] // PACK_GROUP)))
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.is_contiguous():
        return t.data_ptr(), shape[1], 0
    down, across = t.stride()
    if shape[1] > 1 and across != 1:
        raise ValueError(f"{name}'s rows must be contiguous")
    if shape[0] == 1:
        return t.data_ptr(), shape[1], 0
    if down < shape[1]:
        raise ValueError(f"{name}'s rows must not overlap")
    return t.data_ptr(), down, 0


def _code(dtype, what):
    """The C code of an activation type."""
    code = _kda._DTYPES.get(dtype)
    if code is None:
        raise ValueError(f"{what} must be fp32 or bf16")
    return code


def _sequences(cu_seqlens, num_seqs, dev):
    if cu_seqlens is None:
        return 1 if num_seqs is None else int(num_seqs)
    _kda._require(cu_seqlens, "cu_seqlens", _I32, 1)
    if cu_seqlens.get_device() != dev or cu_seqlens.shape[0] < 1:
        raise ValueError(f"cu_seqlens must hold N + 1 entries on device {dev}")
    return cu_seqlens.shape[0] - 1


class _on:
    """Makes device ``dev`` current, and ``stream`` where one is given, for a call and
    for what it allocates: PyTorch's allocator gives a block out again only to work
    behind the stream that was current when it was allocated."""

    __slots__ = ("inner",)

    def __init__(self, dev, stream):
        self.inner = None
        if stream is not None:
            if stream.device.index != dev:
                raise ValueError(f"the stream must be on device {dev}")
            self.inner = torch.cuda.stream(stream)
        elif torch.cuda.current_device() != dev:
            self.inner = torch.cuda.device(dev)

    def __enter__(self):
        if self.inner is not None:
            self.inner.__enter__()

    def __exit__(self, *exc):
        if self.inner is not None:
            self.inner.__exit__(*exc)


# The handle of a device's current stream; the first form makes no stream object.
_stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _run(call, dev, *args):
    """The C call on the current stream of device ``dev``, which is the current device."""
    st = getattr(_kda._lib or _kda.lib(), call)(*args, _stream_of(dev))
    if st:
        _kda._check(st, call)


def _workspace(query, dims, device):
    n = getattr(_kda.lib(), query)(dims)
    if n < 0:
        raise _kda.KdaError(2, query)
    return torch.empty((n,), dtype=torch.uint8, device=device)


def kda_act_pack8(x, *, codes=None, scales=None, stream=None):
    """An activation x [T, D] (fp32 or bf16, rows may lie a stride apart) in 8
    bits (C entry point ``kda_act_pack8``).  Returns ``(codes, scales)``: int8
    [T, D] and fp32 [T, ceil(D / 32)]; ``codes * scale of the group`` stands for x."""
    dev, code = _device(x, "x"), _code(x.dtype, "x")
    T, D = x.shape
    G = -(-D // PACK_GROUP)
    r = _ROWS.pack(*_rows(x, "x", dev, x.dtype, (T, D)))
    with _on(dev, stream):
        if codes is None:
            codes = torch.empty((T, D), dtype=_I8, device=x.device)
        if scales is None:
            scales = torch.empty((T, G), dtype=_F32, device=x.device)
        _run("kda_act_pack8", dev, T, D, code, r, _is(codes, "codes", dev, _I8, (T, D)),
             _is(scales, "scales", dev, _F32, (T, G)))
    return codes, scales


def kda_ssm_conv(x, weight, bias=None, cu_seqlens=None, conv_state=None, *, num_seqs=None,
                 swish=True, out=None, out_dtype=None, conv_state_out=None,
                 return_conv_state=True, stream=None):
    """Causal convolution of W = 2..4 taps per channel over each sequence, and
    Swish (C entry point ``kda_ssm_conv``).

    x [T, D] fp32 or bf16 (rows may lie a stride apart); weight fp32 [D, W] (last
    tap on the current token); bias fp32 [D] or None; conv_state fp32 [N, W-1, D]
    or None (zeros): the inputs before each sequence, oldest first.  Returns
    ``(out, conv_state_out)``; conv_state_out may be conv_state itself (in place).
    One token per sequence (cu_seqlens None, num_seqs = T) is the decode step."""
    dev, code = _device(x, "x"), _code(x.dtype, "x")
    T, D = x.shape
    N = _sequences(cu_seqlens, num_seqs, dev)
    if weight.dim() != 2:
        raise ValueError("weight must be [D, W]")
    W = weight.shape[1]
    r = _ROWS.pack(*_rows(x, "x", dev, x.dtype, (T, D)))
    w = _is(weight, "weight", dev, _F32, (D, W))
    b = _is(bias, "bias", dev, _F32, (D,))
    cin = _is(conv_state, "conv_state", dev, _F32, (N, W - 1, D))
    odt = out_dtype or x.dtype
    dims = _DIMS.pack(N, T, D, W, code, _code(odt, "out_dtype"))
    with _on(dev, stream):
        if out is None:
            out = torch.empty((T, D), dtype=odt, device=x.device)
        if conv_state_out is None and return_conv_state:
            conv_state_out = torch.empty((N, W - 1, D), dtype=_F32, device=x.device)
        _run("kda_ssm_conv", dev, dims, r, w, b, cin, _p(cu_seqlens), bool(swish),
             _is(out, "out", dev, odt, (T, D)),
             _is(conv_state_out, "conv_state_out", dev, _F32, (N, W - 1, D)))
    return out, conv_state_out


def kda_ssm_conv_backward(x, weight, d_out, bias=None, cu_seqlens=None, conv_state=None, *,
                          x_scales=None, num_seqs=None, swish=True, d_conv_state_out=None,
                          grad_dtype=None, stream=None):
    """Gradients of kda_ssm_conv (C entry point ``kda_ssm_conv_backward``) for
    d_out [T, D] and d_conv_state_out fp32 [N, W-1, D] (None: zero).  x in the
    dtype of d_out, or the int8 codes of kda_act_pack8 with ``x_scales``.  Returns a
    dict with dx (``grad_dtype``, default the dtype of d_out), dweight, dbias and
    d_conv_state (fp32)."""
    dev, code = _device(d_out, "d_out"), _code(d_out.dtype, "d_out")
    T, D = d_out.shape
    N = _sequences(cu_seqlens, num_seqs, dev)
    if weight.dim() != 2:
        raise ValueError("weight must be [D, W]")
    if x is None:
        raise ValueError("x is needed")
    W = weight.shape[1]
    rx = _ROWS.pack(*_rows(x, "x", dev, d_out.dtype, (T, D), x_scales))
    ry = _ROWS.pack(*_rows(d_out, "d_out", dev, d_out.dtype, (T, D)))
    w = _is(weight, "weight", dev, _F32, (D, W))
    b = _is(bias, "bias", dev, _F32, (D,))
    cin = _is(conv_state, "conv_state", dev, _F32, (N, W - 1, D))
    dcout = _is(d_conv_state_out, "d_conv_state_out", dev, _F32, (N, W - 1, D))
    gdt = grad_dtype or d_out.dtype
    dims = _DIMS.pack(N, T, D, W, code, _code(gdt, "grad_dtype"))
    with _on(dev, stream):
        f32 = dict(dtype=_F32, device=d_out.device)
        dx = torch.empty((T, D), dtype=gdt, device=d_out.device)
        dw, db = torch.empty((D, W), **f32), torch.empty((D,), **f32)
        dcin = torch.empty((N, W - 1, D), **f32)
        ws = _workspace("kda_ssm_conv_backward_workspace", dims, d_out.device)
        _run("kda_ssm_conv_backward", dev, dims, rx, w, b, cin, _p(cu_seqlens), bool(swish), ry,
             dcout, dx.data_ptr(), dw.data_ptr(), db.data_ptr(), dcin.data_ptr(), ws.data_ptr(),
             ws.shape[0])
    return dict(dx=dx, dweight=dw, dbias=db, d_conv_state=dcin)


def _scan_args(u, dt, A, B, C, D, z, dt_bias, cu_seqlens, num_seqs, softplus, u_scales=None,
               z_scales=None):
    """Device, type code, N, T, channels, states and the packed inputs of a scan call."""
    dev, dtype = _device(dt, "dt"), dt.dtype
    code = _code(dtype, "dt, B and C")
    T, ch = shape = dt.shape
    if A.dim() != 2:
        raise ValueError("A must be [D, S]")
    if u is None or B is None or C is None:
        raise ValueError("u, B and C are needed")
    S = A.shape[1]
    N = _sequences(cu_seqlens, num_seqs, dev)
    if z is not None and (u_scales is None) != (z_scales is None):
        raise ValueError("u and z must both be packed or neither")
    return dev, code, N, T, ch, S, _INPUTS.pack(
        *_rows(u, "u", dev, dtype, shape, u_scales), *_rows(dt, "dt", dev, dtype, shape),
        *_rows(B, "B", dev, dtype, (T, S)), *_rows(C, "C", dev, dtype, (T, S)),
        *_rows(z, "z", dev, dtype, shape, z_scales), _is(A, "A", dev, _F32, (ch, S)),
        _is(D, "D", dev, _F32, (ch,)), _is(dt_bias, "dt_bias", dev, _F32, (ch,)),
        _p(cu_seqlens), bool(softplus))


def kda_ssm_scan(u, dt, A, B, C, D=None, z=None, dt_bias=None, init_state=None, cu_seqlens=None,
                 *, num_seqs=None, softplus=True, out=None, out_dtype=None, final_state=None,
                 return_final_state=True, chunk_states=None, return_chunk_states=False,
                 stream=None):
    """Selective scan over a packed batch (C entry point ``kda_ssm_scan``):
    Delta = softplus(dt + dt_bias), h_t = exp(Delta A) h_{t-1} + Delta u_t B_t,
    out = (C_t . h_t + D u_t) * Swish(z_t).

    u, dt, z [T, D] and B, C [T, S] in one dtype, fp32 or bf16 (rows may lie a stride
    apart); A fp32 [D, S]; D, dt_bias fp32 [D]; states fp32 [N, D, S].  Returns
    ``(out, final_state)``, and with ``return_chunk_states`` (or a buffer given)
    the states after every 32 tokens of each sequence, which the gradients need
    (cu_seqlens is copied to the host to count them unless a buffer is given)."""
    dev, code, N, T, ch, S, ins = _scan_args(u, dt, A, B, C, D, z, dt_bias, cu_seqlens, num_seqs,
                                             softplus)
    init = _is(init_state, "init_state", dev, _F32, (N, ch, S))
    odt = out_dtype or dt.dtype
    dims = _DIMS.pack(N, T, ch, S, code, _code(odt, "out_dtype"))
    with _on(dev, stream):
        if out is None:
            out = torch.empty((T, ch), dtype=odt, device=dt.device)
        if final_state is None and return_final_state:
            final_state = torch.empty((N, ch, S), dtype=_F32, device=dt.device)
        if chunk_states is None and return_chunk_states:
            rows = _kda.checkpoint_count(T, _kda.CHUNK, cu_seqlens, N)
            chunk_states = torch.empty((rows, ch, S), dtype=_F32, device=dt.device)
        cap = 0 if chunk_states is None else chunk_states.shape[0]
        chunks = _is(chunk_states, "chunk_states", dev, _F32, (cap, ch, S))
        ws = _workspace("kda_ssm_scan_workspace", dims, dt.device)
        _run("kda_ssm_scan", dev, dims, ins, init, _is(out, "out", dev, odt, (T, ch)),
             _is(final_state, "final_state", dev, _F32, (N, ch, S)), chunks, cap, ws.data_ptr(),
             ws.shape[0])
    return (out, final_state) if chunk_states is None else (out, final_state, chunk_states)


def kda_ssm_step(u, dt, A, B, C, state, D=None, z=None, dt_bias=None, *, softplus=True, out=None,
                 out_dtype=None, stream=None):
    """One token of the scan for N sequences (C entry point ``kda_ssm_step``): u,
    dt, z [N, D], B, C [N, S], state fp32 [N, D, S] updated in place.  Returns out
    [N, D]."""
    if state is None:
        raise ValueError("state is needed")
    dev, code, N, _, ch, S, ins = _scan_args(u, dt, A, B, C, D, z, dt_bias, None, dt.shape[0],
                                             softplus)
    st = _is(state, "state", dev, _F32, (N, ch, S))
    odt = out_dtype or dt.dtype
    dims = _DIMS.pack(N, N, ch, S, code, _code(odt, "out_dtype"))
    with _on(dev, stream):
        if out is None:
            out = torch.empty((N, ch), dtype=odt, device=dt.device)
        _run("kda_ssm_step", dev, dims, ins, st, _is(out, "out", dev, odt, (N, ch)))
    return out


def kda_ssm_scan_backward(u, dt, A, B, C, d_out, d_final_state=None, D=None, z=None, dt_bias=None,
                          init_state=None, cu_seqlens=None, *, chunk_states=None, u_scales=None,
                          z_scales=None, num_seqs=None, softplus=True, grad_dtype=None,
                          stream=None):
    """Gradients of kda_ssm_scan (C entry point ``kda_ssm_scan_backward``) for
    d_out [T, D] (dtype of dt) and d_final_state fp32 [N, D, S] (None: zero).

    ``chunk_states`` are the forward's; when None they are computed here by
    kda_ssm_scan.  u and z may be the int8 codes of kda_act_pack8 with
    ``u_scales`` and ``z_scales``; chunk_states must then be given.  Returns a dict: du,
    ddt, dz, dB, dC (``grad_dtype``, default the dtype of dt), dA, dD, ddt_bias,
    d_init_state (fp32); dz, dD and ddt_bias are None without z, D and dt_bias."""
    if d_out is None:
        raise ValueError("d_out is needed")
    dev, code, N, T, ch, S, ins = _scan_args(u, dt, A, B, C, D, z, dt_bias, cu_seqlens, num_seqs,
                                             softplus, u_scales, z_scales)
    ry = _ROWS.pack(*_rows(d_out, "d_out", dev, dt.dtype, (T, ch)))
    init = _is(init_state, "init_state", dev, _F32, (N, ch, S))
    dfin = _is(d_final_state, "d_final_state", dev, _F32, (N, ch, S))
    gdt = grad_dtype or dt.dtype
    dims = _DIMS.pack(N, T, ch, S, code, _code(gdt, "grad_dtype"))
    if chunk_states is None and T > _kda.CHUNK:
        if u_scales is not None:
            raise ValueError("packed u and z need the forward's chunk_states")
        _, _, chunk_states = kda_ssm_scan(u, dt, A, B, C, D, None, dt_bias, init_state, cu_seqlens,
                                          num_seqs=N, softplus=softplus, return_final_state=False,
                                          return_chunk_states=True, stream=stream)
    cap = 0 if chunk_states is None else chunk_states.shape[0]
    chunks = _is(chunk_states, "chunk_states", dev, _F32, (cap, ch, S))
    with _on(dev, stream):
        def new(shape, dtype=_F32, wanted=True):
            return torch.empty(shape, dtype=dtype, device=dt.device) if wanted else None

        res = dict(du=new((T, ch), gdt), ddt=new((T, ch), gdt), dz=new((T, ch), gdt, z is not None),
                   dB=new((T, S), gdt), dC=new((T, S), gdt), dA=new((ch, S)),
                   dD=new((ch,), wanted=D is not None), ddt_bias=new((ch,), wanted=dt_bias is not None),
                   d_init_state=new((N, ch, S)))
        ws = _workspace("kda_ssm_scan_backward_workspace", dims, dt.device)
        _run("kda_ssm_scan_backward", dev, dims, ins, init, chunks, cap, ry, dfin,
             _GRADS.pack(*(_p(res[n]) for n in _GRAD_NAMES)), ws.data_ptr(), ws.shape[0])
    return res
