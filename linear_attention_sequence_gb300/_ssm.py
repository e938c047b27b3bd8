"""Binding of the state space layer calls and the 8-bit packing (see
``include/kda.h``).  As in the rest of the package: pointers, sizes and checks,
no arithmetic of the method and no fallback."""
from __future__ import annotations

import ctypes

import torch

import linear_attention_sequence_gb300 as _kda

PACK_GROUP = 32   # channels that share a scale (KDA_PACK_GROUP)

_vp, _i32, _i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class _Rows(ctypes.Structure):
    _fields_ = [("data", _vp), ("stride", _i64), ("scales", _vp)]


class _SsmDims(ctypes.Structure):
    _fields_ = [(n, _i32) for n in ("num_seqs", "total_tokens", "channels", "state_size",
                                    "in_dtype", "out_dtype")]


class _Inputs(ctypes.Structure):
    _fields_ = [("u", _Rows), ("dt", _Rows), ("B", _Rows), ("C", _Rows), ("z", _Rows),
                ("A", _vp), ("D", _vp), ("dt_bias", _vp), ("cu_seqlens", _vp),
                ("delta_softplus", _i32)]


class _Grads(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("du", "ddt", "dB", "dC", "dz", "dA", "dD", "ddt_bias",
                                   "d_init_state")]


def declare(L):
    """Argument types of the C entry points."""
    P = ctypes.POINTER
    L.kda_act_pack8.argtypes = [_i32, _i32, _i32, P(_Rows), _vp, _vp, _vp]
    L.kda_ssm_conv.argtypes = [P(_SsmDims), P(_Rows), _vp, _vp, _vp, _vp, _i32, _vp, _vp, _vp]
    L.kda_ssm_conv_backward.argtypes = [P(_SsmDims), P(_Rows), _vp, _vp, _vp, _vp, _i32, P(_Rows),
                                        _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp]
    L.kda_ssm_scan.argtypes = [P(_SsmDims), P(_Inputs), _vp, _vp, _vp, _vp, _i64, _vp]
    L.kda_ssm_step.argtypes = [P(_SsmDims), P(_Inputs), _vp, _vp, _vp]
    L.kda_ssm_scan_backward.argtypes = [P(_SsmDims), P(_Inputs), _vp, _vp, _i64, P(_Rows), _vp,
                                        P(_Grads), _vp, _i64, _vp]
    for name in ("kda_act_pack8", "kda_ssm_conv", "kda_ssm_conv_backward", "kda_ssm_scan",
                 "kda_ssm_step", "kda_ssm_scan_backward"):
        getattr(L, name).restype = ctypes.c_int
    for name in ("kda_ssm_conv_backward_workspace", "kda_ssm_scan_backward_workspace"):
        getattr(L, name).argtypes = [P(_SsmDims)]
        getattr(L, name).restype = _i64


def _p(t):
    return None if t is None else t.data_ptr()


def _is(t, name, device, dtype, shape):
    """A contiguous tensor of this shape on this device (None passes)."""
    if t is None:
        return
    _kda._require(t, name, dtype, len(shape))
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _rows(t, name, device, dtype, shape, scales=None):
    """A [tokens, channels] activation whose rows may lie a stride apart, or its
    int8 codes and scales."""
    if t is None:
        return _Rows(None, 0, None)
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be a CUDA tensor on {device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if scales is not None:
        if t.dtype != torch.int8 or not t.is_contiguous():
            raise ValueError(f"{name} with scales must be contiguous int8 codes")
        _is(scales, f"scales of {name}", device, torch.float32,
            (shape[0], -(-shape[1] // PACK_GROUP)))
        return _Rows(_p(t), shape[1], _p(scales))
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}'s rows must be contiguous")
    stride = t.stride(0) if t.shape[0] > 1 else t.shape[1]
    if stride < t.shape[1]:
        raise ValueError(f"{name}'s rows must not overlap")
    return _Rows(_p(t), stride, None)


def _float(dtype, what):
    if dtype not in _kda._DTYPES:
        raise ValueError(f"{what} must be fp32 or bf16")
    return dtype


def _sequences(cu_seqlens, num_seqs, device):
    if cu_seqlens is None:
        return 1 if num_seqs is None else int(num_seqs)
    _kda._require(cu_seqlens, "cu_seqlens", torch.int32, 1)
    if cu_seqlens.device != device or cu_seqlens.shape[0] < 1:
        raise ValueError(f"cu_seqlens must hold N + 1 entries on {device}")
    return cu_seqlens.shape[0] - 1


def _activation(x, name):
    if x is None or x.dim() != 2 or not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor [tokens, channels]")
    return x.device


class _on:
    """Makes ``device`` current, and ``stream`` where one is given, for a call and for
    what it allocates: PyTorch's allocator gives a block out again only to work
    behind the stream that was current when it was allocated."""

    def __init__(self, device, stream):
        self.device, self.stream, self.inner = device, stream, None

    def __enter__(self):
        if self.stream is not None:
            if self.stream.device != self.device:
                raise ValueError(f"the stream must be on {self.device}")
            self.inner = torch.cuda.stream(self.stream)
        elif torch.cuda.current_device() != self.device.index:
            self.inner = torch.cuda.device(self.device)
        if self.inner is not None:
            self.inner.__enter__()

    def __exit__(self, *exc):
        if self.inner is not None:
            self.inner.__exit__(*exc)


def _run(call, device, *args):
    """The C call on the current stream of ``device``, which is the current device."""
    s = torch.cuda.current_stream(device).cuda_stream
    _kda._check(getattr(_kda.lib(), call)(*args, s), call)


def _workspace(query, dims, device):
    n = getattr(_kda.lib(), query)(ctypes.byref(dims))
    if n < 0:
        raise _kda.KdaError(2, query)
    return torch.empty((n,), dtype=torch.uint8, device=device)


def kda_act_pack8(x, *, codes=None, scales=None, stream=None):
    """An activation x [T, D] (fp32 or bf16, rows may lie a stride apart) in 8
    bits (C entry point ``kda_act_pack8``).  Returns ``(codes, scales)``: int8
    [T, D] and fp32 [T, ceil(D / 32)]; ``codes * scale of the group`` stands for x."""
    dev = _activation(x, "x")
    _float(x.dtype, "x")
    T, D = x.shape
    r = _rows(x, "x", dev, x.dtype, (T, D))
    with _on(dev, stream):
        if codes is None:
            codes = torch.empty((T, D), dtype=torch.int8, device=dev)
        if scales is None:
            scales = torch.empty((T, -(-D // PACK_GROUP)), dtype=torch.float32, device=dev)
        _is(codes, "codes", dev, torch.int8, (T, D))
        _is(scales, "scales", dev, torch.float32, (T, -(-D // PACK_GROUP)))
        _run("kda_act_pack8", dev, T, D, _kda._DTYPES[x.dtype], ctypes.byref(r), _p(codes),
             _p(scales))
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
    dev = _activation(x, "x")
    _float(x.dtype, "x")
    T, D = x.shape
    N = _sequences(cu_seqlens, num_seqs, dev)
    if weight.dim() != 2:
        raise ValueError("weight must be [D, W]")
    W = weight.shape[1]
    r = _rows(x, "x", dev, x.dtype, (T, D))
    _is(weight, "weight", dev, torch.float32, (D, W))
    _is(bias, "bias", dev, torch.float32, (D,))
    _is(conv_state, "conv_state", dev, torch.float32, (N, W - 1, D))
    odt = _float(out_dtype or x.dtype, "out_dtype")
    with _on(dev, stream):
        if out is None:
            out = torch.empty((T, D), dtype=odt, device=dev)
        _is(out, "out", dev, odt, (T, D))
        if conv_state_out is None and return_conv_state:
            conv_state_out = torch.empty((N, W - 1, D), dtype=torch.float32, device=dev)
        _is(conv_state_out, "conv_state_out", dev, torch.float32, (N, W - 1, D))
        dims = _SsmDims(N, T, D, W, _kda._DTYPES[x.dtype], _kda._DTYPES[odt])
        _run("kda_ssm_conv", dev, ctypes.byref(dims), ctypes.byref(r), _p(weight), _p(bias),
             _p(conv_state), _p(cu_seqlens), int(bool(swish)), _p(out), _p(conv_state_out))
    return out, conv_state_out


def kda_ssm_conv_backward(x, weight, d_out, bias=None, cu_seqlens=None, conv_state=None, *,
                          x_scales=None, num_seqs=None, swish=True, d_conv_state_out=None,
                          grad_dtype=None, stream=None):
    """Gradients of kda_ssm_conv (C entry point ``kda_ssm_conv_backward``) for
    d_out [T, D] and d_conv_state_out fp32 [N, W-1, D] (None: zero).  x in the
    dtype of d_out, or the int8 codes of kda_act_pack8 with ``x_scales``.  Returns a
    dict with dx (``grad_dtype``, default the dtype of d_out), dweight, dbias and
    d_conv_state (fp32)."""
    dev = _activation(d_out, "d_out")
    _float(d_out.dtype, "d_out")
    T, D = d_out.shape
    N = _sequences(cu_seqlens, num_seqs, dev)
    if weight.dim() != 2:
        raise ValueError("weight must be [D, W]")
    W = weight.shape[1]
    rx = _rows(x, "x", dev, d_out.dtype, (T, D), x_scales)
    ry = _rows(d_out, "d_out", dev, d_out.dtype, (T, D))
    _is(weight, "weight", dev, torch.float32, (D, W))
    _is(bias, "bias", dev, torch.float32, (D,))
    for t, n in ((conv_state, "conv_state"), (d_conv_state_out, "d_conv_state_out")):
        _is(t, n, dev, torch.float32, (N, W - 1, D))
    gdt = _float(grad_dtype or d_out.dtype, "grad_dtype")
    with _on(dev, stream):
        f32 = dict(dtype=torch.float32, device=dev)
        res = dict(dx=torch.empty((T, D), dtype=gdt, device=dev), dweight=torch.empty((D, W), **f32),
                   dbias=torch.empty((D,), **f32), d_conv_state=torch.empty((N, W - 1, D), **f32))
        dims = _SsmDims(N, T, D, W, _kda._DTYPES[d_out.dtype], _kda._DTYPES[gdt])
        ws = _workspace("kda_ssm_conv_backward_workspace", dims, dev)
        _run("kda_ssm_conv_backward", dev, ctypes.byref(dims), ctypes.byref(rx), _p(weight),
             _p(bias), _p(conv_state), _p(cu_seqlens), int(bool(swish)), ctypes.byref(ry),
             _p(d_conv_state_out), _p(res["dx"]), _p(res["dweight"]), _p(res["dbias"]),
             _p(res["d_conv_state"]), _p(ws), ws.numel())
    return res


def _scan_args(u, dt, A, B, C, D, z, dt_bias, cu_seqlens, num_seqs, softplus, dtype,
               u_scales=None, z_scales=None):
    dev = _activation(dt, "dt")
    _float(dtype, "dt, B and C")
    T, ch = dt.shape
    if A.dim() != 2:
        raise ValueError("A must be [D, S]")
    S = A.shape[1]
    N = _sequences(cu_seqlens, num_seqs, dev)
    if z is not None and (u_scales is None) != (z_scales is None):
        raise ValueError("u and z must both be packed or neither")
    ins = _Inputs(_rows(u, "u", dev, dtype, (T, ch), u_scales), _rows(dt, "dt", dev, dtype, (T, ch)),
                  _rows(B, "B", dev, dtype, (T, S)), _rows(C, "C", dev, dtype, (T, S)),
                  _rows(z, "z", dev, dtype, (T, ch), z_scales), _p(A), _p(D), _p(dt_bias),
                  _p(cu_seqlens), int(bool(softplus)))
    _is(A, "A", dev, torch.float32, (ch, S))
    _is(D, "D", dev, torch.float32, (ch,))
    _is(dt_bias, "dt_bias", dev, torch.float32, (ch,))
    return dev, N, T, ch, S, ins


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
    dev, N, T, ch, S, ins = _scan_args(u, dt, A, B, C, D, z, dt_bias, cu_seqlens, num_seqs,
                                       softplus, dt.dtype)
    _is(init_state, "init_state", dev, torch.float32, (N, ch, S))
    odt = _float(out_dtype or dt.dtype, "out_dtype")
    with _on(dev, stream):
        if out is None:
            out = torch.empty((T, ch), dtype=odt, device=dev)
        _is(out, "out", dev, odt, (T, ch))
        if final_state is None and return_final_state:
            final_state = torch.empty((N, ch, S), dtype=torch.float32, device=dev)
        _is(final_state, "final_state", dev, torch.float32, (N, ch, S))
        if chunk_states is None and return_chunk_states:
            rows = _kda.checkpoint_count(T, _kda.CHUNK, cu_seqlens, N)
            chunk_states = torch.empty((rows, ch, S), dtype=torch.float32, device=dev)
        if chunk_states is not None:
            _is(chunk_states, "chunk_states", dev, torch.float32, (chunk_states.shape[0], ch, S))
        dims = _SsmDims(N, T, ch, S, _kda._DTYPES[dt.dtype], _kda._DTYPES[odt])
        some = chunk_states is not None and chunk_states.numel() > 0
        _run("kda_ssm_scan", dev, ctypes.byref(dims), ctypes.byref(ins), _p(init_state),
             _p(out), _p(final_state), _p(chunk_states) if some else None,
             chunk_states.shape[0] if some else 0)
    return (out, final_state) if chunk_states is None else (out, final_state, chunk_states)


def kda_ssm_step(u, dt, A, B, C, state, D=None, z=None, dt_bias=None, *, softplus=True, out=None,
                 out_dtype=None, stream=None):
    """One token of the scan for N sequences (C entry point ``kda_ssm_step``): u,
    dt, z [N, D], B, C [N, S], state fp32 [N, D, S] updated in place.  Returns out
    [N, D]."""
    N = dt.shape[0]
    dev, _, _, ch, S, ins = _scan_args(u, dt, A, B, C, D, z, dt_bias, None, N, softplus, dt.dtype)
    if state is None:
        raise ValueError("state is needed")
    _is(state, "state", dev, torch.float32, (N, ch, S))
    odt = _float(out_dtype or dt.dtype, "out_dtype")
    with _on(dev, stream):
        if out is None:
            out = torch.empty((N, ch), dtype=odt, device=dev)
        _is(out, "out", dev, odt, (N, ch))
        dims = _SsmDims(N, N, ch, S, _kda._DTYPES[dt.dtype], _kda._DTYPES[odt])
        _run("kda_ssm_step", dev, ctypes.byref(dims), ctypes.byref(ins), _p(state), _p(out))
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
    dev, N, T, ch, S, ins = _scan_args(u, dt, A, B, C, D, z, dt_bias, cu_seqlens, num_seqs,
                                       softplus, dt.dtype, u_scales, z_scales)
    ry = _rows(d_out, "d_out", dev, dt.dtype, (T, ch))
    if d_out is None:
        raise ValueError("d_out is needed")
    for t, n in ((init_state, "init_state"), (d_final_state, "d_final_state")):
        _is(t, n, dev, torch.float32, (N, ch, S))
    with _on(dev, stream):
        if chunk_states is None and T > _kda.CHUNK:
            if u_scales is not None:
                raise ValueError("packed u and z need the forward's chunk_states")
            _, _, chunk_states = kda_ssm_scan(u, dt, A, B, C, D, None, dt_bias, init_state, cu_seqlens,
                                              num_seqs=N, softplus=softplus, return_final_state=False,
                                              return_chunk_states=True, stream=stream)
        if chunk_states is not None:
            _is(chunk_states, "chunk_states", dev, torch.float32, (chunk_states.shape[0], ch, S))
        gdt = _float(grad_dtype or dt.dtype, "grad_dtype")

        def new(shape, dtype=torch.float32, wanted=True):
            return torch.empty(shape, dtype=dtype, device=dev) if wanted else None

        res = dict(du=new((T, ch), gdt), ddt=new((T, ch), gdt), dz=new((T, ch), gdt, z is not None),
                   dB=new((T, S), gdt), dC=new((T, S), gdt), dA=new((ch, S)),
                   dD=new((ch,), wanted=D is not None), ddt_bias=new((ch,), wanted=dt_bias is not None),
                   d_init_state=new((N, ch, S)))
        grads = _Grads(*(_p(res[n]) for n, _ in _Grads._fields_))
        dims = _SsmDims(N, T, ch, S, _kda._DTYPES[dt.dtype], _kda._DTYPES[gdt])
        ws = _workspace("kda_ssm_scan_backward_workspace", dims, dev)
        some = chunk_states is not None and chunk_states.numel() > 0
        _run("kda_ssm_scan_backward", dev, ctypes.byref(dims), ctypes.byref(ins),
             _p(init_state), _p(chunk_states) if some else None,
             chunk_states.shape[0] if some else 0, ctypes.byref(ry), _p(d_final_state),
             ctypes.byref(grads), _p(ws), ws.numel())
    return res
