"""Host-side checks of the state space layer calls (no GPU): the C entry points
refuse bad arguments before anything reaches the device, and the binding refuses
what it can see.  Every pointer here is made up and never read."""
import ctypes

import pytest
import torch

import linear_attention_sequence_gb300 as kda
from linear_attention_sequence_gb300 import _build



class _Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride", ctypes.c_int64), ("scales", ctypes.c_void_p)]


class _SsmDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("num_seqs", "total_tokens", "channels", "state_size",
                                              "in_dtype", "out_dtype")]


class _Inputs(ctypes.Structure):
    _fields_ = [(n, _Rows) for n in ("u", "dt", "B", "C", "z")] + [
        (n, ctypes.c_void_p) for n in ("A", "D", "dt_bias", "cu_seqlens")] + [("delta_softplus", ctypes.c_int32)]


class _Grads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("du", "ddt", "dB", "dC", "dz", "dA", "dD", "ddt_bias", "d_init_state")]


INVALID, UNSUPPORTED = 1, 2
BF16 = 1
R = ctypes.byref


@pytest.fixture(scope="module")
def L():
    _build.build()
    return kda.lib()


def at(k):
    """A made-up device address, 16 MB from the next."""
    return 0x10000000 + (k << 24)


def dims(**kw):
    d = dict(num_seqs=2, total_tokens=64, channels=40, state_size=16, in_dtype=BF16, out_dtype=BF16)
    d.update(kw)
    return _SsmDims(*(d[n] for n, _ in _SsmDims._fields_))


def rows(k, width, **kw):
    r = dict(data=at(k), stride=width, scales=None)
    r.update(kw)
    return _Rows(r["data"], r["stride"], r["scales"])


def inputs(S=16, **kw):
    i = dict(u=rows(1, 40), dt=rows(2, 40), B=rows(3, S), C=rows(4, S), z=rows(5, 40), A=at(6), D=at(7),
             dt_bias=at(8), cu_seqlens=None, delta_softplus=1)
    i.update(kw)
    return _Inputs(*(i[n] for n, _ in _Inputs._fields_))


BAD_DIMS = [(dict(num_seqs=-1), INVALID), (dict(total_tokens=-1), INVALID), (dict(channels=0), INVALID),
            (dict(state_size=0), INVALID), (dict(in_dtype=5), INVALID), (dict(out_dtype=-1), INVALID),
            (dict(state_size=65), UNSUPPORTED), (dict(num_seqs=3), INVALID), (dict(num_seqs=0), INVALID),
            (dict(total_tokens=1 << 30, channels=1 << 20), UNSUPPORTED)]

BAD_INPUTS = [dict(u=rows(1, 40, data=None)), dict(dt=rows(2, 40, data=None)), dict(B=rows(3, 16, data=None)),
              dict(C=rows(4, 16, data=None)), dict(A=None), dict(A=at(6) + 2), dict(u=rows(1, 40, stride=39)),
              dict(z=rows(5, 40, stride=-40)), dict(u=rows(1, 40, data=at(1) + 1)), dict(D=at(7) + 1),
              dict(dt_bias=at(8) + 2), dict(cu_seqlens=at(9) + 2), dict(u=rows(1, 40, stride=1 << 41)),
              dict(dt=rows(2, 40, scales=at(20))), dict(B=rows(3, 16, scales=at(20)))]


def scan(L, d, i, init=None, out=at(30), fin=at(31), chunks=None, cap=0, ws=at(60), size=1 << 24):
    return L.kda_ssm_scan(R(d) if d else None, R(i) if i else None, init, out, fin, chunks, cap, ws, size, None)


@pytest.mark.parametrize("over,want", BAD_DIMS)
def test_dims_are_refused(L, over, want):
    d = dims(**over)
    i = inputs(S=d.state_size if d.state_size > 0 else 16)
    assert scan(L, d, i) == want
    assert backward(L, d, i) == want
    if want == INVALID and "num_seqs" not in over:
        assert L.kda_ssm_step(R(d), R(i), at(30), at(31), None) == want
    if "state_size" not in over:
        d.state_size = 4
        assert conv(L, d) == want and conv_backward(L, d) == want


@pytest.mark.parametrize("over", BAD_INPUTS)
def test_scan_inputs_are_refused(L, over):
    assert scan(L, dims(), inputs(**over)) == INVALID
    assert backward(L, dims(), inputs(**over)) == INVALID
    assert L.kda_ssm_step(R(dims(num_seqs=64)), R(inputs(**over)), at(30), at(31), None) == INVALID


@pytest.mark.parametrize("over", [
    dict(out=None), dict(out=at(30) + 1), dict(init=at(33) + 2), dict(fin=at(31) + 1), dict(cap=-1), dict(cap=3),
    dict(chunks=at(32) + 2, cap=3),
    dict(out=at(1)), dict(out=at(5) + 64 * 40 * 2 - 2), dict(fin=at(6)), dict(init=at(31) + 64), dict(out=at(31)),
    dict(chunks=at(31), cap=2), dict(chunks=at(33), cap=2, init=at(33))])
def test_scan_is_refused(L, over):
    assert scan(L, dims(), inputs(), **over) == INVALID
    assert scan(L, None, inputs()) == INVALID and scan(L, dims(), None) == INVALID


def test_scan_workspace(L):
    """A long sequence of few channels needs one; the call refuses a smaller or a
    misplaced one."""
    d = dims(num_seqs=1, total_tokens=4096)
    need = L.kda_ssm_scan_workspace(R(d))
    assert need > 0
    assert scan(L, d, inputs(), size=need - 1) == INVALID
    assert scan(L, d, inputs(), ws=None) == INVALID
    assert scan(L, d, inputs(), ws=at(60) + 8) == INVALID
    assert scan(L, d, inputs(), ws=at(31)) == INVALID
    assert scan(L, d, inputs(), ws=at(2)) == INVALID
    assert L.kda_ssm_scan_workspace(R(dims(state_size=65))) == -1


def test_scan_refuses_codes(L):
    """Packed u and z are for the gradients only."""
    i = inputs(u=rows(1, 40, scales=at(20)), z=rows(5, 40, scales=at(21)))
    assert scan(L, dims(), i) == INVALID


def test_step_is_refused(L):
    d, i = dims(num_seqs=64), inputs()
    call = lambda d, i, st=at(31), out=at(30): L.kda_ssm_step(R(d), R(i), st, out, None)  # noqa: E731
    assert call(dims(), i) == INVALID                             # one token a sequence
    assert call(d, inputs(cu_seqlens=at(9))) == INVALID
    assert call(d, i, st=None) == INVALID and call(d, i, out=None) == INVALID
    assert call(d, i, st=at(1)) == INVALID and call(d, i, out=at(31) + 128) == INVALID
    assert call(d, i, st=at(31) + 1) == INVALID


def grads(**kw):
    g = dict(du=at(40), ddt=at(41), dB=at(42), dC=at(43), dz=at(44), dA=at(45), dD=at(46), ddt_bias=at(47), d_init_state=at(48))
    g.update(kw)
    return _Grads(*(g[n] for n, _ in _Grads._fields_))


def backward(L, d, i, init=None, chunks=at(32), cap=2, y=None, fin=None, g=None, ws=at(60), size=None):
    y = rows(10, 40) if y is None else y
    g = grads() if g is None else g
    size = max(0, L.kda_ssm_scan_backward_workspace(R(d))) if size is None else size
    return L.kda_ssm_scan_backward(R(d), R(i), init, chunks, cap, R(y), fin, R(g), ws, size, None)


@pytest.mark.parametrize("over", [
    dict(cap=-1), dict(chunks=None, cap=2), dict(y=rows(10, 40, data=None)), dict(y=rows(10, 40, stride=8)),
    dict(y=rows(10, 40, scales=at(11))), dict(ws=None), dict(ws=at(60) + 8), dict(size=64), dict(ws=at(32)),
    dict(fin=at(33) + 2), dict(g=grads(du=None)), dict(g=grads(dz=None)), dict(g=grads(dA=None)),
    dict(g=grads(dB=at(42) + 1)), dict(g=grads(du=at(1))), dict(g=grads(dA=at(45) + 2)), dict(g=grads(dz=at(40))),
    dict(g=grads(d_init_state=at(32))), dict(g=grads(dC=at(10)))])
def test_scan_backward_is_refused(L, over):
    assert backward(L, dims(), inputs(), **over) == INVALID


def test_scan_backward_refuses_missing_chunk_states(L):
    assert backward(L, dims(num_seqs=1), inputs(), cap=0, chunks=None) == INVALID
    assert backward(L, dims(num_seqs=2, total_tokens=192), inputs(), cap=4) == INVALID   # 5 are needed


def test_scan_backward_refuses_half_packed(L):
    assert backward(L, dims(), inputs(u=rows(1, 40, scales=at(20)))) == INVALID
    assert backward(L, dims(), inputs(z=rows(5, 40, scales=at(21)))) == INVALID
    assert backward(L, dims(), inputs(u=rows(1, 40, scales=at(20), stride=48), z=rows(5, 40, scales=at(21)))) == INVALID


def conv(L, d, x=None, w=at(2), b=at(3), cin=at(4), cu=None, out=at(30), cout=at(31)):
    x = rows(1, 40) if x is None else x
    return L.kda_ssm_conv(R(d), R(x), w, b, cin, cu, 1, out, cout, None)


def conv_backward(L, d, x=None, w=at(2), b=at(3), cin=at(4), cu=None, y=None, dco=at(5), dx=at(40), dw=at(41), db=at(42),
                  dcin=at(43), ws=at(60), size=1 << 20):
    x = rows(1, 40) if x is None else x
    y = rows(10, 40) if y is None else y
    return L.kda_ssm_conv_backward(R(d), R(x), w, b, cin, cu, 1, R(y), dco, dx, dw, db, dcin, ws, size, None)


@pytest.mark.parametrize("over", [
    dict(x=rows(1, 40, data=None)), dict(x=rows(1, 40, stride=39)), dict(x=rows(1, 40, scales=at(20))), dict(w=None),
    dict(w=at(2) + 2), dict(b=at(3) + 1), dict(cin=at(4) + 2), dict(cu=at(9) + 1), dict(out=None), dict(out=at(30) + 1),
    dict(out=at(1)), dict(cout=at(4) + 4), dict(cout=at(30)), dict(cout=at(2))])
def test_conv_is_refused(L, over):
    assert conv(L, dims(state_size=4), **over) == INVALID


def test_conv_taps(L):
    assert conv(L, dims(state_size=1)) == UNSUPPORTED
    assert conv(L, dims(state_size=5)) == UNSUPPORTED
    assert L.kda_ssm_conv_backward_workspace(R(dims(state_size=5))) == -1
    assert L.kda_ssm_scan_backward_workspace(R(dims(state_size=65))) == -1


@pytest.mark.parametrize("over", [
    dict(x=rows(1, 40, data=None)), dict(y=rows(10, 40, data=None)), dict(y=rows(10, 40, scales=at(20))), dict(w=None),
    dict(dx=None), dict(dw=None), dict(dx=at(1)), dict(dw=at(2)), dict(db=at(41)), dict(dcin=at(4)), dict(dcin=at(5)),
    dict(ws=None), dict(size=16), dict(ws=at(60) + 4), dict(ws=at(10)), dict(dx=at(40) + 1), dict(dcin=at(43) + 2),
    dict(x=rows(1, 40, scales=at(20), stride=64)), dict(x=rows(1, 40, scales=at(20) + 2))])
def test_conv_backward_is_refused(L, over):
    assert conv_backward(L, dims(state_size=4), **over) == INVALID


@pytest.mark.parametrize("n,D,dt,x,codes,scales,want", [
    (-1, 40, BF16, rows(1, 40), at(2), at(3), INVALID), (4, 0, BF16, rows(1, 40), at(2), at(3), INVALID),
    (4, 40, 9, rows(1, 40), at(2), at(3), INVALID), (4, 40, BF16, rows(1, 40, data=None), at(2), at(3), INVALID),
    (4, 40, BF16, rows(1, 39), at(2), at(3), INVALID), (4, 40, BF16, rows(1, 40), None, at(3), INVALID),
    (4, 40, BF16, rows(1, 40), at(2), None, INVALID), (4, 40, BF16, rows(1, 40), at(2), at(3) + 1, INVALID),
    (4, 40, BF16, rows(1, 40), at(1), at(3), INVALID), (4, 40, BF16, rows(1, 40), at(2), at(2), INVALID),
    (4, 40, BF16, rows(1, 40, data=at(1) + 1), at(2), at(3), INVALID),
    (4, 40, BF16, rows(1, 40, scales=at(5)), at(2), at(3), INVALID)])
def test_pack8_is_refused(L, n, D, dt, x, codes, scales, want):
    assert L.kda_act_pack8(n, D, dt, R(x), codes, scales, None) == want


def test_nothing_to_do_launches_nothing(L):
    """No rows, or no sequences, is fine without a device."""
    assert L.kda_act_pack8(0, 40, BF16, None, None, None, None) == 0
    d = dims(num_seqs=0, total_tokens=0)
    assert scan(L, d, inputs(), out=None, fin=None) == 0
    d.state_size = 4
    assert conv(L, d, out=None, cout=None) == 0


def test_binding_packs_the_structures():
    """The binding's byte layouts are those of the C structures."""
    from linear_attention_sequence_gb300 import _ssm
    for packer, struct in ((_ssm._ROWS, _Rows), (_ssm._DIMS, _SsmDims), (_ssm._INPUTS, _Inputs), (_ssm._GRADS, _Grads)):
        assert packer.size == ctypes.sizeof(struct)
    i = inputs(cu_seqlens=at(9))
    v = [x for n in ("u", "dt", "B", "C", "z") for x in (getattr(i, n).data, getattr(i, n).stride, 0)]
    assert _ssm._INPUTS.pack(*v, i.A, i.D, i.dt_bias, i.cu_seqlens, 1) == bytes(i)


def test_binding_refuses():
    t = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_act_pack8(t)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_ssm_conv(t, torch.zeros(8, 4))
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_ssm_scan(t, t, torch.zeros(8, 16), torch.zeros(4, 16), torch.zeros(4, 16))
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_ssm_conv_backward(t, torch.zeros(8, 4), t)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_ssm_step(t, t, torch.zeros(8, 16), torch.zeros(4, 16), torch.zeros(4, 16), torch.zeros(4, 8, 16))
