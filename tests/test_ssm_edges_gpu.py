"""GPU tests of the state space layer calls at their edges: batches without sequences,
states in place, calls close behind one another.  Bounds as in test_ssm_gpu.py."""
import pytest
import torch

import linear_attention_sequence_gb300 as kda
from linear_attention_sequence_gb300 import _ssm
import ssm_reference as ref
from test_ssm_gpu import BF16, DEV, F32, bwd, check, conv_inputs, cu_of, fwd, h, scan_inputs

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ rows, but no sequence

@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("first", [0, 7, 200, -3])
def test_conv_of_rows_without_sequences(first, dtype, packed):
    """A padded buffer whose batch is empty: no row is written, and the parameters'
    gradients are 0."""
    T, D, W = 200, 40, 4
    x = conv_inputs(T, D, W, 0, dtype, 501)
    cu = torch.tensor([first], dtype=torch.int32, device=DEV)
    out = torch.full((T, D), 7.0, device=DEV, dtype=dtype)
    _, last = kda.kda_ssm_conv(x["x"], x["weight"], x["bias"], cu, x["state"], out=out)
    assert last.shape == (0, W - 1, D) and bool((out == 7).all())
    xi, sc = kda.kda_act_pack8(x["x"]) if packed else (x["x"], None)
    g = kda.kda_ssm_conv_backward(xi, x["weight"], x["d_out"], x["bias"], cu, x["state"], x_scales=sc,
                                  d_conv_state_out=x["d_state"])
    assert not g["dweight"].any() and not g["dbias"].any() and g["d_conv_state"].shape == (0, W - 1, D)
    # the C call, for the rows of dx
    dx, dw = torch.full((T, D), 7.0, device=DEV, dtype=dtype), torch.full((D, W), 7.0, device=DEV)
    rows = lambda t: _ssm._ROWS.pack(t.data_ptr(), t.stride(0), 0)  # noqa: E731
    dims = _ssm._DIMS.pack(0, T, D, W, *[_ssm._code(dtype, "x")] * 2)
    _ssm._run("kda_ssm_conv_backward", torch.cuda.current_device(), dims, rows(x["x"]), x["weight"].data_ptr(), 0, 0,
              cu.data_ptr(), 1, rows(x["d_out"]), 0, dx.data_ptr(), dw.data_ptr(), 0, 0, 0, 0)
    assert bool((dx == 7).all()) and not dw.any()
    assert kda.kda_get_last_device_error() == 0


@pytest.fixture
def nan_workspaces(monkeypatch):
    """Every workspace holds NaN before the call."""
    plain = _ssm._workspace
    monkeypatch.setattr(_ssm, "_workspace", lambda query, dims, device: plain(query, dims, device).fill_(255))


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("T,D", [(1, 40), (32, 40), (200, 40), (2000, 40), (64, 5000)])
def test_scan_of_rows_without_sequences(T, D, packed, nan_workspaces):
    """The same of the scan: the gradients of A, D and dt_bias are sums over nothing."""
    S = 16
    x = scan_inputs(T, D, S, 0, BF16, 502)
    cu = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.full((T, D), 7.0, device=DEV, dtype=BF16)
    _, fin, chunks = fwd(x, cu_seqlens=cu, out=out, chunk_states=torch.empty(3, D, S, device=DEV))
    assert fin.shape == (0, D, S) and bool((out == 7).all())
    kw = {}
    if packed:
        (x["u"], kw["u_scales"]), (x["z"], kw["z_scales"]) = kda.kda_act_pack8(x["u"]), kda.kda_act_pack8(x["z"])
    g = bwd(x, cu_seqlens=cu, chunk_states=chunks, **kw)
    for n in ("dA", "dD", "ddt_bias"):
        assert bool((g[n] == 0).all()), n
    assert g["d_init_state"].shape == (0, D, S)
    # the C call, for the rows of the others
    gr = {n: torch.full((T, S if n in ("dB", "dC") else D), 7.0, device=DEV, dtype=BF16) for n in ("du", "ddt", "dB", "dC", "dz")}
    dA = torch.full((D, S), 7.0, device=DEV)
    dims = _ssm._DIMS.pack(0, T, D, S, 1, 1)
    ins = _ssm._scan_args(x["u"], x["dt"], x["A"], x["B"], x["C"], x["D"], x["z"], x["dt_bias"], cu, None, True,
                          kw.get("u_scales"), kw.get("z_scales"))[-1]
    ws = _ssm._workspace("kda_ssm_scan_backward_workspace", dims, DEV)
    _ssm._run("kda_ssm_scan_backward", torch.cuda.current_device(), dims, ins, 0, 0, 0,
              _ssm._ROWS.pack(x["d_out"].data_ptr(), D, 0), 0,
              _ssm._GRADS.pack(*(gr[n].data_ptr() for n in gr), dA.data_ptr(), 0, 0, 0), ws.data_ptr(), ws.shape[0])
    assert bool((dA == 0).all()) and all(bool((t == 7).all()) for t in gr.values())
    assert kda.kda_get_last_device_error() == 0


# ------------------------------------------------------------------ states in place

def misaligned(t):
    """The same values one fp32 element past an allocation's start."""
    v = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)[1:].view(t.shape)
    return v.copy_(t)


@pytest.mark.parametrize("place", [torch.clone, misaligned])
@pytest.mark.parametrize("dtype,D,S", [(F32, 40, 16), (BF16, 72, 5), (F32, 24, 64), (BF16, 520, 16)])
@pytest.mark.parametrize("N,lens", [(1, [257]), (3, [736] * 3), (1, [1500]), (None, [700]), (None, [257, 0, 900, 5, 1]),
                                    (None, [1] * 290 + [700, 0, 333])])
def test_scan_of_cut_sequences_in_place(N, lens, dtype, D, S, place, nan_workspaces):
    """The final state in the initial state's place, of sequences that are cut into parts
    (257 tokens: parts of 32, the last of one token): the bits of the call with two buffers,
    every time."""
    x = scan_inputs(sum(lens), D, S, len(lens), dtype, 600 + sum(lens) + D)
    kw = dict(num_seqs=N) if N else dict(cu_seqlens=cu_of(lens))
    x["state"] = start = place(x["state"])
    out, fin, chunks = fwd(x, return_chunk_states=True, out_dtype=F32, **kw)
    w = ref.scan(h(x), lens)
    for n, t in (("out", out), ("final", fin), ("chunks", chunks)):
        check(n, t, w[n])
    states = [place(start) for _ in range(10)]
    outs = [fwd(dict(x, state=st), out_dtype=F32, final_state=st, **kw)[0] for st in states]
    for st, o in zip(states, outs):
        assert torch.equal(st, fin) and torch.equal(o, out)


def test_long_prompt_in_pieces_in_place():
    """A prompt given in pieces that are each cut, with one buffer for its state."""
    T, D, S = 1800, 40, 16
    x = scan_inputs(T, D, S, 1, F32, 611)
    w = ref.scan(h(x), [T])
    st, outs = x["state"].clone(), []
    for a, b in ((0, 600), (600, 601), (601, 1225), (1225, T)):
        part = {k: (v[a:b] if k in ("u", "dt", "B", "C", "z") else v) for k, v in x.items()}
        outs.append(fwd(dict(part, state=st), final_state=st)[0])
    check("out", torch.cat(outs), w["out"])
    check("state", st, w["final"])


def test_scan_in_place_in_graphs_and_on_a_stream():
    """A cut scan in place, captured and replayed, two graphs in turn on one state, and on a
    stream of its own: each call goes on from the state that the one before left."""
    lens, D, S = [700, 0, 257], 40, 16
    cu, N = cu_of(lens), len(lens)
    sets = [scan_inputs(sum(lens), D, S, N, BF16, seed) for seed in (631, 632)]
    start, want = sets[0]["state"].clone(), []
    st = start.clone()
    for i in range(6):
        out, st = fwd(dict(sets[i % 2], state=st), cu_seqlens=cu)
        want.append((out, st))
    here = start.clone()
    call = lambda x, **kw: fwd(dict(x, state=here), cu_seqlens=cu, final_state=here, **kw)[0]  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [call(sets[i % 2], stream=side) for i in range(6)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, (w, _) in zip(outs, want)) and torch.equal(here, want[-1][1])
    graphs, outs = [], []
    for x in sets:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(call(x))
    here.copy_(start)
    for i, (o, f) in enumerate(want):
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i % 2], o) and torch.equal(here, f)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("N,D", [(1, 1), (3, 70), (256, 2048), (5, 12288)])
def test_conv_tokens_in_place(N, D, W, dtype):
    """Tokens one at a time with the state moved in its own buffer: the bits of calls with
    two buffers, over many in a row."""
    T = 9
    x = conv_inputs(N * T, D, W, N, dtype, 615)
    rows = x["x"].view(T, N, D)
    one, here = x["state"], x["state"].clone()
    call = lambda t, st, to: kda.kda_ssm_conv(rows[t], x["weight"], x["bias"], conv_state=st, conv_state_out=to, num_seqs=N)  # noqa: E731
    outs = [call(t, here, here)[0] for t in range(T)]
    for t in range(T):
        y, one = call(t, one, torch.empty_like(one))
        assert torch.equal(y, outs[t])
    assert torch.equal(one, here)
    line = torch.cat([x["state"].transpose(0, 1).double(), rows.double()])          # [W - 1 + T, N, D]
    assert torch.equal(here.double(), line[T:].transpose(0, 1))
    c = x["bias"].double() + sum(line[k:k + T] * x["weight"][:, k].double() for k in range(W))
    check("out", torch.stack(outs), (c / (1 + torch.exp(-c))).cpu())


# ------------------------------------------------------------------ calls close behind one another

@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("T,D,S", [(600, 1032, 16), (2048, 264, 24), (333, 40, 8)])
def test_gradients_behind_one_another_share_a_workspace(T, D, S, packed, monkeypatch):
    """Calls on a stream with one workspace, of two sets of inputs in turn and nothing
    between them: each gives the bits of a call alone, whose kernels nobody's were in front
    of.  What a kernel adds up is what the one before it in its own call wrote."""
    sets = []
    for seed in (621, 622):
        x, c = scan_inputs(T, D, S, 1, BF16, seed), conv_inputs(T, D, 4, 1, BF16, seed)
        chunks, kw, cx = fwd(x, return_chunk_states=True)[2], {}, {}
        if packed:
            (x["u"], kw["u_scales"]), (x["z"], kw["z_scales"]) = kda.kda_act_pack8(x["u"]), kda.kda_act_pack8(x["z"])
            c["x"], cx["x_scales"] = kda.kda_act_pack8(c["x"])
        sets.append((x, chunks, kw, c, cx))

    def both(s):
        x, chunks, kw, c, cx = s
        return bwd(x, chunk_states=chunks, **kw), kda.kda_ssm_conv_backward(
            c["x"], c["weight"], c["d_out"], c["bias"], None, c["state"], d_conv_state_out=c["d_state"], **cx)

    want = []
    for s in sets:
        torch.cuda.synchronize()
        want.append(both(s))
        torch.cuda.synchronize()
    plain, held = _ssm._workspace, {}

    def shared(query, dims, device):
        if (query, dims) not in held:
            held[query, dims] = plain(query, dims, device).fill_(255)
        return held[query, dims]

    monkeypatch.setattr(_ssm, "_workspace", shared)
    got = [both(sets[i % 2]) for i in range(16)]
    for i, pair in enumerate(got):
        for g, w in zip(pair, want[i % 2]):
            for n in w:
                assert torch.equal(g[n], w[n]), (i, n)
