"""GPU tests of the state space layer calls and the 8-bit packing against plain
implementations in 64 bits, token by token on the CPU.

Bounds.  The kernels compute in fp32 with fast exponentials (relative error
2^-22 each).  A state is a sum of products with at most a few thousand decay
factors, each of which carries the rounding of its argument (|Delta A| 2^-23) and of the
exponential: errors of the factors in one product add up, but a term whose product
has k factors is weighed by their product, so with k factors e^-x the relative
error k 2^-22 counts e^{-kx}: at most 2^-22 / (e x), and with the smallest x of these
inputs, 1e-3, 9e-5 of a term in the worst case that all errors agree in sign, and
its square root over the count otherwise.  An fp32 result is therefore held to 1e-4 of
its tensor's rms elementwise and to 1e-5 in the 2-norm, a bf16 result to half a bf16
step (2^-9 of the value between powers of two, at most 2^-8) more.  Codes, scales and
convolution states are exact."""
import numpy as np
import pytest
import torch

import linear_attention_sequence_gb300 as kda
import ssm_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
LENS = [37, 0, 5, 130, 1, 2, 64, 33]


def cu_of(lens, lead=0):
    return torch.tensor(lead + np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=DEV)


def check(name, got, want):
    """`got` a tensor of the GPU, `want` float64 on the CPU."""
    g, w = got.detach().double().cpu(), want
    assert g.shape == w.shape, name
    if not w.numel():
        return
    rms = float(w.square().mean().sqrt())
    step = torch.finfo(got.dtype).eps / 2 if got.dtype == BF16 else 0.0
    err = (g - w).abs()
    lim = 1e-4 * rms + (1e-5 + step) * w.abs()
    assert bool((err <= lim).all()), f"{name}: {float((err - lim).max()):.3e} over, rms {rms:.3e}"
    norm = float(w.norm())
    assert float((g - w).norm()) <= (1e-5 + step) * norm + 1e-30, f"{name}: 2-norm {float((g - w).norm()) / norm:.3e}"


def rnd(gen, *shape, std=1.0, dtype=F32):
    return (torch.randn(shape, generator=gen) * std).to(dtype).to(DEV)


def scan_inputs(T, D, S, N, dtype, seed, gated=True, stride=0):
    gen = torch.Generator().manual_seed(seed)
    x = {}
    for n, w in (("u", D), ("dt", D), ("B", S), ("C", S), ("z", D), ("d_out", D)):
        t = rnd(gen, T, w + stride, std=0.5 if n == "dt" else 1.0, dtype=dtype)
        x[n] = t[:, stride // 2:stride // 2 + w] if stride else t
    if not gated:
        x["z"] = None
    step = torch.exp(torch.rand(D, generator=gen) * np.log(100.0) + np.log(1e-3))
    x["dt_bias"] = (step + torch.log(-torch.expm1(-step))).to(DEV)
    x["A"] = (-torch.arange(1, S + 1).float() * torch.exp(0.1 * torch.randn(D, S, generator=gen))).to(DEV)
    x["D"] = rnd(gen, D) + 1
    x["state"] = rnd(gen, N, D, S, std=0.3)
    x["d_final"] = rnd(gen, N, D, S)
    return x


def fwd(x, **kw):
    return kda.kda_ssm_scan(x["u"], x["dt"], x["A"], x["B"], x["C"], D=x["D"], z=x["z"],
                            dt_bias=x["dt_bias"], init_state=x["state"], **kw)


def bwd(x, **kw):
    args = dict(D=x["D"], z=x["z"], dt_bias=x["dt_bias"], init_state=x["state"])
    args.update(kw)
    return kda.kda_ssm_scan_backward(x["u"], x["dt"], x["A"], x["B"], x["C"], x["d_out"], x["d_final"], **args)


def h(x):
    return {k: (v.detach().double().cpu() if v is not None else None) for k, v in x.items()}


# ------------------------------------------------------------------ packing

@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,D,stride", [(1, 1, 0), (3, 31, 0), (5, 33, 0), (70, 96, 32), (33, 1000, 5), (257, 256, 0)])
def test_pack8(T, D, stride, dtype):
    gen = torch.Generator().manual_seed(T + D)
    full = (torch.randn(T, D + stride, generator=gen) * torch.exp(2 * torch.randn(D + stride, generator=gen))).to(dtype)
    full[0] = 0
    x = full.to(DEV)[:, :D]
    codes, scales = kda.kda_act_pack8(x)
    want_codes, want_scales = ref.pack8(full[:, :D])
    assert torch.equal(scales.cpu(), want_scales)
    assert torch.equal(codes.cpu(), want_codes)
    # half a scale, and the rounding of x * (127 / m), of 127 / m and of code * scale
    back = codes.cpu().double() * scales.cpu().double().repeat_interleave(32, 1)[:, :D]
    lim = scales.cpu().double().repeat_interleave(32, 1)[:, :D] * (0.5 + 127 * 3 * 2.0 ** -24)
    assert bool(((back - full[:, :D].double()).abs() <= lim).all())


def test_pack8_special_values():
    x = torch.ones(4, 96, device=DEV)
    x[0, 3], x[1, 40], x[2, 70] = float("inf"), float("nan"), float("-inf")
    x[3, :32] = 1e-38
    codes, scales = kda.kda_act_pack8(x)
    bad = torch.zeros(4, 3, dtype=torch.bool, device=DEV)
    bad[0, 0] = bad[1, 1] = bad[2, 2] = True
    assert torch.equal(scales.isnan(), bad)
    assert scales[3, 0] == 0 and bool((codes[3, :32] == 0).all())
    assert bool((codes[3, 32:] == 127).all())


# ------------------------------------------------------------------ convolution

def conv_inputs(T, D, W, N, dtype, seed, stride=0):
    gen = torch.Generator().manual_seed(seed)
    x = dict(x=rnd(gen, T, D + stride, dtype=dtype), d_out=rnd(gen, T, D + stride, dtype=dtype),
             weight=rnd(gen, D, W, std=W ** -0.5), bias=rnd(gen, D, std=0.3), state=rnd(gen, N, W - 1, D),
             d_state=rnd(gen, N, W - 1, D))
    if stride:
        x["x"], x["d_out"] = x["x"][:, stride:], x["d_out"][:, :D]
    return x


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("D,stride", [(64, 0), (1, 0), (70, 3), (1032, 24)])
@pytest.mark.parametrize("dtype,out_dtype", [(F32, F32), (BF16, BF16), (BF16, F32), (F32, BF16)])
def test_conv_ragged(W, D, stride, dtype, out_dtype):
    x = conv_inputs(sum(LENS), D, W, len(LENS), dtype, 7 + W, stride)
    y, last = kda.kda_ssm_conv(x["x"], x["weight"], x["bias"], cu_of(LENS), x["state"], out_dtype=out_dtype)
    c = h(x)
    wy, wl = ref.conv(c["x"], c["weight"], c["bias"], c["state"], LENS)
    check("out", y, wy)
    assert torch.equal(last.double().cpu(), wl)


def test_conv_without_bias_state_swish():
    x = conv_inputs(50, 40, 4, 2, F32, 3)
    y, last = kda.kda_ssm_conv(x["x"], x["weight"], num_seqs=2, swish=False)
    c = h(x)
    wy, wl = ref.conv(c["x"], c["weight"], torch.zeros(40).double(), torch.zeros_like(c["state"]), [25, 25], swish=False)
    check("out", y, wy)
    assert torch.equal(last.double().cpu(), wl)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("W,D", [(2, 33), (4, 136)])
def test_conv_tokens_equal_one_call(dtype, W, D):
    """Single tokens with the state in place give what one call over the whole
    sequences gives, bit for bit; so does a call cut in two."""
    N, Lq = 5, 9
    x = conv_inputs(N * Lq, D, W, N, dtype, 11)
    y, last = kda.kda_ssm_conv(x["x"], x["weight"], x["bias"], conv_state=x["state"], num_seqs=N)
    st = x["state"].clone()
    xs = x["x"].view(N, Lq, D)
    for i in range(Lq):
        o, s = kda.kda_ssm_conv(xs[:, i], x["weight"], x["bias"], conv_state=st, conv_state_out=st, num_seqs=N)
        assert s is st and torch.equal(o, y.view(N, Lq, D)[:, i])
    assert torch.equal(st, last)
    st = x["state"].clone()
    a, _ = kda.kda_ssm_conv(xs[:, :2].reshape(-1, D), x["weight"], x["bias"], conv_state=st, conv_state_out=st, num_seqs=N)
    b, _ = kda.kda_ssm_conv(xs[:, 2:].reshape(-1, D), x["weight"], x["bias"], conv_state=st, conv_state_out=st, num_seqs=N)
    assert torch.equal(torch.cat([a.view(N, 2, D), b.view(N, Lq - 2, D)], 1).view(-1, D), y)
    assert torch.equal(st, last)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("W,D,stride", [(2, 64, 0), (3, 70, 3), (4, 1032, 24), (4, 1, 0)])
@pytest.mark.parametrize("dtype,grad_dtype", [(F32, F32), (BF16, BF16), (BF16, F32)])
def test_conv_backward_ragged(W, D, stride, dtype, grad_dtype, packed):
    x = conv_inputs(sum(LENS), D, W, len(LENS), dtype, 17 + W, stride)
    c = h(x)
    inp, scales = x["x"], None
    if packed:
        inp, scales = kda.kda_act_pack8(inp)
        c["x"] = ref.unpack8(inp.cpu(), scales.cpu())
    g = kda.kda_ssm_conv_backward(inp, x["weight"], x["d_out"], x["bias"], cu_of(LENS), x["state"], x_scales=scales,
                                  d_conv_state_out=x["d_state"], grad_dtype=grad_dtype)
    w = ref.conv_backward(c["x"], c["weight"], c["bias"], c["state"], LENS, c["d_out"], c["d_state"])
    for n in w:
        check(n, g[n], w[n])


def test_conv_backward_long_runs():
    """Runs of 64 tokens (a large call), against the formula on a window of channels."""
    T, D, W = 4099, 4096, 4
    x = conv_inputs(T, D, W, 1, BF16, 5)
    g = kda.kda_ssm_conv_backward(x["x"], x["weight"], x["d_out"], x["bias"], conv_state=x["state"])
    c = h({k: v[..., 40:56] if k not in ("weight", "bias") else v[40:56] for k, v in x.items()})
    w = ref.conv_backward(c["x"], c["weight"], c["bias"], c["state"], [T], c["d_out"], torch.zeros_like(c["d_state"]))
    check("dx", g["dx"][:, 40:56], w["dx"])
    check("dweight", g["dweight"][40:56], w["dweight"])
    check("dbias", g["dbias"][40:56], w["dbias"])
    check("d_conv_state", g["d_conv_state"][..., 40:56], w["d_conv_state"])


def test_conv_backward_against_differences():
    """The gradient of a scalar of the outputs against central differences of the
    forward call in 64 bits."""
    x = conv_inputs(sum(LENS), 3, 4, len(LENS), F32, 23)
    c = h(x)
    g = kda.kda_ssm_conv_backward(x["x"], x["weight"], x["d_out"], x["bias"], cu_of(LENS), x["state"],
                                  d_conv_state_out=x["d_state"])

    def value(**over):
        a = dict(c, **over)
        y, last = ref.conv(a["x"], a["weight"], a["bias"], a["state"], LENS)
        return float((y * c["d_out"]).sum() + (last * c["d_state"]).sum())

    gen = torch.Generator().manual_seed(1)
    for n, gn in (("x", "dx"), ("weight", "dweight"), ("bias", "dbias"), ("state", "d_conv_state")):
        way = torch.randn(c[n].shape, generator=gen).double()
        diff = (value(**{n: c[n] + 1e-5 * way}) - value(**{n: c[n] - 1e-5 * way})) / 2e-5
        got = float((g[gn].double().cpu() * way).sum())
        scale = float(g[gn].double().norm().cpu() * way.norm())
        assert abs(diff - got) <= 1e-5 * scale, n


# ------------------------------------------------------------------ scan

@pytest.mark.parametrize("S", [1, 4, 7, 8, 16, 18, 32, 64])
@pytest.mark.parametrize("D,stride", [(64, 0), (1, 0), (77, 3)])
@pytest.mark.parametrize("dtype,out_dtype,gated", [(F32, F32, True), (BF16, BF16, True), (BF16, F32, False), (F32, BF16, False)])
def test_scan_ragged(S, D, stride, dtype, out_dtype, gated):
    x = scan_inputs(sum(LENS), D, S, len(LENS), dtype, 100 + S, gated, stride)
    out, fin, chunks = fwd(x, cu_seqlens=cu_of(LENS), out_dtype=out_dtype, return_chunk_states=True)
    w = ref.scan(h(x), LENS)
    check("out", out, w["out"])
    check("final", fin, w["final"])
    check("chunks", chunks, w["chunks"])


def test_scan_defaults():
    """No skip, gate, bias, state or softplus; equal sequences."""
    x = scan_inputs(66, 40, 16, 2, F32, 5)
    dt = x["dt"].abs() * 0.1
    out, fin = kda.kda_ssm_scan(x["u"], dt, x["A"], x["B"], x["C"], num_seqs=2, softplus=False)
    c = h(dict(x, dt=dt, z=None, D=torch.zeros(40), dt_bias=torch.zeros(40), state=torch.zeros_like(x["state"])))
    w = ref.scan(c, [33, 33], softplus=False)
    check("out", out, w["out"])
    check("final", fin, w["final"])


@pytest.mark.parametrize("T,D,S,N", [(1500, 520, 16, 1), (3001, 40, 16, 1), (700, 24, 8, 3)])
def test_scan_long(T, D, S, N):
    lens = [T // N] * N
    x = scan_inputs(sum(lens), D, S, N, BF16, 9)
    out, fin, chunks = fwd(x, num_seqs=N, out_dtype=F32, return_chunk_states=True)
    w = ref.scan(h(x), lens)
    check("out", out, w["out"])
    check("final", fin, w["final"])
    check("chunks", chunks, w["chunks"])


@pytest.mark.parametrize("D", [24, 520])
@pytest.mark.parametrize("lens", [[3, 2500, 0, 40, 700], [1300, 1, 0, 0, 1999], [0, 0, 3000, 128, 129], [400], [321], [320, 0]])
def test_scan_long_sequences_in_a_ragged_batch(lens, D):
    x = scan_inputs(sum(lens), D, 16, len(lens), F32, 15)
    out, fin, chunks = fwd(x, cu_seqlens=cu_of(lens), return_chunk_states=True)
    w = ref.scan(h(x), lens)
    check("out", out, w["out"])
    check("final", fin, w["final"])
    check("chunks", chunks, w["chunks"])


def test_scan_many_sequences():
    """More sequences than a warp has lanes, one of them long."""
    lens = [5] * 40 + [1500] + [7] * 30
    x = scan_inputs(sum(lens), 24, 16, len(lens), F32, 16)
    out, fin = fwd(x, cu_seqlens=cu_of(lens))
    w = ref.scan(h(x), lens)
    check("out", out, w["out"])
    check("final", fin, w["final"])


def test_malformed_lengths_stay_in_bounds():
    """Decreasing and out-of-range entries are clamped: the calls end and a
    guard around the outputs keeps its value (what the outputs hold is unspecified)."""
    T, D, S = 2000, 24, 16
    x = scan_inputs(T, D, S, 6, F32, 17)
    cu = torch.tensor([0, 1990, 0, 1990, -5, 1990, 99999], dtype=torch.int32, device=DEV)
    guard = 4096
    out = torch.full((T * D + 2 * guard,), 7.0, device=DEV)
    fin = torch.full((6 * D * S + 2 * guard,), 7.0, device=DEV)
    fwd(x, cu_seqlens=cu, out=out[guard:guard + T * D].view(T, D), final_state=fin[guard:guard + 6 * D * S].view(6, D, S))
    torch.cuda.synchronize()
    for t in (out, fin):
        assert bool((t[:guard] == 7).all()) and bool((t[-guard:] == 7).all())
    bwd(x, cu_seqlens=cu, chunk_states=torch.zeros(400, D, S, device=DEV))
    c = conv_inputs(T, D, 4, 6, F32, 18)
    kda.kda_ssm_conv(c["x"], c["weight"], c["bias"], cu, c["state"])
    kda.kda_ssm_conv_backward(c["x"], c["weight"], c["d_out"], c["bias"], cu, c["state"])
    torch.cuda.synchronize()
    kda.kda_get_last_device_error()


def test_scan_extreme_steps():
    """Steps so large that the state is forgotten (decay 0) and so small that they
    vanish: no NaN, and the definition's values."""
    x = scan_inputs(70, 32, 16, 1, F32, 12)
    x["dt"][::3] = 60.0
    x["dt"][1::3] = -80.0
    out, fin = fwd(x)
    w = ref.scan(h(x), [70])
    check("out", out, w["out"])
    check("final", fin, w["final"])


def test_scan_cut_in_two_and_steps():
    """A sequence cut in two, and single tokens, carry the state."""
    N, T, D, S = 3, 50, 40, 16
    x = scan_inputs(N * T, D, S, N, F32, 13)
    out, fin = fwd(x, num_seqs=N)
    part = lambda a, b: {k: (v.view(N, T, -1)[:, a:b].reshape(N * (b - a), -1) if k in ("u", "dt", "B", "C", "z", "d_out") else v)
                         for k, v in x.items()}  # noqa: E731
    one, two = part(0, 17), part(17, T)
    st = x["state"].clone()
    o1, _ = fwd(dict(one, state=st), num_seqs=N, final_state=st)
    o2, _ = fwd(dict(two, state=st), num_seqs=N, final_state=st)
    w = ref.scan(h(x), [T] * N)
    check("out", torch.cat([o1.view(N, 17, D), o2.view(N, T - 17, D)], 1).view(-1, D), w["out"])
    check("final", st, w["final"])
    st = x["state"].clone()
    for i in range(T):
        p = part(i, i + 1)
        o = kda.kda_ssm_step(p["u"], p["dt"], p["A"], p["B"], p["C"], st, D=p["D"], z=p["z"], dt_bias=p["dt_bias"])
        check("step", o, w["out"].view(N, T, D)[:, i])
    check("state", st, w["final"])


@pytest.mark.parametrize("S", [1, 7, 16, 24, 64])
@pytest.mark.parametrize("N,D,stride", [(1, 1, 0), (3, 70, 5), (2, 256, 0)])
@pytest.mark.parametrize("dtype,out_dtype,gated", [(F32, F32, True), (BF16, BF16, True), (BF16, F32, False)])
def test_step(S, N, D, stride, dtype, out_dtype, gated):
    x = scan_inputs(N, D, S, N, dtype, 50 + S, gated, stride)
    w = ref.scan(h(x), [1] * N)
    st = x["state"].clone()
    o = kda.kda_ssm_step(x["u"], x["dt"], x["A"], x["B"], x["C"], st, D=x["D"], z=x["z"], dt_bias=x["dt_bias"],
                         out_dtype=out_dtype)
    check("out", o, w["out"])
    check("state", st, w["final"])


def test_step_large_batch():
    """Enough sequences for several a lane, one more than a multiple of four."""
    N, D, S = 129, 1536, 16
    x = scan_inputs(N, D, S, N, BF16, 61)
    st = x["state"].clone()
    o = kda.kda_ssm_step(x["u"], x["dt"], x["A"], x["B"], x["C"], st, D=x["D"], z=x["z"], dt_bias=x["dt_bias"])
    w = ref.scan(h(x), [1] * N)
    check("out", o, w["out"])
    check("state", st, w["final"])


# ------------------------------------------------------------------ gradients

@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("S", [1, 4, 7, 16, 24, 64])
@pytest.mark.parametrize("D,stride", [(64, 0), (1, 0), (77, 3)])
@pytest.mark.parametrize("dtype,grad_dtype,gated", [(F32, F32, True), (BF16, BF16, True), (BF16, F32, False)])
def test_scan_backward_ragged(S, D, stride, dtype, grad_dtype, gated, packed):
    x = scan_inputs(sum(LENS), D, S, len(LENS), dtype, 200 + S, gated, stride)
    chunks = fwd(x, cu_seqlens=cu_of(LENS), return_chunk_states=True)[2]
    c, kw = h(x), {}
    if packed:
        x["u"], kw["u_scales"] = kda.kda_act_pack8(x["u"])
        c["u"] = ref.unpack8(x["u"].cpu(), kw["u_scales"].cpu())
        if gated:
            x["z"], kw["z_scales"] = kda.kda_act_pack8(x["z"])
            c["z"] = ref.unpack8(x["z"].cpu(), kw["z_scales"].cpu())
    g = bwd(x, cu_seqlens=cu_of(LENS), chunk_states=chunks, grad_dtype=grad_dtype, **kw)
    w = ref.scan_backward(c, LENS, chunks.double().cpu())
    assert (g["dz"] is None) == (not gated)
    for n in w:
        check(n, g[n], w[n])
    assert kda.kda_get_last_device_error() == 0


@pytest.mark.parametrize("T,D,N", [(1000, 136, 1), (2400, 24, 2)])
def test_scan_backward_long(T, D, N):
    """Chunk states computed by the call itself."""
    x = scan_inputs(T, D, 16, N, F32, 31)
    g = bwd(x, num_seqs=N)
    w = ref.scan_backward(h(x), [T // N] * N, None)
    for n in w:
        check(n, g[n], w[n])


@pytest.mark.parametrize("D", [24, 520])
@pytest.mark.parametrize("lens", [[3, 1500, 0, 40, 700], [0, 0, 1000, 128, 129], [321]])
def test_scan_backward_long_sequences_in_a_ragged_batch(lens, D):
    x = scan_inputs(sum(lens), D, 16, len(lens), F32, 35)
    chunks = fwd(x, cu_seqlens=cu_of(lens), return_chunk_states=True)[2]
    g = bwd(x, cu_seqlens=cu_of(lens), chunk_states=chunks)
    w = ref.scan_backward(h(x), lens, chunks.double().cpu())
    for n in w:
        check(n, g[n], w[n])


def test_scan_backward_without_options():
    x = scan_inputs(66, 40, 16, 2, F32, 5)
    dt = x["dt"].abs() * 0.1
    g = kda.kda_ssm_scan_backward(x["u"], dt, x["A"], x["B"], x["C"], x["d_out"], num_seqs=2, softplus=False)
    zero = torch.zeros(40)
    c = h(dict(x, dt=dt, z=None, D=zero, dt_bias=zero, state=torch.zeros_like(x["state"]),
               d_final=torch.zeros_like(x["d_final"])))
    w = ref.scan_backward(c, [33, 33], None, softplus=False)
    assert g["dz"] is None and g["dD"] is None and g["ddt_bias"] is None
    for n in ("du", "ddt", "dB", "dC", "dA", "d_init_state"):
        check(n, g[n], w[n])


def test_scan_backward_against_differences():
    x = scan_inputs(sum(LENS), 3, 5, len(LENS), F32, 41)
    c = h(x)
    g = bwd(x, cu_seqlens=cu_of(LENS))

    def value(**over):
        w = ref.scan(dict(c, **over), LENS)
        return float((w["out"] * c["d_out"]).sum() + (w["final"] * c["d_final"]).sum())

    gen = torch.Generator().manual_seed(1)
    for n, gn in (("u", "du"), ("dt", "ddt"), ("A", "dA"), ("B", "dB"), ("C", "dC"), ("D", "dD"), ("z", "dz"),
                  ("dt_bias", "ddt_bias"), ("state", "d_init_state")):
        way = torch.randn(c[n].shape, generator=gen).double()
        e = 1e-6
        diff = (value(**{n: c[n] + e * way}) - value(**{n: c[n] - e * way})) / (2 * e)
        got = float((g[gn].double().cpu() * way).sum())
        scale = float(g[gn].double().norm().cpu() * way.norm())
        assert abs(diff - got) <= 2e-5 * scale, n


# ------------------------------------------------------------------ what stays as it was

def test_rows_outside_every_sequence_stay():
    """A padded batch: rows before the first and behind the last sequence keep
    what they held, in every output; garbage in those input rows reaches nothing."""
    lens, lead, tail = [37, 5, 64], 3, 40
    T, D, S, N = sum(lens) + lead + tail, 40, 16, 3
    cu = cu_of(lens, lead)
    x = scan_inputs(T, D, S, N, F32, 71)
    inside = slice(lead, lead + sum(lens))
    cut = {k: (v[inside] if k in ("u", "dt", "B", "C", "z", "d_out") else v) for k, v in x.items()}
    for k in ("u", "dt", "B", "C", "z", "d_out"):
        x[k][:lead] = float("nan")
        x[k][lead + sum(lens):] = float("nan")
    w = ref.scan(h(cut), lens)
    out = torch.full((T, D), 7.0, device=DEV)
    rows = kda.checkpoint_count(T, kda.CHUNK, cu)
    _, fin, chunks = fwd(x, cu_seqlens=cu, out=out, chunk_states=torch.empty(rows, D, S, device=DEV))
    check("out", out[inside], w["out"])
    check("final", fin, w["final"])
    keep = torch.cat([out[:lead], out[lead + sum(lens):]])
    assert bool((keep == 7).all())
    g = bwd(x, cu_seqlens=cu, chunk_states=chunks)
    wg = ref.scan_backward(h(cut), lens, chunks.double().cpu())
    for n in wg:
        check(n, g[n][inside] if n in ("du", "ddt", "dz", "dB", "dC") else g[n], wg[n])
    xc = conv_inputs(T, D, 4, N, F32, 72)
    cc = {k: (v[inside] if k in ("x", "d_out") else v) for k, v in xc.items()}
    for k in ("x", "d_out"):
        xc[k][:lead] = float("nan")
        xc[k][lead + sum(lens):] = float("nan")
    out = torch.full((T, D), 7.0, device=DEV)
    _, last = kda.kda_ssm_conv(xc["x"], xc["weight"], xc["bias"], cu, xc["state"], out=out)
    c = h(cc)
    wy, wl = ref.conv(c["x"], c["weight"], c["bias"], c["state"], lens)
    check("conv", out[inside], wy)
    assert torch.equal(last.double().cpu(), wl)
    assert bool((torch.cat([out[:lead], out[lead + sum(lens):]]) == 7).all())
    g = kda.kda_ssm_conv_backward(xc["x"], xc["weight"], xc["d_out"], xc["bias"], cu, xc["state"])
    wg = ref.conv_backward(c["x"], c["weight"], c["bias"], c["state"], lens, c["d_out"], torch.zeros_like(c["d_state"]))
    for n in wg:
        check(n, g[n][inside] if n == "dx" else g[n], wg[n])


def test_nan_stays_in_its_sequence_and_channel():
    x = scan_inputs(96, 40, 16, 3, F32, 81)
    x["u"][40, 7] = float("nan")          # sequence 1, its token 8
    out, fin = fwd(x, num_seqs=3)
    bad = torch.zeros(96, 40, dtype=torch.bool, device=DEV)
    bad[40:64, 7] = True
    assert torch.equal(out.isnan(), bad)
    assert bool(fin[1, 7].isnan().all()) and int(fin.isnan().sum()) == 16


def test_empty_batches():
    D, S = 40, 16
    e = lambda w: torch.empty((0, w), device=DEV)  # noqa: E731
    A, st = -torch.ones(D, S, device=DEV), torch.randn(3, D, S, device=DEV)
    cu = torch.zeros(4, dtype=torch.int32, device=DEV)
    out, fin = kda.kda_ssm_scan(e(D), e(D), A, e(S), e(S), init_state=st, cu_seqlens=cu)
    assert out.shape == (0, D) and torch.equal(fin, st)
    g = kda.kda_ssm_scan_backward(e(D), e(D), A, e(S), e(S), e(D), st, cu_seqlens=cu)
    assert torch.equal(g["d_init_state"], st) and not g["dA"].any()
    w, cs = torch.randn(D, 4, device=DEV), torch.randn(3, 3, D, device=DEV)
    y, last = kda.kda_ssm_conv(e(D), w, cu_seqlens=cu, conv_state=cs)
    assert y.shape == (0, D) and torch.equal(last, cs)
    g = kda.kda_ssm_conv_backward(e(D), w, e(D), cu_seqlens=cu, conv_state=cs, d_conv_state_out=cs)
    assert torch.equal(g["d_conv_state"], cs) and not g["dweight"].any() and not g["dbias"].any()
    codes, scales = kda.kda_act_pack8(e(D))
    assert codes.shape == (0, D) and scales.shape == (0, 2)
    g = kda.kda_ssm_scan_backward(e(D), e(D), A, e(S), e(S), e(D), num_seqs=0)
    assert not g["dA"].any()


def test_missing_chunk_states_are_reported():
    x = scan_inputs(sum(LENS), 40, 16, len(LENS), F32, 91)
    bwd(x, cu_seqlens=cu_of(LENS), chunk_states=torch.zeros(1, 40, 16, device=DEV))
    assert kda.kda_get_last_device_error() == 1
    assert kda.kda_get_last_device_error() == 0
    with pytest.raises(kda.KdaError):
        bwd(scan_inputs(100, 40, 16, 1, F32, 92), chunk_states=torch.zeros(2, 40, 16, device=DEV))


# ------------------------------------------------------------------ a run of them together

def layer(p, x, cu, N, conv_state=None, state=None):
    """One state space layer: projections, convolution, scan."""
    xz = x @ p["w_in"]
    D = xz.shape[1] // 2
    xi, z = xz[:, :D], xz[:, D:]
    u, conv_state = kda.kda_ssm_conv(xi, p["conv_w"], p["conv_b"], cu, conv_state, num_seqs=N)
    dbc = u @ p["w_dbc"]
    R, S = p["w_dt"].shape[0], p["A"].shape[1]
    dt = dbc[:, :R] @ p["w_dt"]
    B, C = dbc[:, R:R + S], dbc[:, R + S:]
    return xi, z, u, dt, B, C, conv_state


def layer_weights(M, D, R, S, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    step = torch.exp(torch.rand(D, generator=gen) * np.log(100.0) + np.log(1e-3))
    return dict(w_in=rnd(gen, M, 2 * D, std=M ** -0.5, dtype=dtype), conv_w=rnd(gen, D, 4, std=0.5), conv_b=rnd(gen, D, std=0.1),
                w_dbc=rnd(gen, D, R + 2 * S, std=D ** -0.5, dtype=dtype), w_dt=rnd(gen, R, D, std=0.5 * R ** -0.5, dtype=dtype),
                A=-torch.arange(1, S + 1).float().repeat(D, 1).to(DEV), D=torch.ones(D, device=DEV),
                dt_bias=(step + torch.log(-torch.expm1(-step))).to(DEV))


def test_layer_prompt_then_tokens():
    """A packed batch of prompts, then decode steps with the states carried on,
    equal one longer prompt call."""
    M, D, R, S, N, T, more = 48, 72, 6, 16, 3, 45, 6
    p = layer_weights(M, D, R, S, F32, 1)
    gen = torch.Generator().manual_seed(2)
    x = rnd(gen, N, T + more, M)

    def whole(xs, N, conv_state, state):
        _, z, u, dt, B, C, cs = layer(p, xs, None, N, conv_state)
        y, st = kda.kda_ssm_scan(u, dt, p["A"], B, C, D=p["D"], z=z, dt_bias=p["dt_bias"], init_state=state, num_seqs=N)
        return y, cs, st

    want, cs_w, st_w = whole(x.reshape(-1, M), N, None, None)
    want = want.view(N, T + more, D)
    y, cs, st = whole(x[:, :T].reshape(-1, M), N, None, None)
    # projections of other row counts differ in their last bits
    tol = dict(rtol=1e-4, atol=1e-5)
    torch.testing.assert_close(y.view(N, T, D), want[:, :T], **tol)
    for i in range(more):
        xt = x[:, T + i]
        xz = xt @ p["w_in"]
        u, _ = kda.kda_ssm_conv(xz[:, :D], p["conv_w"], p["conv_b"], conv_state=cs, conv_state_out=cs, num_seqs=N)
        dbc = u @ p["w_dbc"]
        o = kda.kda_ssm_step(u, dbc[:, :R] @ p["w_dt"], p["A"], dbc[:, R:R + S], dbc[:, R + S:], st, D=p["D"], z=xz[:, D:],
                             dt_bias=p["dt_bias"])
        torch.testing.assert_close(o, want[:, T + i], **tol)
    torch.testing.assert_close(cs, cs_w, **tol)
    torch.testing.assert_close(st, st_w, **tol)


@pytest.mark.parametrize("packed", [False, True])
def test_layer_training_step(packed):
    """Convolution, scan and both gradients in a chain, against the formulas in 64
    bits at the values the backward pass has (the packed ones where it has those)."""
    M, D, R, S = 48, 72, 6, 16
    p = layer_weights(M, D, R, S, F32, 3)
    gen = torch.Generator().manual_seed(4)
    T = sum(LENS)
    cu = cu_of(LENS)
    xi, z, u, dt, B, C, _ = layer(p, rnd(gen, T, M), cu, len(LENS))
    _, _, chunks = kda.kda_ssm_scan(u, dt, p["A"], B, C, D=p["D"], z=z, dt_bias=p["dt_bias"], cu_seqlens=cu, return_chunk_states=True)
    dy = rnd(gen, T, D)
    kept = dict(u=(u, None), z=(z, None), xi=(xi, None))
    if packed:
        kept = {k: kda.kda_act_pack8(v[0]) for k, v in kept.items()}
    g = kda.kda_ssm_scan_backward(kept["u"][0], dt, p["A"], B, C, dy, D=p["D"], z=kept["z"][0], dt_bias=p["dt_bias"], cu_seqlens=cu,
                                  chunk_states=chunks, u_scales=kept["u"][1], z_scales=kept["z"][1])
    gc = kda.kda_ssm_conv_backward(kept["xi"][0], p["conv_w"], g["du"], p["conv_b"], cu, x_scales=kept["xi"][1])
    back = {k: (v[0].double().cpu() if v[1] is None else ref.unpack8(v[0].cpu(), v[1].cpu())) for k, v in kept.items()}
    c = dict(u=back["u"], z=back["z"], dt=dt.double().cpu(), B=B.double().cpu(), C=C.double().cpu(), A=p["A"].double().cpu(),
             D=p["D"].double().cpu(), dt_bias=p["dt_bias"].double().cpu(), d_out=dy.double().cpu(),
             state=torch.zeros(len(LENS), D, S).double(), d_final=torch.zeros(len(LENS), D, S).double())
    w = ref.scan_backward(c, LENS, chunks.double().cpu())
    for n in w:
        check(n, g[n], w[n])
    zero = torch.zeros(len(LENS), 3, D).double()
    wc = ref.conv_backward(back["xi"], p["conv_w"].double().cpu(), p["conv_b"].double().cpu(), zero, LENS, g["du"].double().cpu(), zero)
    for n in wc:
        check(n, gc[n], wc[n])


# ------------------------------------------------------------------ streams, graphs, repetition

def test_repeats_streams_and_graphs():
    """The same bits again: from a second call, from two streams at once, and from
    a captured graph replayed on new inputs."""
    x = scan_inputs(sum(LENS), 136, 16, len(LENS), BF16, 55)
    cx = conv_inputs(sum(LENS), 136, 4, len(LENS), BF16, 56)
    cu = cu_of(LENS)
    rows = kda.checkpoint_count(sum(LENS), kda.CHUNK, cu)

    def all_of(stream=None):
        chunks = torch.empty(rows, 136, 16, device=DEV)
        out, fin, _ = fwd(x, cu_seqlens=cu, chunk_states=chunks, stream=stream)
        g = bwd(x, cu_seqlens=cu, chunk_states=chunks, stream=stream)
        y, last = kda.kda_ssm_conv(cx["x"], cx["weight"], cx["bias"], cu, cx["state"], stream=stream)
        gc = kda.kda_ssm_conv_backward(cx["x"], cx["weight"], cx["d_out"], cx["bias"], cu, cx["state"], stream=stream)
        codes, scales = kda.kda_act_pack8(x["u"], stream=stream)
        return [out, fin, chunks, y, last, codes, scales, *g.values(), *gc.values()]

    want = all_of()
    for a, b in zip(all_of(), want):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = [all_of(s1), all_of(s2)]
    torch.cuda.synchronize()
    for r in got:
        for a, b in zip(r, want):
            assert torch.equal(a, b)
    with torch.cuda.stream(s1):
        all_of()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = all_of()
    new = scan_inputs(sum(LENS), 136, 16, len(LENS), BF16, 57)
    for k in x:
        x[k].copy_(new[k])
    graph.replay()
    torch.cuda.synchronize()
    first = [t.clone() for t in held]
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(held, first, all_of()):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_decode_step_in_a_graph():
    N, D, S = 4, 136, 16
    x = scan_inputs(N, D, S, N, BF16, 58)
    cx = conv_inputs(N, D, 4, N, BF16, 59)
    st, cs = x["state"].clone(), cx["state"].clone()

    def step():
        y, _ = kda.kda_ssm_conv(cx["x"], cx["weight"], cx["bias"], conv_state=cs, conv_state_out=cs, num_seqs=N)
        return kda.kda_ssm_step(y, x["dt"], x["A"], x["B"], x["C"], st, D=x["D"], z=x["z"], dt_bias=x["dt_bias"])

    want = [step().clone() for _ in range(3)]
    st.copy_(x["state"])
    cs.copy_(cx["state"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = step()
    st.copy_(x["state"])
    cs.copy_(cx["state"])
    for w in want:
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, w)


# ------------------------------------------------------------------ addresses

def off_by_one(t):
    """The same values one fp32 element past an allocation's start: contiguous, not 16-byte aligned."""
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    v = flat[1:].view(t.shape)
    v.copy_(t)
    return v


def test_misaligned_parameters_and_states():
    x = scan_inputs(sum(LENS), 72, 16, len(LENS), F32, 301)
    cu = cu_of(LENS)
    for n in ("A", "D", "dt_bias", "state", "d_final"):
        x[n] = off_by_one(x[n])
    rows = kda.checkpoint_count(sum(LENS), kda.CHUNK, cu)
    fin, chunks = off_by_one(torch.empty_like(x["state"])), off_by_one(torch.empty(rows, 72, 16, device=DEV))
    out = off_by_one(torch.empty(sum(LENS), 72, device=DEV))
    fwd(x, cu_seqlens=cu, out=out, final_state=fin, chunk_states=chunks)
    w = ref.scan(h(x), LENS)
    for n, t in (("out", out), ("final", fin), ("chunks", chunks)):
        check(n, t, w[n])
    g, wg = bwd(x, cu_seqlens=cu, chunk_states=chunks), ref.scan_backward(h(x), LENS, chunks.double().cpu())
    for n in wg:
        check(n, g[n], wg[n])
    one = {k: (v[:8] if k in ("u", "dt", "B", "C", "z") else v) for k, v in x.items()}
    st = off_by_one(x["state"])
    o = kda.kda_ssm_step(one["u"], one["dt"], x["A"], one["B"], one["C"], st, D=x["D"], z=one["z"], dt_bias=x["dt_bias"])
    w = ref.scan(h(dict(one, d_out=None)), [1] * 8)
    check("step", o, w["out"])
    check("state", st, w["final"])
    c = conv_inputs(sum(LENS), 72, 4, len(LENS), F32, 302)
    for n in ("weight", "bias", "state", "d_state"):
        c[n] = off_by_one(c[n])
    last = off_by_one(torch.empty_like(c["state"]))
    y, _ = kda.kda_ssm_conv(c["x"], c["weight"], c["bias"], cu, c["state"], conv_state_out=last)
    d = h(c)
    wy, wl = ref.conv(d["x"], d["weight"], d["bias"], d["state"], LENS)
    check("conv", y, wy)
    assert torch.equal(last.double().cpu(), wl)
    g = kda.kda_ssm_conv_backward(c["x"], c["weight"], c["d_out"], c["bias"], cu, c["state"], d_conv_state_out=c["d_state"])
    w = ref.conv_backward(d["x"], d["weight"], d["bias"], d["state"], LENS, d["d_out"], d["d_state"])
    for n in w:
        check(n, g[n], w[n])
    codes, scales = kda.kda_act_pack8(off_by_one(c["x"]))
    want = ref.pack8(c["x"].cpu())
    assert torch.equal(codes.cpu(), want[0]) and torch.equal(scales.cpu(), want[1])


def test_offsets_past_32_bits():
    """Rows a stride of 2^30 elements apart: the third starts past 2^31."""
    T, D, S, stride = 3, 40, 16, (1 << 30) + 8
    x = scan_inputs(T, D, S, 1, BF16, 311)
    c = conv_inputs(T, D, 4, 1, BF16, 312)
    big = torch.empty(2 * stride + 4096, dtype=BF16, device=DEV)
    at = 0

    def far(t):
        nonlocal at
        v = big.as_strided((T, t.shape[1]), (stride, 1), at)
        v.copy_(t)
        at += 64
        return v

    for n in ("u", "dt", "B", "C", "z", "d_out"):
        x[n] = far(x[n])
    c["x"], c["d_out"] = far(c["x"]), far(c["d_out"])
    out, fin = fwd(x, out_dtype=F32)
    w = ref.scan(h(x), [T])
    check("out", out, w["out"])
    check("final", fin, w["final"])
    g, wg = bwd(x, grad_dtype=F32), ref.scan_backward(h(x), [T], None)
    for n in wg:
        check(n, g[n], wg[n])
    d = h(c)
    y, last = kda.kda_ssm_conv(c["x"], c["weight"], c["bias"], conv_state=c["state"], out_dtype=F32)
    wy, wl = ref.conv(d["x"], d["weight"], d["bias"], d["state"], [T])
    check("conv", y, wy)
    assert torch.equal(last.double().cpu(), wl)
    g = kda.kda_ssm_conv_backward(c["x"], c["weight"], c["d_out"], c["bias"], conv_state=c["state"], grad_dtype=F32)
    w = ref.conv_backward(d["x"], d["weight"], d["bias"], d["state"], [T], d["d_out"], torch.zeros_like(d["d_state"]))
    for n in w:
        check(n, g[n], w[n])
    codes, scales = kda.kda_act_pack8(c["x"])
    want = ref.pack8(c["x"].float().cpu())
    assert torch.equal(codes.cpu(), want[0]) and torch.equal(scales.cpu(), want[1])
    st = torch.stack([x["state"][0]] * 3)
    o = kda.kda_ssm_step(x["u"], x["dt"], x["A"], x["B"], x["C"], st, D=x["D"], z=x["z"], dt_bias=x["dt_bias"], out_dtype=F32)
    w = ref.scan(h(dict(x, state=torch.stack([x["state"][0]] * 3))), [1] * 3)
    check("step", o, w["out"])
    del big
    torch.cuda.empty_cache()


def test_states_past_32_bits():
    """More than 2^31 state entries: the last sequence's last channels."""
    N, D, S = 260, 524288 + 16, 16
    A = torch.full((D, S), -0.5, device=DEV)
    st = torch.ones((N, D, S), device=DEV)
    u = torch.full((N, D), 0.25, dtype=BF16, device=DEV)
    dt = torch.zeros((N, D), dtype=BF16, device=DEV)
    bc = torch.ones((N, S), dtype=BF16, device=DEV)
    out = kda.kda_ssm_step(u, dt, A, bc, bc, st, out_dtype=F32)
    delta = np.log(2.0)                     # softplus(0)
    want = np.exp(-0.5 * delta) + delta * 0.25
    for t, v in ((st[-1, -40:], want), (st[0, :40], want), (out[-1, -40:], 16 * want)):
        assert float((t.double() - v).abs().max()) <= 1e-5 * v
    assert float((st.double().sum(-1)[[0, 100, 259]] / 16 - want).abs().max()) <= 1e-5
    del A, st, u, dt, out
    torch.cuda.empty_cache()


def test_two_graphs_of_a_call_replayed_side_by_side():
    """Two captures of the same calls have workspaces of their own: replayed at once on two
    streams they give what the calls give."""
    x = scan_inputs(3000, 72, 16, 1, BF16, 321)
    chunks = fwd(x, return_chunk_states=True)[2]

    def calls():
        out, fin = fwd(x)
        return [out, fin, *(v for v in bwd(x, chunk_states=chunks).values() if v is not None)]

    want = calls()
    torch.cuda.synchronize()
    graphs, held = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held.append(calls())
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for r in held:
        for a, b in zip(r, want):
            assert torch.equal(a, b)


def test_binding_refuses_on_the_gpu():
    x = scan_inputs(64, 40, 16, 2, F32, 331)
    with pytest.raises(ValueError, match="dt_bias"):
        fwd(dict(x, dt_bias=x["dt_bias"][:39]), num_seqs=2)
    with pytest.raises(ValueError, match="init_state"):
        fwd(x, num_seqs=1)
    with pytest.raises(ValueError, match="rows must be contiguous"):
        fwd(dict(x, u=x["u"].t().contiguous().t()), num_seqs=2)
    with pytest.raises(ValueError, match="overlap"):
        fwd(dict(x, B=x["B"][:1].expand(64, 16)), num_seqs=2)
    with pytest.raises(ValueError, match="z must be"):
        fwd(dict(x, z=x["z"].to(BF16)), num_seqs=2)
    with pytest.raises(ValueError, match="both be packed"):
        codes, scales = kda.kda_act_pack8(x["u"])
        bwd(dict(x, u=codes), u_scales=scales, num_seqs=2)
    with pytest.raises(ValueError, match="chunk_states"):
        kda.kda_ssm_scan_backward(codes, x["dt"], x["A"], x["B"], x["C"], x["d_out"], u_scales=scales, num_seqs=2)
    with pytest.raises(kda.KdaError):
        fwd(x, num_seqs=2, out=x["u"])
    with pytest.raises(kda.KdaError):
        kda.kda_ssm_conv(x["u"], torch.zeros(40, 5, device=DEV))
    with pytest.raises(ValueError, match="fp32 or bf16"):
        kda.kda_act_pack8(x["u"].half())


# ------------------------------------------------------------------ how a batch is cut

@pytest.mark.parametrize("singles", [6, 250, 251, 300])
@pytest.mark.parametrize("D,S", [(72, 16), (520, 5)])
def test_ragged_batches_with_long_sequences_among_many(singles, D, S):
    """Long sequences among many short ones, fewer and more sequences than a block has
    threads (256): the long ones are cut, wherever they stand."""
    lens = [700] + [1] * (singles // 2) + [0, 333, 49] + [1] * (singles - singles // 2) + [48, 0]
    x = scan_inputs(sum(lens), D, S, len(lens), F32, 400 + singles)
    cu = cu_of(lens)
    out, fin, chunks = fwd(x, cu_seqlens=cu, return_chunk_states=True)
    w = ref.scan(h(x), lens)
    for n, t in (("out", out), ("final", fin), ("chunks", chunks)):
        check(n, t, w[n])
    g, wg = bwd(x, cu_seqlens=cu, chunk_states=chunks), ref.scan_backward(h(x), lens, chunks.double().cpu())
    for n in wg:
        check(n, g[n], wg[n])
    # the same bits again
    again = fwd(x, cu_seqlens=cu)[0]
    assert torch.equal(again, out)


@pytest.mark.parametrize("T", [33, 64, 95, 96, 257])
def test_short_prompts_are_cut_too(T):
    x = scan_inputs(T, 40, 16, 1, BF16, 450 + T)
    out, fin, chunks = fwd(x, return_chunk_states=True, out_dtype=F32)
    w = ref.scan(h(x), [T])
    for n, t in (("out", out), ("final", fin), ("chunks", chunks)):
        check(n, t, w[n])
    g, wg = bwd(x, chunk_states=chunks, grad_dtype=F32), ref.scan_backward(h(x), [T], chunks.double().cpu())
    for n in wg:
        check(n, g[n], wg[n])
