"""Cases of the state space layer operators: the short causal convolution, the
selective scan (prompt and single token), their gradients, and the 8-bit packing
of the activations that the gradients read.

For one channel d of D, state entry n of S and the tokens t of one sequence:

    c_t   = bias + sum_k w[k] x_{t-(W-1-k)},   conv out = c_t Sigmoid(c_t)
    Delta = softplus(dt + dt_bias)
    h_t[d,n] = exp(Delta_t[d] A[d,n]) h_{t-1}[d,n] + Delta_t[d] u_t[d] B_t[n]
    y_t[d]   = (sum_n C_t[n] h_t[d,n] + D[d] u_t[d]) * z_t[d] Sigmoid(z_t[d])

8-bit packing: 32 neighbouring channels of a token share scale = max|x| / 127 and
hold code = round(x * (127 / max|x|)), half to even.

Sizes: 8192 tokens, 256 single tokens and 12288 = 96 x 128 channels are the sizes of
this repository's layer workloads; 2048 to 8192 channels with 16 states are
generic sizes of such layers.  A packed batch has ragged lengths, some of them 0.
"""
import math
import random

import torch

own = False

CHUNK = 32   # tokens between the states that a forward pass leaves for the gradients
GROUP = 32   # channels that share a scale in the 8-bit packing


def listed():
    return [
        # what a training step keeps of one 8192-token layer, in 8 bits
        dict(name="pack8 layer 8k", op="pack8", T=8192, D=12288, dtype="bf16"),
        # the same of a short packed batch in fp32; the last group of a row is partial
        dict(name="pack8 short fp32", op="pack8", T=1001, D=1000, dtype="f32"),
        # convolution over a whole prompt; x is one half of a projection's rows
        dict(name="conv prompt 8k", op="conv", T=8192, D=8192, N=1, W=4, dtype="bf16"),
        # the convolution of one decode step of 256 sequences, its state in place
        dict(name="conv token 256", op="conv_token", T=256, D=12288, N=256, W=4, dtype="bf16"),
        # a training step's gradient of the convolution, from the 8-bit input
        dict(name="conv backward 8k, 8 bits", op="conv_backward", T=8192, D=8192, N=1, W=4, dtype="bf16", packed=True),
        # the same for a packed fp32 batch with odd sizes, from the input itself
        dict(name="conv backward ragged fp32", op="conv_backward", T=2111, D=1000, N=7, W=4, dtype="f32", packed=False),
        # one long prompt through a 4096-channel layer
        dict(name="scan prompt 8k", op="scan", T=8192, D=4096, S=16, N=1, dtype="bf16", gated=True, states=False),
        # a packed fp32 training batch; leaves the chunk states for the gradients
        dict(name="scan ragged fp32", op="scan", T=2111, D=1000, S=16, N=7, dtype="f32", gated=False, states=True),
        # one decode step of a single sequence: latency
        dict(name="step 1", op="step", T=1, D=2048, S=16, N=1, dtype="bf16", gated=True),
        # one decode step of 256 sequences: the states stream through once
        dict(name="step 256", op="step", T=256, D=12288, S=16, N=256, dtype="bf16", gated=True),
        # a training step's gradient of the 8192-token scan, u and z kept in 8 bits
        dict(name="scan backward 8k, 8 bits", op="scan_backward", T=8192, D=4096, S=16, N=1, dtype="bf16", gated=True, packed=True),
        # the same for a packed fp32 batch with odd sizes, from the inputs themselves
        dict(name="scan backward ragged fp32", op="scan_backward", T=2111, D=1000, S=16, N=7, dtype="f32", gated=True, packed=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["pack8", "conv", "conv_token", "conv_backward", "scan", "step", "scan_backward"])
    dtype = rng.choice(["bf16", "f32"])
    if op == "pack8":
        D = _log(rng, 8, 12288)
        return dict(op=op, T=_log(rng, 1, 8192), D=D, dtype=dtype)
    if op in ("conv_token", "step"):
        T = _log(rng, 1, 256)
        c = dict(op=op, T=T, D=_log(rng, 64, 12288), N=T, dtype=dtype)
        if op == "conv_token":
            return dict(c, W=rng.choice([2, 3, 4]))
        return dict(c, S=rng.choice([8, 16, 16, 24, 64]) if c["D"] <= 2048 else 16, gated=rng.random() < 0.7)
    T = _log(rng, 1, 8192)
    N = rng.choice([1, 1, 2, 5, 13])
    if op in ("conv", "conv_backward"):
        c = dict(op=op, T=T, D=_log(rng, 64, 8192), N=N, W=rng.choice([2, 3, 4, 4]), dtype=dtype)
        return dict(c, packed=rng.random() < 0.5) if op == "conv_backward" else c
    S = rng.choice([8, 16, 16, 16, 24, 64])
    D = _log(rng, 64, 4096)
    while T * D * S > 8192 * 4096 * 16:
        T //= 2
    c = dict(op=op, T=T, D=D, S=S, N=N, dtype=dtype, gated=rng.random() < 0.7)
    if op == "scan":
        return dict(c, states=rng.random() < 0.5)
    return dict(c, packed=rng.random() < 0.5)


# ---------------------------------------------------------------- inputs

def _bounds(case):
    """cu_seqlens of the packed batch: ragged lengths, some of them 0."""
    T, N = case["T"], case["N"]
    if N == T:
        return list(range(T + 1))
    r = random.Random(T * 131 + N)
    return [0] + sorted(r.randint(0, T) for _ in range(N - 1)) + [T]


def _pack8_plain(x):
    """(codes int8 [T, D], scales fp32 [T, ceil(D / 32)])"""
    T, D = x.shape
    G = -(-D // GROUP)
    v = torch.zeros((T, G * GROUP), dtype=torch.float32, device=x.device)
    v[:, :D] = x
    v = v.view(T, G, GROUP)
    amax = v.abs().amax(-1)
    most = torch.full_like(amax, 127.0)
    scales = amax / most
    inv = torch.where(amax > 0, most / amax, torch.zeros_like(amax))
    codes = torch.round(v * inv[..., None]).to(torch.int8).view(T, G * GROUP)[:, :D].contiguous()
    return codes, scales


def _unpack8(codes, scales):
    s = scales.repeat_interleave(GROUP, 1)[:, :codes.shape[1]]
    return codes.to(s.dtype) * s


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(int(seed) * 2 + 1)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    T, D, op = case["T"], case["D"], case["op"]

    def rnd(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=gen, device=dev) * std).to(dtype)

    if op == "pack8":
        # activations with a few large channels, as layers have them
        return dict(op=op, x=(rnd(T, D) * torch.exp(rnd(D))).to(dt))
    N = case["N"]
    cu = _bounds(case)
    s = dict(op=op, cu_host=cu)
    s["cu"] = None if N in (1, T) else torch.tensor(cu, dtype=torch.int32, device=dev)
    s["num_seqs"] = N
    s["plan"] = _plan(cu, T, dev)
    if op.startswith("conv"):
        W = case["W"]
        if op == "conv":
            s["x"] = rnd(T, 2 * D, dtype=dt)[:, :D]   # one half of the projection's rows
        else:
            s["x"] = rnd(T, D, dtype=dt)
        s["weight"] = rnd(D, W, std=W ** -0.5)
        s["bias"] = rnd(D, std=0.1)
        s["state"] = rnd(N, W - 1, D)
        if op == "conv_backward":
            s["d_out"] = rnd(T, D, dtype=dt)
            s["x_scales"] = None
            if case["packed"]:
                s["x"], s["x_scales"] = _pack8_plain(s["x"])
        return s
    S, gated = case["S"], case["gated"]
    s["u"] = rnd(T, D, dtype=dt)
    s["dt"] = rnd(T, D, std=0.5, dtype=dt)
    # step sizes spread over [0.001, 0.1] in their logarithm; decay rates 1 .. S
    step = torch.exp(torch.rand(D, generator=gen, device=dev) * math.log(100.0) + math.log(0.001))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["A"] = -(torch.arange(1, S + 1, device=dev, dtype=torch.float32).repeat(D, 1)
               * torch.exp(rnd(D, S, std=0.1)))
    s["B"] = rnd(T, S, dtype=dt)
    s["C"] = rnd(T, S, dtype=dt)
    s["D"] = 1.0 + rnd(D, std=0.1)
    s["z"] = rnd(T, D, dtype=dt) if gated else None
    s["state"] = rnd(N, D, S, std=0.1)
    if op == "scan":
        s["states"], s["chunk_rows"] = case["states"], len(_chunk_rows(cu))
    if op == "scan_backward":
        s["d_out"] = rnd(T, D, dtype=dt)
        s["d_final"] = rnd(N, D, S)
        s["chunk_states"] = _scan_plain(s, True)[2]
        s["u_scales"] = s["z_scales"] = None
        if case["packed"]:
            s["u"], s["u_scales"] = _pack8_plain(s["u"])
            if gated:
                s["z"], s["z_scales"] = _pack8_plain(s["z"])
    return s


# ---------------------------------------------------------------- plain forms

def _plan(cu, T, dev):
    """The indices that the plain forms work with: of every token its sequence and its place in it, ..."""
    ends, rows = cu, _chunk_rows(cu)
    cu = torch.tensor(cu, device=dev)
    row = torch.arange(T, device=dev)
    seq = torch.searchsorted(cu, row, right=True) - 1
    at = row - cu[seq]
    some = [n for n in range(len(ends) - 1) if ends[n + 1] > ends[n]]   # the sequences with a token
    inner = [j for j, r in enumerate(rows) if r + 1 not in ends]         # the chunk states that a token follows
    index = lambda v: torch.tensor(v, dtype=torch.long, device=dev)      # noqa: E731
    return dict(row=row, seq=seq, at=at, cu=cu, some=index(some), first=index([ends[n] for n in some]),
                last=index([ends[n + 1] - 1 for n in some]), chunk_rows=index(rows), inner=index(inner),
                inner_rows=index([rows[j] + 1 for j in inner]), heads=torch.nonzero(at % CHUNK == 0)[:, 0],
                early=[torch.nonzero(at < back)[:, 0] for back in range(4)])


def _conv_taps(x, state, s):
    """x_{t-(W-1)} .. x_t of every token, [W, T, D]: before a sequence's start, its carried state."""
    W = s["weight"].shape[1]
    row, seq, at = (s["plan"][k] for k in ("row", "seq", "at"))
    taps = []
    for k in range(W):
        back = W - 1 - k
        inside = (at >= back)[:, None]
        taps.append(torch.where(inside, x[(row - back).clamp(min=0)], state[seq, (W - 1 + at - back).clamp(max=W - 2)]))
    return torch.stack(taps)


def _conv_last(x, state, s):
    """The last W - 1 inputs of every sequence, [N, W-1, D]."""
    W = s["weight"].shape[1]
    cu = s["plan"]["cu"]
    length = (cu[1:] - cu[:-1])[:, None]
    at = length - (W - 1) + torch.arange(W - 1, device=x.device)   # place in the sequence; < 0: in the old state
    row = (cu[:-1, None] + at).clamp(min=0)
    old = state.gather(1, (W - 1 + at).clamp(0, W - 2)[..., None].expand_as(state))
    if not x.shape[0]:
        return old
    return torch.where((at >= 0)[..., None], x[row.clamp(max=x.shape[0] - 1)], old)


def _conv_plain(s):
    x = s["x"].float()
    taps = _conv_taps(x, s["state"], s)
    c = s["bias"] + (taps * s["weight"].t()[:, None]).sum(0)
    return (c * torch.sigmoid(c)).to(s["x"].dtype), _conv_last(x, s["state"], s)


def _conv_backward_plain(s):
    x = s["x"].float() if s["x_scales"] is None else _unpack8(s["x"], s["x_scales"])
    w, W, T = s["weight"], s["weight"].shape[1], x.shape[0]
    taps = _conv_taps(x, s["state"], s)
    c = s["bias"] + (taps * w.t()[:, None]).sum(0)
    sg = torch.sigmoid(c)
    dc = s["d_out"].float() * (sg * (1.0 + c * (1.0 - sg)))
    seq, at, early = (s["plan"][k] for k in ("seq", "at", "early"))
    dx = torch.zeros_like(x)
    dstate = torch.zeros_like(s["state"])
    for k in range(W):
        back = W - 1 - k
        part = dc * w[:, k]
        inside = at >= back
        dx[: T - back] += torch.where(inside[back:, None], part[back:], torch.zeros_like(part[back:]))
        rows = early[back]
        dstate.index_put_((seq[rows], W - 1 + at[rows] - back), part[rows], accumulate=True)
    return dict(dx=dx.to(s["d_out"].dtype), dweight=(dc * taps).sum(1).t().contiguous(), dbias=dc.sum(0),
                d_conv_state=dstate)


def _recur(a, b):
    """h_t = a_t h_{t-1} + b_t along dimension 0, h before the first 0: all chunks at once, then from chunk to chunk."""
    T = a.shape[0]
    L = max(1, int(math.sqrt(T)))
    n = -(-T // L)
    p = torch.ones((n * L,) + a.shape[1:], dtype=a.dtype, device=a.device)
    h = torch.zeros_like(p)
    p[:T], h[:T] = a, b
    p, h = p.view(n, L, *a.shape[1:]), h.view(n, L, *a.shape[1:])
    for i in range(1, L):
        h[:, i] += p[:, i] * h[:, i - 1]
        p[:, i] *= p[:, i - 1]
    for c in range(1, n):
        h[c] += p[c] * h[c - 1, -1]
    return h.view(n * L, *a.shape[1:])[:T]


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def _chunk_rows(cu):
    """The tokens whose states a forward pass leaves: the last of each whole chunk of each sequence."""
    return [a + CHUNK * (j + 1) - 1 for a, b in zip(cu[:-1], cu[1:]) for j in range((b - a) // CHUNK)]


def _scan_plain(s, states):
    """(out, final state[, chunk states])"""
    u, B, C = s["u"].float(), s["B"].float(), s["C"].float()
    plan = s["plan"]
    first, some = plan["first"], plan["some"]
    delta = _softplus(s["dt"].float() + s["dt_bias"])
    a = torch.exp(delta[..., None] * s["A"])
    b = (delta * u)[..., None] * B[:, None]
    b[first] += a[first] * s["state"][some]
    a[first] = 0.0
    h = _recur(a, b)
    y = (h * C[:, None]).sum(-1) + s["D"] * u
    if s["z"] is not None:
        z = s["z"].float()
        y = y * (z * torch.sigmoid(z))
    final = s["state"].clone()
    final[some] = h[plan["last"]]
    out = (y.to(s["u"].dtype), final)
    return out + (h[plan["chunk_rows"]],) if states else out


def _step_plain(s):
    u, B, C = s["u"].float(), s["B"].float(), s["C"].float()
    delta = _softplus(s["dt"].float() + s["dt_bias"])
    h = torch.exp(delta[..., None] * s["A"]) * s["state"] + (delta * u)[..., None] * B[:, None]
    y = (h * C[:, None]).sum(-1) + s["D"] * u
    if s["z"] is not None:
        z = s["z"].float()
        y = y * (z * torch.sigmoid(z))
    s["state"].copy_(h)
    return y.to(s["u"].dtype), s["state"]


def _scan_backward_plain(s):
    packed = s["u_scales"] is not None
    u = _unpack8(s["u"], s["u_scales"]) if packed else s["u"].float()
    z = s["z"]
    if z is not None:
        z = _unpack8(z, s["z_scales"]) if packed else z.float()
    B, C, dy, A = s["B"].float(), s["C"].float(), s["d_out"].float(), s["A"]
    T, dev, kind = u.shape[0], u.device, s["d_out"].dtype
    plan = s["plan"]
    at, some, first, heads = (plan[k] for k in ("at", "some", "first", "heads"))
    raw = s["dt"].float() + s["dt_bias"]
    delta = _softplus(raw)
    a = torch.exp(delta[..., None] * A)
    # the states again, from the state at the start of each chunk
    start = torch.zeros((T,) + tuple(A.shape), device=dev)
    start[first] = s["state"][some]
    start[plan["inner_rows"]] = s["chunk_states"][plan["inner"]]
    b = (delta * u)[..., None] * B[:, None]
    b[heads] += a[heads] * start[heads]
    link = a.clone()
    link[heads] = 0.0
    h = _recur(link, b)
    del b
    before = torch.cat([h[:1], h[:-1]])
    before[heads] = start[heads]
    del start
    y = (h * C[:, None]).sum(-1) + s["D"] * u
    res, dyp = {}, dy
    if z is not None:
        sg = torch.sigmoid(z)
        res["dz"] = (dy * y * (sg * (1.0 + z * (1.0 - sg)))).to(kind)
        dyp = dy * (z * sg)
    # the adjoint of the state, from the last token back
    link = torch.zeros_like(a)
    link[:-1] = torch.where((at[1:] > 0)[:, None, None], a[1:], torch.zeros_like(a[1:]))
    g = dyp[..., None] * C[:, None]
    g[plan["last"]] += s["d_final"][some]
    g = _recur(link.flip(0), g.flip(0)).flip(0)
    del link
    res["dC"] = (dyp[..., None] * h).sum(1).to(kind)
    del h
    res["dB"] = (g * (delta * u)[..., None]).sum(1).to(kind)
    gb = (g * B[:, None]).sum(-1)
    d_init = s["d_final"].clone()
    d_init[some] = a[first] * g[first]
    gah = g * a * before
    ddt = (u * gb + (gah * A).sum(-1)) * torch.sigmoid(raw)
    res.update(du=(delta * gb + s["D"] * dyp).to(kind), ddt=ddt.to(kind), ddt_bias=ddt.sum(0),
               dA=(gah * delta[..., None]).sum(0), dD=(dyp * u).sum(0), d_init_state=d_init)
    return res


# ---------------------------------------------------------------- the framework's calls

def _run_own(s):
    import linear_attention_sequence_gb300 as kda
    op = s["op"]
    if op == "pack8":
        return kda.kda_act_pack8(s["x"])
    seqs = dict(cu_seqlens=s["cu"], num_seqs=s["num_seqs"])
    if op == "conv":
        return kda.kda_ssm_conv(s["x"], s["weight"], s["bias"], conv_state=s["state"], **seqs)
    if op == "conv_token":
        return kda.kda_ssm_conv(s["x"], s["weight"], s["bias"], conv_state=s["state"],
                                conv_state_out=s["state"], **seqs)
    if op == "conv_backward":
        return kda.kda_ssm_conv_backward(s["x"], s["weight"], s["d_out"], s["bias"], conv_state=s["state"],
                                         x_scales=s["x_scales"], **seqs)
    args = (s["u"], s["dt"], s["A"], s["B"], s["C"])
    more = dict(D=s["D"], z=s["z"], dt_bias=s["dt_bias"])
    if op == "scan":
        # a program knows its batch's lengths on the host, and so the number of chunk states
        chunks = torch.empty((s["chunk_rows"],) + tuple(s["A"].shape), device="cuda") if s["states"] else None
        return kda.kda_ssm_scan(*args, init_state=s["state"], chunk_states=chunks, **more, **seqs)
    if op == "step":
        return kda.kda_ssm_step(*args, s["state"], **more), s["state"]
    res = kda.kda_ssm_scan_backward(*args, s["d_out"], s["d_final"], init_state=s["state"],
                                    chunk_states=s["chunk_states"], u_scales=s["u_scales"],
                                    z_scales=s["z_scales"], **more, **seqs)
    return {k: v for k, v in res.items() if v is not None}


def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "pack8":
        return _pack8_plain(s["x"])
    if op == "conv":
        return _conv_plain(s)
    if op == "conv_token":
        y, last = _conv_plain(s)
        s["state"].copy_(last)
        return y, s["state"]
    if op == "conv_backward":
        return _conv_backward_plain(s)
    if op == "scan":
        return _scan_plain(s, s["states"])
    if op == "step":
        return _step_plain(s)
    return _scan_backward_plain(s)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    T, D, op = case["T"], case["D"], case["op"]
    e = 2 if case["dtype"] == "bf16" else 4
    G = -(-D // GROUP)
    if op == "pack8":
        return dict(bytes=T * D * (e + 1) + T * G * 4, flops=T * D * 3)
    x8 = T * D + T * G * 4   # a packed input
    N = case["N"]
    if op.startswith("conv"):
        W = case["W"]
        small = D * (W + 1) * 4 + N * (W - 1) * D * 4
        if op == "conv_backward":
            return dict(bytes=(x8 if case["packed"] else T * D * e) + 2 * T * D * e + 2 * small,
                        flops=T * D * (6 * W + 12))
        return dict(bytes=2 * T * D * e + small + N * (W - 1) * D * 4, flops=T * D * (2 * W + 5))
    S, z = case["S"], int(case["gated"])
    state, bc = N * D * S * 4, T * S * e
    par = D * S * 4 + 2 * D * 4
    if op == "scan_backward":
        chunks = len(_chunk_rows(_bounds(case))) * D * S * 4
        x = x8 if case["packed"] else T * D * e
        return dict(bytes=x * (1 + z) + T * D * e * (2 + 2 + z) + 4 * bc + 3 * state + chunks + 2 * par,
                    flops=T * D * (S * 21 + 30))
    chunks = len(_chunk_rows(_bounds(case))) * D * S * 4 if op == "scan" and case["states"] else 0
    return dict(bytes=T * D * e * (3 + z) + 2 * bc + 2 * state + par + chunks, flops=T * D * (S * 7 + 20))


# ---------------------------------------------------------------- the definitions in 64 bits, token by token

def exact(case, seed):
    s = prepare(case, seed)
    f64 = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    op, cu = case["op"], s.get("cu_host")
    if op == "pack8":
        x = f64["x"]
        pad = -x.shape[1] % GROUP
        x = torch.nn.functional.pad(x, (0, pad)).unflatten(1, (-1, GROUP))
        return None, x.abs().max(-1).values / 127
    if op in ("conv", "conv_token"):
        return _exact_conv(f64, cu)
    if op == "conv_backward":
        return _exact_conv_backward(f64, cu)
    if op in ("scan", "step"):
        y, final, chunks = _exact_scan(f64, cu)
        return (y, final, chunks) if op == "scan" and case["states"] else (y, final)
    return _exact_scan_backward(f64, cu)


def _exact_conv(s, cu):
    w, W = s["weight"], s["weight"].shape[1]
    ys, lasts = [], []
    for n, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        line = torch.cat([s["state"][n], s["x"][a:b]])   # the carried inputs, then the sequence's
        c = s["bias"].expand(b - a, -1).clone()
        for k in range(W):
            c += w[:, k] * line[k:k + b - a]
        ys.append(c / (1 + torch.exp(-c)))
        lasts.append(line[b - a:])
    return torch.cat(ys), torch.stack(lasts)


def _exact_conv_backward(s, cu):
    x = s["x"]
    if s["x_scales"] is not None:
        x = torch.stack([x[:, j].double() * s["x_scales"][:, j // GROUP] for j in range(x.shape[1])], 1)
    w, W = s["weight"], s["weight"].shape[1]
    dx, dw, db, ds = [], torch.zeros_like(w), torch.zeros_like(s["bias"]), []
    for n, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        L = b - a
        line = torch.cat([s["state"][n], x[a:b]])
        c = s["bias"].expand(L, -1).clone()
        for k in range(W):
            c += w[:, k] * line[k:k + L]
        e = 1 / (1 + torch.exp(-c))
        dc = s["d_out"][a:b] * (e + c * e * (1 - e))
        d_line = torch.zeros_like(line)
        for k in range(W):
            d_line[k:k + L] += w[:, k] * dc
            dw[:, k] += (dc * line[k:k + L]).sum(0)
        db += dc.sum(0)
        ds.append(d_line[:W - 1])
        dx.append(d_line[W - 1:])
    return dict(dx=torch.cat(dx), dweight=dw, dbias=db, d_conv_state=torch.stack(ds))


def _exact_scan(s, cu):
    y, final, chunks = [], [], []
    for n, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        h = s["state"][n].clone()
        for t in range(a, b):
            step = torch.logaddexp(s["dt"][t] + s["dt_bias"], torch.zeros_like(s["dt_bias"]))[:, None]
            h = h * torch.exp(step * s["A"]) + step * s["u"][t][:, None] * s["B"][t]
            y.append(h @ s["C"][t])
            if (t - a + 1) % CHUNK == 0:
                chunks.append(h)
        final.append(h)
    y = torch.stack(y) + s["D"] * s["u"]
    if s["z"] is not None:
        y = y * s["z"] / (1 + torch.exp(-s["z"]))
    return y, torch.stack(final), torch.stack(chunks) if chunks else s["state"].new_zeros((0,) + s["A"].shape)


def _exact_scan_backward(s, cu):
    u, z, A = s["u"], s["z"], s["A"]
    if s["u_scales"] is not None:
        u = torch.stack([u[:, j].double() * s["u_scales"][:, j // GROUP] for j in range(u.shape[1])], 1)
        if z is not None:
            z = torch.stack([z[:, j].double() * s["z_scales"][:, j // GROUP] for j in range(z.shape[1])], 1)
    T, D, S = u.shape[0], A.shape[0], A.shape[1]
    raw = s["dt"] + s["dt_bias"]
    step = torch.logaddexp(raw, torch.zeros_like(raw))
    dyp = s["d_out"]
    if z is not None:
        e = 1 / (1 + torch.exp(-z))
        dyp = s["d_out"] * z * e
    new = lambda *shape: torch.zeros(shape, dtype=torch.float64, device=u.device)  # noqa: E731
    y, du, dstep, dB, dC = new(T, D), new(T, D), new(T, D), new(T, S), new(T, S)
    dA, d_init, row0 = torch.zeros_like(A), [], 0
    h_all = new(max([b - a for a, b in zip(cu[:-1], cu[1:])] + [0]) + 1, D, S)
    for n, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        starts = {0: s["state"][n]}
        for j in range((b - a) // CHUNK):
            starts[CHUNK * (j + 1)] = s["chunk_states"][row0 + j]
        row0 += (b - a) // CHUNK
        prev = lambda i: starts[i] if i % CHUNK == 0 else h_all[i]  # noqa: E731
        for i in range(b - a):
            t = a + i
            torch.mul(prev(i), torch.exp(step[t][:, None] * A), out=h_all[i + 1])
            h_all[i + 1] += (step[t] * u[t])[:, None] * s["B"][t]
        g = s["d_final"][n].clone()
        for i in range(b - a - 1, -1, -1):
            t = a + i
            y[t] = h_all[i + 1] @ s["C"][t]
            g = g + dyp[t][:, None] * s["C"][t]
            dC[t] = dyp[t] @ h_all[i + 1]
            dB[t] = (step[t] * u[t]) @ g
            gb = g @ s["B"][t]
            du[t] = step[t] * gb
            decay = torch.exp(step[t][:, None] * A)
            g = g * decay
            gh = g * prev(i)
            dstep[t] = u[t] * gb + (gh * A).sum(1)
            dA += gh * step[t][:, None]
        d_init.append(g)
    res = dict(dC=dC, dB=dB, du=du + s["D"] * dyp, dA=dA, dD=(dyp * u).sum(0), d_init_state=torch.stack(d_init))
    res["ddt"] = dstep / (1 + torch.exp(-raw))
    res["ddt_bias"] = res["ddt"].sum(0)
    if z is not None:
        res["dz"] = s["d_out"] * (y + s["D"] * u) * (e + z * e * (1 - e))
    return res
