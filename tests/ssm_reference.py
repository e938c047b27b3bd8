"""Plain implementations in 64 bits of the state space layer calls, one token at
a time, for the tests.  Inputs are CPU tensors; `lens` the lengths of the packed
sequences."""
import torch

GROUP, CHUNK = 32, 32


def pack8(x):
    """Codes and scales of [T, D], each step rounded in fp32 as documented."""
    T, D = x.shape
    x = x.float()
    G = -(-D // GROUP)
    codes, scales = torch.zeros(T, D, dtype=torch.int8), torch.zeros(T, G)
    for g in range(G):
        part = x[:, g * GROUP:(g + 1) * GROUP]
        m = part.abs().max(1).values
        scales[:, g] = m / torch.full_like(m, 127.0)
        inv = torch.where(m > 0, torch.full_like(m, 127.0) / m, torch.zeros_like(m))
        codes[:, g * GROUP:(g + 1) * GROUP] = torch.round(part * inv[:, None]).to(torch.int8)
    return codes, scales


def unpack8(codes, scales):
    """The fp32 products, as the kernels form them."""
    return (codes.float() * scales.repeat_interleave(GROUP, 1)[:, :codes.shape[1]]).double()


def _starts(lens):
    at, res = 0, []
    for n in lens:
        res.append((at, at + n))
        at += n
    return res


def _line(x, state, w, b, a, e, n, swish):
    W = w.shape[1]
    line = torch.cat([state[n], x[a:e]])
    c = b + sum(line[k:k + e - a] * w[:, k] for k in range(W))
    return line, c, (c / (1 + torch.exp(-c)) if swish else c)


def conv(x, w, b, state, lens, swish=True):
    ys, last = [], []
    for n, (a, e) in enumerate(_starts(lens)):
        line, _, y = _line(x, state, w, b, a, e, n, swish)
        ys.append(y)
        last.append(line[e - a:])
    return torch.cat(ys), torch.stack(last)


def conv_backward(x, w, b, state, lens, dy, d_last):
    W = w.shape[1]
    dx, dw, db, ds = torch.zeros_like(x), torch.zeros_like(w), torch.zeros_like(b), torch.zeros_like(state)
    for n, (a, e) in enumerate(_starts(lens)):
        line, c, _ = _line(x, state, w, b, a, e, n, True)
        s = 1 / (1 + torch.exp(-c))
        dc = dy[a:e] * (s + c * s * (1 - s))
        d_line = torch.zeros_like(line)
        d_line[e - a:] += d_last[n]
        for k in range(W):
            d_line[k:k + e - a] += dc * w[:, k]
            dw[:, k] += (dc * line[k:k + e - a]).sum(0)
        db += dc.sum(0)
        ds[n], dx[a:e] = d_line[:W - 1], d_line[W - 1:]
    return dict(dx=dx, dweight=dw, dbias=db, d_conv_state=ds)


def _delta(x, softplus):
    raw = x["dt"] + x["dt_bias"]
    return raw, (torch.logaddexp(raw, torch.zeros_like(raw)) if softplus else raw)


def scan(x, lens, softplus=True):
    _, dl = _delta(x, softplus)
    y, fin, chunks = torch.zeros_like(x["u"]), [], []
    for n, (a, e) in enumerate(_starts(lens)):
        h = x["state"][n]
        for t in range(a, e):
            h = torch.exp(dl[t][:, None] * x["A"]) * h + (dl[t] * x["u"][t])[:, None] * x["B"][t]
            y[t] = (h * x["C"][t]).sum(1) + x["D"] * x["u"][t]
            if (t - a + 1) % CHUNK == 0:
                chunks.append(h)
        fin.append(h)
    if x["z"] is not None:
        y = y * x["z"] / (1 + torch.exp(-x["z"]))
    none = x["A"].new_zeros((0,) + tuple(x["A"].shape))
    return dict(out=y, final=torch.stack(fin), chunks=torch.stack(chunks) if chunks else none)


def scan_backward(x, lens, chunks, softplus=True):
    """`chunks`: the states to run on from (None: the run's own)."""
    u, A, B, C, z = x["u"], x["A"], x["B"], x["C"], x["z"]
    raw, dl = _delta(x, softplus)
    sg = None if z is None else 1 / (1 + torch.exp(-z))
    dyp = x["d_out"] if z is None else x["d_out"] * z * sg
    y, du, dd = torch.zeros_like(u), torch.zeros_like(u), torch.zeros_like(u)
    dB, dC, dA, d_init, row0 = torch.zeros_like(B), torch.zeros_like(C), torch.zeros_like(A), [], 0
    for n, (a, e) in enumerate(_starts(lens)):
        h, before, after = x["state"][n], [], []
        for t in range(a, e):
            if chunks is not None and t > a and (t - a) % CHUNK == 0:
                h = chunks[row0 + (t - a) // CHUNK - 1]
            before.append(h)
            h = torch.exp(dl[t][:, None] * A) * h + (dl[t] * u[t])[:, None] * B[t]
            after.append(h)
        row0 += (e - a) // CHUNK
        g = x["d_final"][n]
        for t in range(e - 1, a - 1, -1):
            g = g + dyp[t][:, None] * C[t]
            y[t] = (after[t - a] * C[t]).sum(1) + x["D"] * u[t]
            dC[t] = (dyp[t][:, None] * after[t - a]).sum(0)
            dB[t] = ((dl[t] * u[t])[:, None] * g).sum(0)
            p = (g * B[t]).sum(1)
            g = g * torch.exp(dl[t][:, None] * A)
            gh = g * before[t - a]
            du[t] = dl[t] * p + x["D"] * dyp[t]
            dd[t] = u[t] * p + (gh * A).sum(1)
            dA += gh * dl[t][:, None]
        d_init.append(g)
    if softplus:
        dd = dd / (1 + torch.exp(-raw))
    res = dict(du=du, ddt=dd, dB=dB, dC=dC, dA=dA, dD=(dyp * u).sum(0), ddt_bias=dd.sum(0), d_init_state=torch.stack(d_init))
    if z is not None:
        res["dz"] = x["d_out"] * y * (sg + z * sg * (1 - sg))
    return res
