"""Softmax attention in 64 bits for the tests, one head at a time, and how far the kernels'
documented arithmetic may be from it.

The bounds count roundings (u = eps / 2 of a type, half a step).  The kernels round
each weight p_ij to the 16-bit type, so that out moves by at most u16 sum_j p_ij |v_j|.
Everything else is fp32: a score is a sum of d products in d / 16 steps, each good to a few
units of the last place of the sum of magnitudes, e_s = (4 d / 16 + 8) u32 max sum |q k| scale (8:
the scale, the shift and the exponential), and moves p by the factor 1 + e_s; sums over n keys
take n / 16 steps and the joining of shares: (n / 16 + 64) u32."""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def rows(q, k, v, first, scale):
    """Attention of q [t, H, d] (token i sees keys 0 .. first + i) over k, v [n, H_kv, d] in
    fp64: (out, lse, sum p |v|, largest sum |q k| scale)."""
    q, k, v = q.double(), k.double(), v.double()
    t, H, d = q.shape
    n, Hkv = k.shape[:2]
    out, lse = torch.zeros_like(q), torch.full((t, H), -math.inf, dtype=torch.float64, device=q.device)
    mag, most = torch.zeros_like(q), 0.0
    if n == 0 or t == 0:
        return out, lse, mag, most
    seen = torch.arange(n, device=q.device) <= first + torch.arange(t, device=q.device)[:, None]
    for h in range(H):
        g = h // (H // Hkv)
        s = (q[:, h] @ k[:, g].T) * scale
        most = max(most, float((q[:, h].abs() @ k[:, g].abs().T).max()) * scale)
        s = torch.where(seen, s, torch.full_like(s, -math.inf))
        lse[:, h] = torch.logsumexp(s, 1)
        some = torch.isfinite(lse[:, h])
        p = torch.exp(s - torch.where(some, lse[:, h], torch.zeros_like(lse[:, h]))[:, None])
        # a key that is not seen adds nothing, whatever it holds
        for x, to in ((v[:, g], out), (v[:, g].abs(), mag)):
            to[:, h] = p @ torch.where(seen.any(0)[:, None], x, torch.zeros_like(x))
    return out, lse, mag, most


def score_error(most, d):
    return (4 * d / 16 + 8) * U[torch.float32] * most


def check_rows(out, lse, q, k, v, first, scale, what=""):
    """Asserts that out (and lse) are within the bounds of `rows`."""
    want, wl, mag, most = rows(q, k, v, first, scale)
    n, d = k.shape[0], q.shape[2]
    e = score_error(most, d)
    tol = (U[q.dtype] + 2 * e + (n / 16 + 64) * U[torch.float32]) * mag + U[out.dtype] * want.abs()
    if out.dtype == torch.float16:
        tol = tol + 2.0 ** -25   # half a step of the smallest numbers
    if q.dtype == torch.float16:
        # the same of each weight, next to one that is 1 or more
        tol = tol + 2.0 ** -25 * v.double().abs().nan_to_num(0.0).sum(0).repeat_interleave(q.shape[1] // v.shape[1], 0)
    off = (out.double() - want).abs()
    bad = ~(off <= tol)
    assert not bad.any(), f"{what} out: off by {float(off[bad].max())}, {int(bad.sum())} of {bad.numel()} outside"
    if lse is not None:
        tol = e + (n / 16 + 64) * U[torch.float32] + 4 * U[torch.float32] * wl.abs().clamp(min=1)
        off = torch.where(torch.isinf(wl), (lse.double() != wl).double() * 1e9, (lse.double() - wl).abs())
        bad = ~(off <= torch.where(torch.isinf(wl), torch.zeros_like(tol), tol))
        assert not bad.any(), f"{what} lse: off by {float(off[bad].max())}"


def backward(q, k, v, out, lse, dy, scale):
    """The documented formulas of one sequence in fp64, and for each gradient the magnitudes that
    its bound counts: (grads, of the weights' (dS's) rounding, of the other factors of dS)."""
    T, H, d = q.shape
    Hkv = k.shape[1]
    qd, kd, vd, od, yd, ld = (x.double() for x in (q, k, v, out, dy, lse))
    g = {n: torch.zeros_like(x) for n, x in (("dq", qd), ("dk", kd), ("dv", vd))}
    mag, err = {n: torch.zeros_like(x) for n, x in g.items()}, {n: torch.zeros_like(x) for n, x in g.items()}
    seen = torch.ones(T, T, dtype=torch.bool, device=q.device).tril()
    most = 0.0
    for h in range(H):
        c = h // (H // Hkv)
        s = qd[:, h] @ kd[:, c].T * scale
        most = max(most, float((qd[:, h].abs() @ kd[:, c].abs().T).max()) * scale)
        p = torch.where(seen, torch.exp(s - ld[:, h:h + 1]), torch.zeros_like(s))
        delta = (yd[:, h] * od[:, h]).sum(1, keepdim=True)
        ds = p * (yd[:, h] @ vd[:, c].T - delta)
        # fp32 sums of dP and delta: in units of u32
        e = p * (yd[:, h].abs() @ vd[:, c].abs().T + (yd[:, h] * od[:, h]).abs().sum(1, keepdim=True))
        g["dv"][:, c] += p.T @ yd[:, h]
        mag["dv"][:, c] += p.T @ yd[:, h].abs()
        for n, x, y, at in (("dq", ds, kd[:, c], h), ("dk", ds.T, qd[:, h], c)):
            g[n][:, at] += scale * (x @ y)
            mag[n][:, at] += scale * (x.abs() @ y.abs())
            err[n][:, at] += scale * ((e if n == "dq" else e.T) @ y.abs())
    return g, mag, err, most


def backward_bounds(g, mag, err, most, q, k, lse, dy, scale, dtype):
    """How far each gradient may be off: the weights (dS) rounded to 16 bits, moved by the errors of
    the scores and of lse, fp32 sums, and the result's own rounding."""
    T, _, d = q.shape
    u = U[torch.float32]
    e = 2 * (score_error(most, d) + 4 * u * float(lse.abs().max().clamp(min=1)))
    H = q.shape[1]
    tol = {}
    small = dict(dq=scale * k.double().abs().sum(0).repeat_interleave(H // k.shape[1], 0),
                 dk=scale * q.double().abs().sum(0).unflatten(0, (k.shape[1], -1)).sum(1),
                 dv=dy.double().abs().sum(0).unflatten(0, (k.shape[1], -1)).sum(1))
    for n in g:
        sums = (T * (H if n != "dq" else 1) / 16 + 64) * u
        tol[n] = (U[q.dtype] + e + sums) * mag[n] + (4 * d / 16 + 8) * u * err[n] + U[dtype] * g[n].abs()
        if dtype == torch.float16:
            tol[n] = tol[n] + 2.0 ** -25
        if q.dtype == torch.float16:
            # a weight (dS) below fp16's normal numbers is off by half a step of 2^-24
            tol[n] = tol[n] + 2.0 ** -25 * small[n]
    return tol
