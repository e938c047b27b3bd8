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
    off = (out.double() - want).abs()
    bad = ~(off <= tol)
    assert not bad.any(), f"{what} out: off by {float(off[bad].max())}, {int(bad.sum())} of {bad.numel()} outside"
    if lse is not None:
        tol = e + (n / 16 + 64) * U[torch.float32] + 4 * U[torch.float32] * wl.abs().clamp(min=1)
        off = torch.where(torch.isinf(wl), (lse.double() != wl).double() * 1e9, (lse.double() - wl).abs())
        bad = ~(off <= torch.where(torch.isinf(wl), torch.zeros_like(tol), tol))
        assert not bad.any(), f"{what} lse: off by {float(off[bad].max())}"
