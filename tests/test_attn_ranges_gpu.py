"""GPU tests of softmax attention in fp16 over the range of its weights and of its gradients' inputs: small weights
next to a large one, upstream gradients and values far from 1, rows of different size, weights of long prompts.

Bounds: those of attn_reference.py for roundings, and instead of its allowance for small fp16 numbers (half a
step of 2^-24 of each weight) what the documented powers of two leave: P is stored times 2^15, so that below
the normal numbers it is off by 2^-25 / 2^15; dS is stored times s with |dS| s <= 2^15 for |dS| <= 2 b, b =
|d_out_i| max |v_j|, and s a power of two that is at least 2^14 / (2 b) (two halvings at the most: one of the power
of two itself, one of its root), so that it is off by 2^-25 / s <= 2^-38 b; b is the row's own for dq, that of the
queries that see the key for dk (here: of the sequence and the heads of the group)."""
import pytest
import torch

import linear_attention_sequence_gb300 as kda
from attn_reference import U, backward as ref_backward, backward_bounds, rows, score_error
from test_attn_gpu import DEV, F16, F32, cu_of, prompt_inputs, rnd, starts

pytestmark = pytest.mark.gpu


def check(got, q, k, v, out, lse, dy, lens):
    """Asserts every sequence's gradients (fp32) against the formulas in 64 bits."""
    scale, H, Hkv = q.shape[2] ** -0.5, q.shape[1], k.shape[1]
    at = starts(lens)
    for n, (a, b) in enumerate(zip(at[:-1], at[1:])):
        if a == b:
            continue
        x = [t[a:b] for t in (q, k, v, out, lse, dy)]
        want, mag, err, most = ref_backward(*x, scale)
        old = 2.0 ** -25
        tol = backward_bounds(want, mag, err, most, x[0], x[1], x[4], x[5], scale, F32)
        vmax = x[2].double().norm(dim=2).amax(0).repeat_interleave(H // Hkv)            # [H]
        size = x[5].double().norm(dim=2) * vmax                                          # [T, H]
        small = dict(dq=scale * x[1].double().abs().sum(0).repeat_interleave(H // Hkv, 0),
                     dk=scale * x[0].double().abs().sum(0).unflatten(0, (Hkv, -1)).sum(1),
                     dv=x[5].double().abs().sum(0).unflatten(0, (Hkv, -1)).sum(1))
        left = dict(dq=2.0 ** -38 * size[..., None] * small["dq"],
                    dk=2.0 ** -38 * size.amax(0).unflatten(0, (Hkv, -1)).amax(1)[:, None] * small["dk"],
                    dv=2.0 ** -40 * small["dv"])
        for name in want:
            bound = tol[name] - old * small[name] + left[name]
            off = (got[name][a:b].double() - want[name]).abs()
            bad = ~(off <= bound)
            assert not bad.any(), (f"sequence {n} {name}: off by {float((off / bound)[bad].max())} bounds, {int(bad.sum())} of "
                                   f"{bad.numel()} outside")


def gradients(q, k, v, dy, cu):
    out, lse = kda.kda_attn_prefill(q, k, v, cu, return_lse=True)
    got = kda.kda_attn_backward(q, k, v, out, lse, dy, cu, grad_dtype=F32)
    assert kda.kda_get_last_device_error() == 0
    return got, out, lse


@pytest.mark.parametrize("std", [2.0 ** -18, 2.0 ** -13, 1.0, 2.0 ** 10])
@pytest.mark.parametrize("H,Hkv,d", [(3, 1, 64), (4, 2, 128)])
@pytest.mark.parametrize("lens", [[1], [3, 0, 100], [129], [255, 1, 700], [1500]])
def test_sizes_of_upstream_gradients(lens, H, Hkv, d, std):
    """(2^-18 is below fp16's normal numbers itself: d_out holds what is left of it.)"""
    q, k, v = prompt_inputs(sum(lens), H, Hkv, d, F16, 10)
    dy = rnd(20, F16, sum(lens), H, d, std=std)
    cu = cu_of(lens)
    got, out, lse = gradients(q, k, v, dy, cu)
    check(got, q, k, v, out, lse, dy, lens)


@pytest.mark.parametrize("vstd,ystd", [(2.0 ** 9, 2.0 ** 9), (2.0 ** -13, 2.0 ** -13), (2.0 ** 9, 2.0 ** -13)])
def test_sizes_of_values(vstd, ystd):
    """Products of d_out and v from 2^-23 to 2^21."""
    lens, H, Hkv, d = [3, 300, 40], 4, 2, 64
    q, k, _ = prompt_inputs(sum(lens), H, Hkv, d, F16, 30)
    v, dy = rnd(31, F16, sum(lens), Hkv, d, std=vstd), rnd(32, F16, sum(lens), H, d, std=ystd)
    got, out, lse = gradients(q, k, v, dy, cu_of(lens))
    assert all(bool(torch.isfinite(x).all()) for x in got.values())
    check(got, q, k, v, out, lse, dy, lens)


def test_rows_of_different_size():
    """d_out from 1 down to 2^-14 from row to row, and rows of zeros."""
    lens, H, Hkv, d = [500, 90], 6, 2, 64
    T = sum(lens)
    q, k, v = prompt_inputs(T, H, Hkv, d, F16, 40)
    dy = rnd(43, F32, T, H, d) * 2.0 ** -(torch.arange(T, device=DEV) % 15)[:, None, None]
    dy[::7] = 0
    dy = dy.to(F16)
    got, out, lse = gradients(q, k, v, dy, cu_of(lens))
    check(got, q, k, v, out, lse, dy, lens)
    zero = kda.kda_attn_backward(q, k, v, out, lse, torch.zeros_like(dy), cu_of(lens), grad_dtype=F32)
    assert all(bool((x == 0).all()) for x in zero.values())


def test_sequences_keep_to_themselves():
    """Other sequences 2^12 times as large, or of infinities and NaN: the same bits."""
    lens, H, Hkv, d = [200, 60, 129, 5], 4, 2, 64
    q, k, v = prompt_inputs(sum(lens), H, Hkv, d, F16, 50)
    dy = rnd(53, F16, sum(lens), H, d, std=2.0 ** -14)
    cu, at = cu_of(lens), starts(lens)
    got, out, lse = gradients(q, k, v, dy, cu)
    for change in (lambda x: x * 2.0 ** 12, lambda x: x * float("inf")):
        y, w = dy.clone(), v.clone()
        for n in (1, 3):
            y[at[n]:at[n + 1]], w[at[n]:at[n + 1]] = change(y[at[n]:at[n + 1]]), change(w[at[n]:at[n + 1]])
        again = kda.kda_attn_backward(q, k, w, out, lse, y, cu, grad_dtype=F32)
        for n in (0, 2):
            assert all(torch.equal(again[m][at[n]:at[n + 1]], got[m][at[n]:at[n + 1]]) for m in got)
    # an infinity inside the sequence reaches the gradients that the formulas have it in
    y = dy.clone()
    y[150, 1, 3] = float("inf")
    again = kda.kda_attn_backward(q, k, v, out, lse, y, cu, grad_dtype=F32)
    assert not bool(torch.isfinite(again["dq"][150, 1]).any()) and not bool(torch.isfinite(again["dv"][100, 0, 3]))
    part = slice(at[1], at[2])
    assert all(torch.equal(again[m][part], got[m][part]) for m in got)
    assert torch.equal(again["dq"][:, 2:], got["dq"][:, 2:]) and torch.equal(again["dk"][:, 1], got["dk"][:, 1])


def test_weights_of_a_long_prompt():
    """32,768 equal scores: every weight of the last rows is 2^-15, which fp16 alone holds to ten bits, and dS
    for small d_out is below all of its numbers.  Checked by blocks of rows."""
    T, d, scale = 32768, 64, 0.125
    q, k, v = rnd(60, F16, T, 1, d, std=2.0 ** -4), rnd(61, F16, T, 1, d, std=2.0 ** -4), rnd(62, F16, T, 1, d)
    dy = rnd(63, F16, T, 1, d, std=2.0 ** -13)
    got, out, lse = gradients(q, k, v, dy, None)
    qd, kd, vd, od, yd = (x[:, 0].double() for x in (q, k, v, out, dy))
    want, mag, err = ({n: torch.zeros(T, d, dtype=torch.float64, device=DEV) for n in ("dq", "dk", "dv")} for _ in range(3))
    for a in range(0, T, 2048):
        b = a + 2048
        seen = torch.arange(b, device=DEV) <= torch.arange(a, b, device=DEV)[:, None]
        p = torch.exp(qd[a:b] @ kd[:b].T * scale - lse[a:b].double()) * seen
        delta = (yd[a:b] * od[a:b]).sum(1, keepdim=True)
        ds = p * (yd[a:b] @ vd[:b].T - delta)
        e = p * (yd[a:b].abs() @ vd[:b].abs().T + (yd[a:b] * od[a:b]).abs().sum(1, keepdim=True))
        want["dq"][a:b], mag["dq"][a:b], err["dq"][a:b] = (scale * (x @ y) for x, y in ((ds, kd[:b]), (ds.abs(), kd[:b].abs()),
                                                                                        (e, kd[:b].abs())))
        want["dk"][:b] += scale * (ds.T @ qd[a:b])
        mag["dk"][:b] += scale * (ds.abs().T @ qd[a:b].abs())
        err["dk"][:b] += scale * (e.T @ qd[a:b].abs())
        want["dv"][:b] += p.T @ yd[a:b]
        mag["dv"][:b] += p.T @ yd[a:b].abs()
    # as in backward_bounds, with sums |q k| scale below 1 and |lse| below 16
    size = yd.norm(dim=1) * vd.norm(dim=1).max()
    left = dict(dq=2.0 ** -38 * scale * size[:, None] * kd.abs().sum(0), dk=2.0 ** -38 * scale * size.max() * qd.abs().sum(0),
                dv=2.0 ** -40 * yd.abs().sum(0))
    u = U[F32]
    for n in want:
        tol = (U[F16] + (2 * (4 * d / 16 + 8 + 64) + T / 16 + 64) * u) * mag[n] + (4 * d / 16 + 8) * u * err[n] + left[n] + u * want[n].abs()
        off = (got[n][:, 0].double() - want[n]).abs()
        bad = ~(off <= tol)
        assert not bad.any(), (n, float((off / tol)[bad].max()), int(bad.sum()))


def test_captured_with_inputs_of_other_sizes():
    """One capture, replayed for d_out and v of other sizes: the scales are each replay's own."""
    lens, H, Hkv, d = [300, 1, 77], 6, 2, 128
    T, cu = sum(lens), cu_of(lens)
    q, k, v = prompt_inputs(T, H, Hkv, d, F16, 90)
    dy = rnd(93, F16, T, H, d)

    def call(**kw):
        out, lse = kda.kda_attn_prefill(q, k, v, cu, return_lse=True, **kw)
        return [out, lse, *kda.kda_attn_backward(q, k, v, out, lse, dy, cu, grad_dtype=F32, **kw).values()]

    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for ystd, vstd in ((2.0 ** -14, 1.0), (2.0 ** 8, 2.0 ** 5), (2.0 ** -3, 2.0 ** -14)):
        dy.copy_(rnd(94, F16, T, H, d, std=ystd))
        v.copy_(rnd(95, F16, T, Hkv, d, std=vstd))
        graph.replay()
        torch.cuda.synchronize()
        own = torch.cuda.Stream()
        own.wait_stream(torch.cuda.current_stream())
        for want in (call(), call(stream=own)):
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        check(dict(zip(("dq", "dk", "dv"), got[2:])), q, k, v, got[0], got[1], dy, lens)


# ------------------------------------------------------------------ the forward's weights

def check_small_weights(out, lse, q, k, v, first, rest=False):
    """out [t, H, d] and lse of tokens that see keys 0 .. first + i.  A weight is rounded by half a step, or by 2^-25 /
    2^11 of a row's largest (the documented factor), which the sum of weights is at least; with `rest` what that leaves
    follows as a second operand, and of it the same is left."""
    want, wl, mag, most = rows(q, k, v, first, 1.0)
    n, e = k.shape[0], score_error(most, q.shape[2])
    tol = ((U[F16] ** 2 if rest else U[F16]) + 2 * e + (n / 8 + 64) * U[F32]) * mag + U[F32] * want.abs()
    tol = tol + 2.0 ** -36 * v.double().abs().sum(0).repeat_interleave(q.shape[1] // v.shape[1], 0)
    off = (out.double() - want).abs()
    assert bool((off <= tol).all()), float((off / tol).max())
    assert bool(((lse.double() - wl).abs() <= e + (n / 16 + 64) * U[F32] + 4 * U[F32] * wl.abs()).all())


def one_and_many(n, d, seed):
    """Keys of which the first has a score 17.40625 above all others: their weights are 2^-25.1 next to it; values that are 0
    there, so that the result is what those weights give."""
    k, v = torch.zeros(n, 1, d, device=DEV, dtype=F16), rnd(seed, F16, n, 1, d).abs()
    k[0, 0, 0], v[0] = 17.40625, 0
    return k, v


@pytest.mark.parametrize("d", [64, 128])
def test_many_small_weights_of_a_prompt(d):
    T = 32768
    k, v = one_and_many(T, d, 70)
    q = torch.zeros(T, 1, d, device=DEV, dtype=F16)
    q[:, 0, 0] = 1
    out, lse = kda.kda_attn_prefill(q, k, v, scale=1.0, out_dtype=F32, return_lse=True)
    for a in (1000, T - 3):
        check_small_weights(out[a:a + 3], lse[a:a + 3], q[a:a + 3], k[:a + 3], v[:a + 3], a)


@pytest.mark.parametrize("new", [1, 20])
@pytest.mark.parametrize("N", [1, 2500])
@pytest.mark.parametrize("d", [64, 128])
def test_many_small_weights_of_a_cache(d, N, new):
    """One sequence, whose keys are split over blocks, and so many (of the same pages) that they are not."""
    n, page = 16384, 128
    k, v = one_and_many(n, d, 80)
    kp, vp = (x.view(n // page, page, 1, d) for x in (k, v))
    table = torch.arange(n // page, dtype=torch.int32, device=DEV).expand(N, -1).contiguous()
    lens = torch.full((N,), n, dtype=torch.int32, device=DEV)
    q = torch.zeros(N * new, 1, d, device=DEV, dtype=F16)
    q[:, 0, 0] = 1
    out, lse = kda.kda_attn_paged(q, kp, vp, table, lens, scale=1.0, out_dtype=F32, return_lse=True)
    for i in {0, N // 2, N - 1}:
        part = slice(i * new, (i + 1) * new)
        check_small_weights(out[part], lse[part], q[part], k, v, n - new, rest=new == 1)
    assert kda.kda_get_last_device_error() == 0
