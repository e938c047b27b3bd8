"""GPU tests of softmax attention: whole prompts, new tokens over a paged cache."""
import math

import pytest
import torch

import linear_attention_sequence_gb300 as kda
from attn_reference import backward as ref_backward, backward_bounds, check_rows

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def starts(lens, first=0):
    at = [first]
    for n in lens:
        at.append(at[-1] + n)
    return at


def cu_of(lens, first=0):
    return torch.tensor(starts(lens, first), dtype=torch.int32, device=DEV)


def rnd(seed, dtype, *shape, std=1.0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=gen, device=DEV) * std).to(dtype)


def prompt_inputs(T, H, Hkv, d, dtype, seed, std=1.5):
    return (rnd(seed, dtype, T, H, d, std=std), rnd(seed + 1, dtype, T, Hkv, d), rnd(seed + 2, dtype, T, Hkv, d))


def check_prompts(out, lse, q, k, v, lens, first=0, scale=None):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    at = starts(lens, first)
    for n, (a, b) in enumerate(zip(at[:-1], at[1:])):
        check_rows(out[a:b], None if lse is None else lse[a:b], q[a:b], k[a:b], v[a:b], 0, scale, f"sequence {n}")


HEADS = [(1, 1), (3, 1), (8, 2), (12, 1), (5, 5), (96, 2)]


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F16, 64), (F16, 128), (BF16, 64)])
@pytest.mark.parametrize("H,Hkv", HEADS)
@pytest.mark.parametrize("lens", [[1], [2], [127], [128], [129], [255, 1, 0, 257], [37, 0, 0, 64, 130], [700]])
def test_prompts(lens, H, Hkv, d, dtype):
    T = sum(lens)
    q, k, v = prompt_inputs(T, H, Hkv, d, dtype, 10 + T)
    cu = None if len(lens) == 1 else cu_of(lens)
    out, lse = kda.kda_attn_prefill(q, k, v, cu, out_dtype=F32, return_lse=True)
    check_prompts(out, lse, q, k, v, lens)
    rounded = kda.kda_attn_prefill(q, k, v, cu)
    assert rounded.dtype == dtype and torch.equal(rounded, out.to(dtype))
    assert kda.kda_get_last_device_error() == 0


def make_cache(total, Hkv, d, page, dtype, seed, spare=3, order="NHD", fill=float("nan")):
    """A cache with the sequences' keys and values on shuffled pages; everything else in it,
    the places behind each sequence's last token too, holds `fill`."""
    need = [-(-n // page) for n in total]
    P, wide = sum(need) + spare, max(need + [1]) + 2
    shape = (P, page, Hkv, d) if order == "NHD" else (P, Hkv, page, d)
    kp, vp = (torch.full(shape, fill, device=DEV, dtype=dtype) for _ in range(2))
    if order == "HND":
        kp, vp = kp.transpose(1, 2), vp.transpose(1, 2)
    gen = torch.Generator().manual_seed(seed)
    pages = torch.randperm(P, generator=gen).tolist()
    table = torch.full((len(total), wide), -1, dtype=torch.int32)
    ks, vs, at = [], [], 0
    for n, length in enumerate(total):
        k, v = rnd(seed + 2 * n, dtype, length, Hkv, d), rnd(seed + 2 * n + 1, dtype, length, Hkv, d)
        for j in range(need[n]):
            p = pages[at + j]
            table[n, j] = p
            part = slice(j * page, min((j + 1) * page, length))
            kp[p, :part.stop - part.start] = k[part]
            vp[p, :part.stop - part.start] = v[part]
        at += need[n]
        ks.append(k)
        vs.append(v)
    return kp, vp, table.to(DEV), torch.tensor(total, dtype=torch.int32, device=DEV), ks, vs


def check_paged(out, lse, q, new, total, ks, vs, first=0, scale=None):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    at = starts(new, first)
    for n, (a, b) in enumerate(zip(at[:-1], at[1:])):
        check_rows(out[a:b], None if lse is None else lse[a:b], q[a:b], ks[n], vs[n], total[n] - new[n], scale,
                   f"sequence {n}")


# (new tokens, tokens in the cache)
CHUNKS = [
    ([1], [1]), ([1], [63]), ([1], [64]), ([1], [65]), ([1], [5000]),
    ([1, 1, 1], [17, 0, 300]),                      # a length of 0 sees nothing
    ([2, 0, 1, 16], [2, 40, 700, 129]),
    ([129, 1, 0, 300], [129, 2000, 5, 431]),
    ([40], [3000]), ([300], [6000]),
    ([5, 200], [3, 100]),                           # fewer tokens in the cache than new: the first see nothing
]


@pytest.mark.parametrize("H,Hkv", [(1, 1), (8, 2), (12, 1), (5, 5), (32, 1)])
@pytest.mark.parametrize("new,total", CHUNKS)
@pytest.mark.parametrize("dtype,d,page", [(BF16, 128, 64), (F16, 64, 16), (BF16, 64, 8), (F16, 128, 256)])
def test_paged(dtype, d, page, new, total, H, Hkv):
    kp, vp, table, lens, ks, vs = make_cache(total, Hkv, d, page, dtype, 100 + sum(total))
    q = rnd(7, dtype, sum(new), H, d, std=1.5)
    cu = None if len(set(new)) == 1 else cu_of(new)
    out, lse = kda.kda_attn_paged(q, kp, vp, table, lens, cu, out_dtype=F32, return_lse=True)
    check_paged(out, lse, q, new, total, ks, vs)
    rounded = kda.kda_attn_paged(q, kp, vp, table, lens, cu)
    assert rounded.dtype == dtype and torch.equal(rounded, out.to(dtype))
    assert kda.kda_get_last_device_error() == 0


def check_backward(got, q, k, v, out, lse, dy, lens, first=0, scale=None):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    at = starts(lens, first)
    for n, (a, b) in enumerate(zip(at[:-1], at[1:])):
        if a == b:
            continue
        args = (q[a:b], k[a:b], v[a:b], out[a:b], lse[a:b], dy[a:b])
        want, mag, err, most = ref_backward(*args, scale)
        tol = backward_bounds(want, mag, err, most, q[a:b], k[a:b], lse[a:b], dy[a:b], scale, got["dq"].dtype)
        for name in want:
            off = (got[name][a:b].double() - want[name]).abs()
            bad = ~(off <= tol[name])
            assert not bad.any(), (f"sequence {n} {name}: off by {float(off[bad].max())}, bound there "
                                   f"{float(tol[name][bad].min())}, {int(bad.sum())} of {bad.numel()} outside")


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F16, 64), (F16, 128), (BF16, 64)])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 1), (8, 2), (5, 5), (12, 1)])
@pytest.mark.parametrize("lens", [[1], [2], [127], [128], [129], [255, 1, 0, 257], [37, 0, 0, 64, 130], [700]])
def test_backward(lens, H, Hkv, d, dtype):
    T = sum(lens)
    q, k, v = prompt_inputs(T, H, Hkv, d, dtype, 50 + T)
    dy = rnd(60 + T, dtype, T, H, d)
    cu = None if len(lens) == 1 else cu_of(lens)
    out, lse = kda.kda_attn_prefill(q, k, v, cu, return_lse=True)
    grads = kda.kda_attn_backward(q, k, v, out, lse, dy, cu, grad_dtype=F32)
    check_backward(grads, q, k, v, out, lse, dy, lens)
    rounded = kda.kda_attn_backward(q, k, v, out, lse, dy, cu)
    for n in grads:
        assert rounded[n].dtype == dtype and torch.equal(rounded[n], grads[n].to(dtype))
    assert kda.kda_get_last_device_error() == 0
