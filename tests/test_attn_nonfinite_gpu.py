"""GPU tests of an infinity or NaN inside a sequence: who sees it has it, and how far before (and in the gradients
behind) it may reach is documented; everything farther away keeps its bits."""
import pytest
import torch

import linear_attention_sequence_gb300 as kda
from test_attn_gpu import BF16, DEV, F16, F32, make_cache, prompt_inputs, rnd

pytestmark = pytest.mark.gpu

PROMPTS, CHUNKS = 127, 382   # tokens before it, as in include/kda.h


def reached(a, b):
    """Tokens whose results differ in any bit (NaN equals NaN here: it is what it was)."""
    same = (a == b) | (torch.isnan(a) & torch.isnan(b))
    return (~same).flatten(1).any(1)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("H,Hkv,d,dtype", [(1, 1, 64, BF16), (3, 1, 128, F16), (12, 1, 64, BF16)])
@pytest.mark.parametrize("x", [0, 200, 383, 384, 699])
def test_prompts(x, H, Hkv, d, dtype, bad):
    T = 700
    q, k, v = prompt_inputs(T, H, Hkv, d, dtype, 10)
    was = kda.kda_attn_prefill(q, k, v, out_dtype=F32)
    v[x, 0, 5] = bad
    now = kda.kda_attn_prefill(q, k, v, out_dtype=F32)
    assert not bool(torch.isfinite(now[x:, :, 5]).any())
    assert not bool(reached(was, now)[:max(0, x - PROMPTS)].any())
    v[x, 0, 5] = 0
    k[x, 0, 5] = bad          # scores: masked before anything is made of them
    now = kda.kda_attn_prefill(q, k, v, out_dtype=F32)
    assert bool(reached(was, now)[x:].all()) and not bool(reached(was, now)[:x].any())


@pytest.mark.parametrize("H,Hkv,d,dtype", [(1, 1, 64, BF16), (2, 1, 128, F16), (20, 1, 64, BF16)])
@pytest.mark.parametrize("new,total", [(255, 256), (300, 6001), (512, 33000), (600, 40001), (16, 700)])
def test_chunks(new, total, H, Hkv, d, dtype):
    """Positions that start anywhere, pieces that are turned: 254 tokens by the first, up to 382 by both."""
    kp, vp, table, lens, ks, vs = make_cache([total], Hkv, d, 16, dtype, 20)
    q = rnd(21, dtype, new, H, d, std=1.5)
    was = kda.kda_attn_paged(q, kp, vp, table, lens, out_dtype=F32)
    for x in (total - 1, total - new // 2, total - new):
        page, at = int(table[0, x // 16]), x % 16
        keep = vp[page, at, 0, 3].clone()
        vp[page, at, 0, 3] = float("nan")
        now = kda.kda_attn_paged(q, kp, vp, table, lens, out_dtype=F32)
        first = x - (total - new)                      # the token whose own key it is
        assert bool(torch.isnan(now[first:, :, 3]).all())
        assert not bool(reached(was, now)[:max(0, first - CHUNKS)].any())
        vp[page, at, 0, 3] = keep
    assert torch.equal(was, kda.kda_attn_paged(q, kp, vp, table, lens, out_dtype=F32))


@pytest.mark.parametrize("H,Hkv,d", [(1, 1, 64), (6, 2, 128)])
@pytest.mark.parametrize("x", [0, 130, 383, 599])
def test_gradients(x, H, Hkv, d):
    """d_out of one token, v of one token: where the formulas have it, and at most 127 tokens to either side."""
    T = 600
    q, k, v = prompt_inputs(T, H, Hkv, d, BF16, 30)
    dy = rnd(31, BF16, T, H, d)
    out, lse = kda.kda_attn_prefill(q, k, v, return_lse=True)
    was = kda.kda_attn_backward(q, k, v, out, lse, dy, grad_dtype=F32)
    y = dy.clone()
    y[x, 0] = float("nan")
    now = kda.kda_attn_backward(q, k, v, out, lse, y, grad_dtype=F32)
    r = {n: reached(was[n], now[n]) for n in was}
    assert int(r["dq"].sum()) == 1 and bool(r["dq"][x])
    for n in ("dk", "dv"):
        assert bool(torch.isnan(now[n][:x + 1, 0]).all()) and not bool(r[n][x + 128:].any())
    if H > 1:   # heads of the other group
        assert all(torch.equal(was[n][:, -1], now[n][:, -1]) for n in was)
    w = v.clone()
    w[x] = float("inf")
    out2, lse2 = kda.kda_attn_prefill(q, k, w, return_lse=True)
    now = kda.kda_attn_backward(q, k, w, out2, lse2, dy, grad_dtype=F32)
    assert not bool(reached(was["dq"], now["dq"])[:max(0, x - 2 * 127)].any())   # (out reaches 127 tokens back itself)
    assert not bool(torch.isfinite(now["dq"][x:]).any())
    assert torch.equal(was["dv"], now["dv"])
