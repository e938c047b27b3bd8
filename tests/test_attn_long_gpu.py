"""GPU tests of softmax attention at the lengths it is meant for, against 64 bits: prompts of 8192 tokens and
their gradients, chunks and single tokens behind tens of thousands.  Bounds as in attn_reference.py."""
import pytest
import torch

import linear_attention_sequence_gb300 as kda
from test_attn_gpu import (BF16, F16, F32, check_backward, check_paged, check_prompts, cu_of, make_cache, prompt_inputs,
                           rnd)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,Hkv,d,dtype", [(3, 1, 128, BF16), (2, 2, 64, F16), (12, 1, 64, BF16), (4, 2, 128, F16)])
@pytest.mark.parametrize("lens", [[8192], [5003, 1, 3188]])
def test_prompts_and_gradients(lens, H, Hkv, d, dtype):
    T = sum(lens)
    q, k, v = prompt_inputs(T, H, Hkv, d, dtype, 10)
    cu = None if len(lens) == 1 else cu_of(lens)
    exact, lse = kda.kda_attn_prefill(q, k, v, cu, out_dtype=F32, return_lse=True)
    check_prompts(exact, lse, q, k, v, lens)
    out, again = kda.kda_attn_prefill(q, k, v, cu, return_lse=True)
    assert torch.equal(out, exact.to(dtype)) and torch.equal(lse, again)
    dy = rnd(20, dtype, T, H, d)
    got = kda.kda_attn_backward(q, k, v, out, lse, dy, cu, grad_dtype=F32)
    check_backward(got, q, k, v, out, lse, dy, lens)
    twice = kda.kda_attn_backward(q, k, v, out, lse, dy, cu, grad_dtype=F32)
    assert all(torch.equal(got[n], twice[n]) for n in got)
    assert kda.kda_get_last_device_error() == 0


@pytest.mark.parametrize("H,Hkv,d,dtype,page", [(4, 1, 128, BF16, 64), (3, 3, 64, F16, 16)])
@pytest.mark.parametrize("new,total", [([512], [32768]), ([1], [100003]), ([1, 700, 1, 30], [32768, 20001, 7, 9000])])
def test_long_caches(new, total, H, Hkv, d, dtype, page):
    kp, vp, table, lens, ks, vs = make_cache(total, Hkv, d, page, dtype, 30)
    q = rnd(40, dtype, sum(new), H, d, std=1.5)
    cu = cu_of(new) if len(new) > 1 else None
    out, lse = kda.kda_attn_paged(q, kp, vp, table, lens, cu, out_dtype=F32, return_lse=True)
    check_paged(out, lse, q, new, total, ks, vs)
    assert kda.kda_get_last_device_error() == 0
