"""Host-side checks of the softmax attention and cache calls (no GPU): the C entry points
refuse bad arguments before anything reaches the device, and the binding refuses what it
can see.  Every pointer here is made up and never read."""
import ctypes

import pytest
import torch

import linear_attention_sequence_gb300 as kda
from linear_attention_sequence_gb300 import _build


class _Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class _Pages(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p)] + [(n, ctypes.c_int64) for n in ("page_stride", "token_stride", "head_stride")]


class _Dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("num_seqs", "total_tokens", "q_heads", "kv_heads", "head_dim", "in_dtype",
                                              "out_dtype")] + [("scale", ctypes.c_float)]


class _Cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("num_pages", "page_size", "max_pages")]


OK, INVALID, UNSUPPORTED = 0, 1, 2
F32, BF16, F16 = 0, 1, 2
R = ctypes.byref


@pytest.fixture(scope="module")
def L():
    _build.build()
    return kda.lib()


def at(k):
    """A made-up device address, 1 GB from the next."""
    return 0x1000000000 + (k << 30)


def dims(**kw):
    d = dict(num_seqs=2, total_tokens=64, q_heads=8, kv_heads=2, head_dim=128, in_dtype=BF16, out_dtype=BF16, scale=0.1)
    d.update(kw)
    return _Dims(*(d[n] for n, _ in _Dims._fields_))


def cache(**kw):
    c = dict(num_pages=100, page_size=16, max_pages=9)
    c.update(kw)
    return _Cache(*(c[n] for n, _ in _Cache._fields_))


def heads(k, H=8, d=128, **kw):
    h = dict(data=at(k), token_stride=H * d, head_stride=d)
    h.update(kw)
    return _Heads(h["data"], h["token_stride"], h["head_stride"])


def pages(k, H=2, d=128, page=16, **kw):
    p = dict(data=at(k), page_stride=page * H * d, token_stride=H * d, head_stride=d)
    p.update(kw)
    return _Pages(p["data"], p["page_stride"], p["token_stride"], p["head_stride"])


def prefill(L, d=None, **kw):
    a = dict(q=heads(1), k=heads(2, 2), v=heads(3, 2), cu=None, out=at(10), lse=None)
    a.update(kw)
    d = d or dims()
    return L.kda_attn_prefill(R(d), *(R(a[n]) if a[n] else None for n in "qkv"), a["cu"], a["out"], a["lse"], None)


def backward(L, d=None, **kw):
    a = dict(q=heads(1), k=heads(2, 2), v=heads(3, 2), o=heads(4), lse=at(5), y=heads(6), cu=None, dq=at(10), dk=at(11),
             dv=at(12), ws=at(13), size=1 << 20)
    a.update(kw)
    d = d or dims()
    p = lambda n: R(a[n]) if a[n] else None  # noqa: E731
    return L.kda_attn_backward(R(d), p("q"), p("k"), p("v"), p("o"), a["lse"], p("y"), a["cu"], a["dq"], a["dk"], a["dv"],
                               a["ws"], a["size"], None)


def paged(L, d=None, c=None, **kw):
    a = dict(q=heads(1), k=pages(2), v=pages(3), table=at(4), lens=at(5), cu=None, out=at(10), lse=None, ws=at(11),
             size=1 << 30)
    a.update(kw)
    d, c = d or dims(), c or cache()
    p = lambda n: R(a[n]) if a[n] else None  # noqa: E731
    return L.kda_attn_paged(R(d), R(c), p("q"), p("k"), p("v"), a["table"], a["lens"], a["cu"], a["out"], a["lse"], a["ws"],
                            a["size"], None)


BAD_DIMS = [(dict(num_seqs=-1), INVALID), (dict(total_tokens=-1), INVALID), (dict(q_heads=0), INVALID),
            (dict(kv_heads=0), INVALID), (dict(head_dim=0), INVALID), (dict(q_heads=7), INVALID), (dict(in_dtype=3), INVALID),
            (dict(out_dtype=-1), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID),
            (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(num_seqs=3), INVALID),
            (dict(num_seqs=0), INVALID), (dict(in_dtype=F32, out_dtype=F32), UNSUPPORTED), (dict(out_dtype=F16), UNSUPPORTED),
            (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=256), UNSUPPORTED),
            (dict(total_tokens=1 << 28, num_seqs=1), UNSUPPORTED)]


@pytest.mark.parametrize("over,want", BAD_DIMS)
def test_dims_are_refused(L, over, want):
    d = dims(**over)
    assert prefill(L, d) == want and backward(L, d) == want and paged(L, d) == want
    if "num_seqs" not in over:
        assert L.kda_attn_backward_workspace(R(d)) == -1
    assert L.kda_attn_paged_workspace(R(d), R(cache()), None) == -1


BAD_Q = [dict(q=None), dict(q=heads(1, data=None)), dict(q=heads(1, data=at(1) + 8)), dict(q=heads(1, token_stride=1028)),
         dict(q=heads(1, head_stride=132)), dict(q=heads(1, token_stride=120)), dict(q=heads(1, head_stride=64)),
         dict(q=heads(1, token_stride=-1024)), dict(q=heads(1, token_stride=1 << 40)), dict(out=None), dict(out=at(10) + 8),
         dict(lse=at(12) + 2), dict(cu=at(9) + 1), dict(out=at(1) + 64 * 1024 * 2 - 16), dict(lse=at(10) + 1024)]


@pytest.mark.parametrize("over", BAD_Q)
def test_attention_is_refused(L, over):
    assert prefill(L, **over) == INVALID
    assert paged(L, **over) == INVALID


@pytest.mark.parametrize("over", [dict(k=None), dict(v=None), dict(k=heads(2, 2, data=at(2) + 2)),
                                  dict(v=heads(3, 2, token_stride=64)), dict(k=heads(2, 2, head_stride=8)),
                                  dict(out=at(3)), dict(out=at(2) + 1024)])
def test_prompts_are_refused(L, over):
    assert prefill(L, **over) == INVALID
    if "out" not in over:
        assert backward(L, **over) == INVALID


@pytest.mark.parametrize("over", [
    dict(q=None), dict(o=None), dict(y=None), dict(lse=None), dict(lse=at(5) + 2), dict(dq=None), dict(dk=None), dict(dv=None),
    dict(dk=at(11) + 8), dict(ws=None), dict(ws=at(13) + 8), dict(size=64 * 8 * 8 - 1), dict(dq=at(1)), dict(dq=at(11)),
    dict(dv=at(6) + 4096), dict(ws=at(12)), dict(dk=at(5)), dict(y=heads(6, token_stride=1020)), dict(o=heads(4, head_stride=100)),
    dict(cu=at(9) + 2)])
def test_backward_is_refused(L, over):
    assert backward(L, **over) == INVALID


@pytest.mark.parametrize("over", [
    dict(k=None), dict(v=None), dict(k=pages(2, data=at(2) + 2)), dict(v=pages(3, page_stride=100)),
    dict(k=pages(2, token_stride=64)), dict(k=pages(2, page_stride=-4096)), dict(table=None), dict(table=at(4) + 1),
    dict(lens=None), dict(lens=at(5) + 2), dict(ws=None), dict(ws=at(11) + 4), dict(size=4), dict(out=at(2)),
    dict(ws=at(3) + 4096), dict(out=at(4)), dict(lse=at(5))])
def test_paged_is_refused(L, over):
    assert paged(L, **over) == INVALID


@pytest.mark.parametrize("over,want", [
    (dict(num_pages=0), INVALID), (dict(page_size=0), INVALID), (dict(max_pages=0), INVALID), (dict(page_size=4), UNSUPPORTED),
    (dict(page_size=24), UNSUPPORTED), (dict(page_size=2048), UNSUPPORTED), (dict(page_size=1024, max_pages=1 << 21), UNSUPPORTED)])
def test_cache_dims_are_refused(L, over, want):
    c = cache(**over)
    assert paged(L, c=c) == want
    assert L.kda_attn_paged_workspace(R(dims()), R(c), None) == -1
    assert L.kda_cache_workspace(R(c)) == -1
    for call in (reserve, append, free, fork, compact, copy):
        assert call(L, c) == want


def test_empty_batches_are_ok(L):
    for d in (dims(num_seqs=0, total_tokens=0), dims(total_tokens=0)):
        none = dict(q=None, k=None, v=None, out=None)
        assert prefill(L, d, **none) == OK and paged(L, d, **none) == OK
        assert backward(L, d, q=None, k=None, v=None, o=None, y=None, lse=None, dq=None, dk=None, dv=None, ws=None, size=0) == OK
    assert append(L, T=0, k=None, v=None) == OK and free(L, count=0, seqs=None) == OK
    assert fork(L, count=0, parents=None, children=None) == OK and copy(L, count=0, src=None, dst=None) == OK
    assert reserve(L, N=0, table=None, lens=None, new=None) == OK


def reserve(L, c=None, **kw):
    a = dict(N=5, refs=at(1), table=at(2), lens=at(3), new=at(4), src=at(6), dst=at(7), missing=None, ws=at(5), size=1 << 20)
    a.update(kw)
    return L.kda_cache_reserve(R(c or cache()), *a.values(), None)


def append(L, c=None, **kw):
    a = dict(N=5, T=20, H=2, d=128, k=heads(1, 2), v=heads(2, 2), kp=pages(3), vp=pages(4), table=at(5), lens=at(6), cu=None)
    a.update(kw)
    p = lambda n: R(a[n]) if a[n] else None  # noqa: E731
    return L.kda_cache_append(R(c or cache()), a["N"], a["T"], a["H"], a["d"], p("k"), p("v"), p("kp"), p("vp"), a["table"],
                              a["lens"], a["cu"], None)


def free(L, c=None, **kw):
    a = dict(N=5, refs=at(1), table=at(2), lens=at(3), count=4, seqs=at(4), keep=None)
    a.update(kw)
    return L.kda_cache_free(R(c or cache()), *a.values(), None)


def fork(L, c=None, **kw):
    a = dict(N=5, refs=at(1), table=at(2), lens=at(3), count=2, parents=at(4), children=at(5), src=at(6), dst=at(7),
             missing=None, ws=at(8), size=1 << 20)
    a.update(kw)
    return L.kda_cache_fork(R(c or cache()), *a.values(), None)


def compact(L, c=None, **kw):
    a = dict(N=5, refs=at(1), table=at(2), lens=at(3), refs_out=at(4), table_out=at(5), src=at(6), dst=at(7), ws=at(8),
             size=1 << 20)
    a.update(kw)
    return L.kda_cache_compact(R(c or cache()), *a.values(), None)


def copy(L, c=None, **kw):
    a = dict(H=2, d=128, kp=pages(1), vp=pages(2), count=3, src=at(3), dst=at(4))
    a.update(kw)
    p = lambda n: R(a[n]) if a[n] else None  # noqa: E731
    return L.kda_cache_copy(R(c or cache()), a["H"], a["d"], p("kp"), p("vp"), a["count"], a["src"], a["dst"], None)


@pytest.mark.parametrize("call,over", [
    (reserve, o) for o in (dict(N=-1), dict(refs=None), dict(table=None), dict(lens=None), dict(new=None), dict(refs=at(1) + 2),
                           dict(missing=at(9) + 1), dict(ws=None), dict(ws=at(5) + 8), dict(size=100), dict(new=at(3)),
                           dict(lens=at(2)), dict(ws=at(1)), dict(missing=at(3) + 4), dict(src=None), dict(dst=None),
                           dict(dst=at(6) + 4), dict(src=at(6) + 2))] + [
    (append, o) for o in (dict(N=-1), dict(T=-1), dict(T=21), dict(H=0), dict(d=0), dict(k=None), dict(v=None), dict(kp=None),
                          dict(vp=None), dict(table=None), dict(lens=None), dict(lens=at(6) + 2), dict(cu=at(7) + 2),
                          dict(k=heads(1, 2, data=at(1) + 4)), dict(v=heads(2, 2, token_stride=12)),
                          dict(kp=pages(3, token_stride=128)), dict(kp=pages(3, page_stride=256)),
                          dict(kp=pages(3, data=at(1))), dict(vp=pages(4, data=at(3))), dict(table=at(4)))] + [
    (free, o) for o in (dict(N=-1), dict(refs=None), dict(table=None), dict(lens=None), dict(seqs=None), dict(count=-1),
                        dict(keep=at(5) + 1), dict(seqs=at(2)), dict(keep=at(3)), dict(table=at(1)))] + [
    (fork, o) for o in (dict(N=-1), dict(refs=None), dict(table=None), dict(lens=None), dict(parents=None), dict(children=None),
                        dict(src=None), dict(dst=None), dict(count=-1), dict(ws=None), dict(size=8), dict(src=at(7)),
                        dict(parents=at(6)), dict(missing=at(8)), dict(children=at(5) + 2))] + [
    (compact, o) for o in (dict(N=-1), dict(refs=None), dict(table=None), dict(lens=None), dict(refs_out=None),
                           dict(table_out=None), dict(src=None), dict(dst=None), dict(ws=None), dict(size=8),
                           dict(refs_out=at(1) + 4), dict(table_out=at(2) + 4), dict(src=at(7) + 8), dict(ws=at(3)),
                           dict(refs_out=at(5)))] + [
    (copy, o) for o in (dict(H=0), dict(d=-8), dict(kp=None), dict(vp=None), dict(count=-1), dict(src=None), dict(dst=None),
                        dict(src=at(3) + 2), dict(dst=at(2)), dict(vp=pages(1)), dict(kp=pages(1, head_stride=100)))])
def test_cache_calls_are_refused(L, call, over):
    assert call(L, **over) == INVALID


@pytest.mark.parametrize("call", [append, copy])
@pytest.mark.parametrize("d", [4, 12, 2048])
def test_head_sizes_are_refused(L, call, d):
    assert call(L, d=d) == UNSUPPORTED


def test_workspaces(L):
    """One token: shares for one wave of blocks; many tokens in many blocks: bounded."""
    one = L.kda_attn_paged_workspace(R(dims(num_seqs=1, total_tokens=1)), R(cache()), None)
    assert 0 < one < 4 << 20
    many = L.kda_attn_paged_workspace(R(dims(num_seqs=1, total_tokens=100000)), R(cache()), None)
    assert 0 < many < 200 << 20
    assert L.kda_attn_backward_workspace(R(dims())) == 64 * 8 * 8
    assert L.kda_cache_workspace(R(cache())) >= 400


def test_binding_refuses():
    """What the binding sees by itself (CPU tensors, shapes, types)."""
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_attn_prefill(x, x, x)
    with pytest.raises(ValueError):
        kda.kda_attn_prefill(x, x[0], x)
    with pytest.raises(ValueError, match="needed"):
        kda.kda_attn_backward(x, x, x, None, None, x)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_attn_backward(x, x, x, x, torch.zeros(4, 2), x)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        kda.kda_attn_paged(x, x, x, i, i)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_attn_paged(x, torch.zeros(3, 8, 2, 64, dtype=torch.bfloat16), x, i[:, None], i)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_cache_reserve(i, i[:, None], i, i, 16)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_cache_append(x, x, torch.zeros(3, 8, 2, 64, dtype=torch.bfloat16), x, i[:, None], i)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_cache_copy(torch.zeros(3, 8, 2, 64, dtype=torch.bfloat16), x, i, i)


def test_more_blocks_than_a_grid_holds(L):
    """Every sequence has a block a query head at the least in the gradients: 2^20 of them with
    4096 heads are more than 2^31 blocks, and a number that wraps would be a grid of few."""
    d = dims(num_seqs=1 << 20, total_tokens=16, q_heads=4096, kv_heads=1)
    q, k = heads(1, 4096), heads(2, 1)
    cu = at(14)
    assert L.kda_attn_backward_workspace(R(d)) == -1
    assert backward(L, d, q=q, k=k, v=heads(3, 1), o=heads(4, 4096), y=heads(6, 4096), cu=cu) == UNSUPPORTED
    assert prefill(L, d, q=q, k=k, v=heads(3, 1), cu=cu) == UNSUPPORTED
    assert paged(L, d, q=q, k=pages(2, 1), v=pages(3, 1), cu=cu) == UNSUPPORTED
