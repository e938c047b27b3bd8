"""GPU tests of a cache whose reservations are refused: pages that run out, table rows that are full, shared
pages that cannot be replaced.  What a refused sequence had stays, bit by bit, in its own
pages and in those that it shares, and its new tokens see nothing."""
import math

import pytest
import torch

import linear_attention_sequence_gb300 as kda
from test_attn_gpu import BF16, DEV, F16, F32, check_paged, cu_of, rnd, starts

pytestmark = pytest.mark.gpu
INVALID = 1


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Cache:
    """One layer's pages and the state, and beside them each sequence's history."""

    def __init__(self, P, N, wide, page, H, d, dtype):
        self.page, self.N = page, N
        self.refs = torch.zeros(P, dtype=torch.int32, device=DEV)
        self.table = torch.full((N, wide), -1, dtype=torch.int32, device=DEV)
        self.lens = torch.zeros(N, dtype=torch.int32, device=DEV)
        self.kp, self.vp = (torch.full((P, page, H, d), float("nan"), device=DEV, dtype=dtype) for _ in range(2))
        none = torch.zeros(0, H, d, device=DEV, dtype=dtype)
        self.ks, self.vs = [none] * N, [none] * N

    @property
    def state(self):
        return self.refs, self.table, self.lens

    def held(self):
        """What the pages hold of each sequence."""
        for n in range(self.N):
            L = int(self.lens[n])
            pages = self.table[n, :-(-L // self.page)].long()
            yield (self.kp[pages].flatten(0, 1)[:L], self.vp[pages].flatten(0, 1)[:L])

    def add(self, new, k, v, granted):
        at = starts(new)
        for n in range(self.N):
            if granted[n] == new[n]:
                self.ks[n] = torch.cat([self.ks[n], k[at[n]:at[n + 1]]])
                self.vs[n] = torch.cat([self.vs[n], v[at[n]:at[n + 1]]])

    def check(self):
        assert self.lens.tolist() == [x.shape[0] for x in self.ks]
        for n, (k, v) in enumerate(self.held()):
            assert torch.equal(k, self.ks[n]) and torch.equal(v, self.vs[n]), f"sequence {n}"


def step(c, new, seed, H, copies=True):
    """Reserve, append, attend; returns granted."""
    Hkv, d = c.kp.shape[2:]
    T, N = sum(new), c.N
    got = kda.kda_cache_reserve(*c.state, ints(new), c.page, return_copies=copies, return_granted=True)
    if copies:
        src, dst, granted = got
        kda.kda_cache_copy(c.kp, c.vp, src, dst)
    else:
        granted = got
    k, v, q = rnd(seed, c.kp.dtype, T, Hkv, d), rnd(seed + 1, c.kp.dtype, T, Hkv, d), rnd(seed + 2, c.kp.dtype, T, H, d)
    cu = None if len(set(new)) == 1 else cu_of(new)
    kda.kda_cache_append(k, v, c.kp, c.vp, c.table, c.lens, cu, granted=granted)
    g = granted.tolist()
    assert all(x in (0, max(0, y)) for x, y in zip(g, new))
    c.add(new, k, v, g)
    c.check()
    out, lse = kda.kda_attn_paged(q, c.kp, c.vp, c.table, c.lens, cu, granted=granted, out_dtype=F32, return_lse=True)
    at = starts(new)
    for n in range(N):
        part = slice(at[n], at[n + 1])
        if g[n] == new[n]:
            check_paged(out[part], lse[part], q[part], [new[n]], [c.ks[n].shape[0]], [c.ks[n]], [c.vs[n]])
        else:
            assert bool((out[part] == 0).all()) and bool((lse[part] == -math.inf).all())
    return g


@pytest.mark.parametrize("H,Hkv,d,dtype", [(4, 2, 64, BF16), (16, 1, 128, F16)])
@pytest.mark.parametrize("new", [1, 3, 20])
def test_pages_run_out(new, H, Hkv, d, dtype):
    """Children that share full pages with their parent, and two free pages."""
    c = Cache(5, 4, 8, 8, Hkv, d, dtype)
    step(c, [16, 0, 0, 5], 10, H)                         # pages 0, 1 and 2
    kda.kda_cache_fork(*c.state, ints([0, 0]), ints([1, 2]), 8)
    c.ks[1] = c.ks[2] = c.ks[0]
    c.vs[1] = c.vs[2] = c.vs[0]
    c.check()
    tail = 0 if new > 3 else new                          # (sequence 3 has room for 3 more)
    served = 0 if new > 16 else 2                         # pages of 8 for each, in their order
    assert step(c, [new, new, new, tail], 20, H) == [new if i < served else 0 for i in range(3)] + [tail]
    assert step(c, [0, 0, 8, 8], 30, H) == [0, 0] + ([0, 0] if served else [8, 8])
    assert kda.kda_get_last_device_error() == 0           # who asks what was granted is told


def test_row_is_full():
    """A sequence as long as its row: pages are left, and nothing is counted as lacking."""
    c = Cache(9, 2, 2, 16, 1, 64, BF16)
    step(c, [32, 3], 40, 2)
    missing = ints([-1])
    kda.kda_cache_reserve(*c.state, ints([1, 0]), 16, missing=missing)
    assert missing.item() == 0 and c.lens.tolist() == [32, 3]
    for i in range(15):
        assert step(c, [1, 1], 50 + 3 * i, 2) == [0, 1]
    assert kda.kda_get_last_device_error() == 0


def test_shared_page_without_lists():
    """A sequence shortened into a page that another shares, and nowhere to say what to copy."""
    c = Cache(9, 2, 3, 8, 1, 64, BF16)
    step(c, [16, 0], 70, 1)
    kda.kda_cache_fork(*c.state, ints([0]), ints([1]), 8)
    kda.kda_cache_free(*c.state, ints([1]), 8, keep=ints([5]))
    c.ks[1], c.vs[1] = c.ks[0][:5], c.vs[0][:5]
    c.check()
    assert step(c, [2, 2], 80, 1, copies=False) == [2, 0]
    assert kda.kda_get_last_device_error() == INVALID
    assert step(c, [2, 2], 90, 1) == [2, 2]
    assert kda.kda_get_last_device_error() == 0


def test_padded_batch():
    """A token for every row of the batch, sequences that pause and empty rows among them: they were granted
    none, and keep what they have."""
    c = Cache(12, 4, 3, 8, 2, 64, BF16)
    step(c, [8, 3, 0, 16], 100, 4)
    one = ints([1, 0, 0, 1])
    for i in range(6):
        granted = kda.kda_cache_reserve(*c.state, one, 8, return_granted=True)
        k, v, q = rnd(110 + i, BF16, 4, 2, 64), rnd(120 + i, BF16, 4, 2, 64), rnd(130 + i, BF16, 4, 4, 64)
        kda.kda_cache_append(k, v, c.kp, c.vp, c.table, c.lens, granted=granted)
        assert granted.tolist() == [1, 0, 0, 1]
        c.add([1, 1, 1, 1], k, v, [1, 0, 0, 1])
        c.check()
        out = kda.kda_attn_paged(q, c.kp, c.vp, c.table, c.lens, granted=granted, out_dtype=F32)
        assert bool((out[1:3] == 0).all())
        for n in (0, 3):
            check_paged(out[n:n + 1], None, q[n:n + 1], [1], [c.ks[n].shape[0]], [c.ks[n]], [c.vs[n]])


def test_captured_loop_that_runs_out():
    """A decode step captured once and replayed until nothing is left: lengths stop, histories stay."""
    N, H, Hkv, d, page, P = 3, 4, 2, 64, 8, 7
    c = Cache(P, N, 4, page, Hkv, d, BF16)
    step(c, [7, 16, 1], 200, H)
    one, granted, missing = ints([1] * N), ints([0] * N), ints([0])
    q, k, v = (torch.empty(N, h, d, device=DEV, dtype=BF16) for h in (H, Hkv, Hkv))
    out = torch.empty(N, H, d, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_cache_reserve(*c.state, one, page, granted=granted, missing=missing)
        kda.kda_cache_append(k, v, c.kp, c.vp, c.table, c.lens, granted=granted)
        kda.kda_attn_paged(q, c.kp, c.vp, c.table, c.lens, granted=granted, out=out, out_dtype=F32)
    for t in range(25):
        for i, x in enumerate((q, k, v)):
            x.copy_(rnd(210 + 3 * t + i, BF16, *x.shape))
        graph.replay()
        g = granted.tolist()
        c.add([1] * N, k.clone(), v.clone(), g)
        c.check()
        for n in range(N):
            if g[n]:
                check_paged(out[n:n + 1], None, q[n:n + 1], [1], [c.ks[n].shape[0]], [c.ks[n]], [c.vs[n]])
            else:
                assert bool((out[n] == 0).all())
    assert g == [0] * N and missing.item() > 0 and int((c.refs > 0).sum()) == P


def test_refusals_are_recorded_where_nobody_asks():
    for P, wide in ((1, 9), (9, 1)):
        c = Cache(P, 1, wide, 8, 1, 64, BF16)
        kda.kda_cache_reserve(*c.state, ints([9]), 8)
        assert kda.kda_get_last_device_error() == INVALID and c.lens.item() == 0 and bool((c.refs == 0).all())
        kda.kda_cache_reserve(*c.state, ints([8]), 8)
        assert kda.kda_get_last_device_error() == 0 and c.lens.item() == 8


def test_many_sequences_are_granted():
    """More sequences than the block has threads."""
    N = 2500
    c = Cache(1000, N, 3, 8, 1, 64, BF16)
    new = [(7 * n) % 30 - 2 for n in range(N)]
    granted = kda.kda_cache_reserve(*c.state, ints(new), 8, return_granted=True).tolist()
    left, want = 1000, []
    for x in new:
        need = -(-max(0, x) // 8)
        if need > 3:
            want.append(0)
            continue
        left -= need
        want.append(max(0, x) if left >= 0 or need == 0 else 0)
    assert granted == want == c.lens.tolist()


def test_binding_refuses():
    """What was granted: int32 [N], contiguous, on the cache's device."""
    c = Cache(9, 3, 3, 8, 1, 64, BF16)
    new, x = ints([1, 1, 1]), rnd(1, BF16, 3, 1, 64)
    for bad in (ints([1, 1]), ints([1, 1, 1]).long(), ints([1] * 6)[::2], torch.ones(3, dtype=torch.int32)):
        with pytest.raises((ValueError, kda.KdaError)):
            kda.kda_cache_reserve(*c.state, new, 8, granted=bad)
        with pytest.raises((ValueError, kda.KdaError)):
            kda.kda_cache_append(x, x, c.kp, c.vp, c.table, c.lens, granted=bad)
        with pytest.raises((ValueError, kda.KdaError)):
            kda.kda_attn_paged(x, c.kp, c.vp, c.table, c.lens, granted=bad)
    with pytest.raises(kda.KdaError):
        kda.kda_cache_reserve(*c.state, new, 8, granted=new)
    c.check()
