"""GPU tests of the calls on the pages of a cache, against the same bookkeeping in Python lists.
Whole numbers and moved values are compared exactly."""
import random

import pytest
import torch

import linear_attention_sequence_gb300 as kda

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, F16 = torch.bfloat16, torch.float16


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Plain:
    """The documented rules, one entry at a time."""

    def __init__(self, P, N, wide, page):
        self.P, self.N, self.wide, self.page = P, N, wide, page
        self.refs, self.table, self.lens = [0] * P, [[-1] * wide for _ in range(N)], [0] * N

    def pages(self, n):
        return -(-n // self.page)

    def free_list(self):
        return [p for p in range(self.P) if self.refs[p] == 0]

    def reserve(self, new):
        free, upto, src, dst = self.free_list(), 0, [-1] * self.N, [-1] * self.N
        last = [self.table[n][self.lens[n] // self.page] if self.lens[n] % self.page else -1 for n in range(self.N)]
        shared = [p >= 0 and self.refs[p] > 1 for p in last]
        for n, add in enumerate(new):
            add = max(0, add)
            have, want = self.pages(self.lens[n]), self.pages(self.lens[n] + add)
            if want > self.wide:
                continue
            copies = add > 0 and shared[n]
            need = want - have + copies
            at, upto = upto, upto + need
            if need and upto > len(free):
                continue
            if copies:
                src[n], dst[n] = last[n], free[at]
                self.refs[last[n]] -= 1
                have -= 1
            for j in range(have, want):
                p = free[at + j - have]
                self.table[n][j], self.refs[p] = p, 1
            self.lens[n] += add
        return max(0, upto - len(free)), src, dst

    def free(self, seqs, keep=None):
        for i, n in enumerate(seqs):
            left = max(0, keep[i]) if keep else 0
            if self.lens[n] <= left:
                continue
            for j in range(self.pages(left), self.pages(self.lens[n])):
                self.refs[self.table[n][j]] -= 1
                self.table[n][j] = -1
            self.lens[n] = left

    def fork(self, parents, children):
        free, upto, src, dst = self.free_list(), 0, [], []
        for p, c in zip(parents, children):
            whole, part = divmod(self.lens[p], self.page)
            at, upto = upto, upto + (part > 0)
            self.table[c] = [-1] * self.wide
            if part and upto > len(free):
                self.lens[c] = 0
                src.append(-1), dst.append(-1)
                continue
            self.lens[c] = self.lens[p]
            for j in range(whole):
                self.table[c][j] = self.table[p][j]
                self.refs[self.table[p][j]] += 1
            if part:
                q = free[at]
                self.table[c][whole], self.refs[q] = q, 1
                src.append(self.table[p][whole]), dst.append(q)
            else:
                src.append(-1), dst.append(-1)
        return src, dst, max(0, upto - len(free))

    def compact(self):
        live = sum(r > 0 for r in self.refs)
        src = [p for p in range(live, self.P) if self.refs[p] > 0]
        dst = [p for p in range(live) if self.refs[p] == 0]
        to = dict(zip(src, dst))
        for s, d in to.items():
            self.refs[d], self.refs[s] = self.refs[s], 0
        for n in range(self.N):
            for j in range(self.pages(self.lens[n])):
                self.table[n][j] = to.get(self.table[n][j], self.table[n][j])
        pad = [-1] * (self.P - len(src))
        return src + pad, dst + pad


class Both:
    """The same calls on both sides, compared after each."""

    def __init__(self, P, N, wide, page):
        self.plain, self.page = Plain(P, N, wide, page), page
        self.refs = torch.zeros(P, dtype=torch.int32, device=DEV)
        self.table = torch.full((N, wide), -1, dtype=torch.int32, device=DEV)
        self.lens = torch.zeros(N, dtype=torch.int32, device=DEV)
        self.missing = ints([-5])

    @property
    def state(self):
        return self.refs, self.table, self.lens

    def check(self):
        assert self.lens.tolist() == self.plain.lens
        assert self.table.tolist() == self.plain.table
        assert self.refs.tolist() == self.plain.refs
        # what the counts say is what the table says
        used = [0] * self.plain.P
        for n, row in enumerate(self.plain.table):
            assert all(p == -1 for p in row[self.plain.pages(self.plain.lens[n]):])
            for p in row:
                if p >= 0:
                    used[p] += 1
        assert used == self.plain.refs

    def reserve(self, new):
        src, dst = kda.kda_cache_reserve(*self.state, ints(new), self.page, missing=self.missing, return_copies=True)
        want, s, d = self.plain.reserve(new)
        self.check()
        assert self.missing.item() == want and src.tolist() == s and dst.tolist() == d

    def free(self, seqs, keep=None):
        kda.kda_cache_free(*self.state, ints(seqs), self.page, keep=None if keep is None else ints(keep))
        self.plain.free(seqs, keep)
        self.check()

    def fork(self, parents, children):
        src, dst = kda.kda_cache_fork(*self.state, ints(parents), ints(children), self.page, missing=self.missing)
        s, d, want = self.plain.fork(parents, children)
        self.check()
        assert src.tolist() == s and dst.tolist() == d and self.missing.item() == want
        return src, dst

    def compact(self, in_place):
        was = [x.clone() for x in self.state]
        kw = dict(refs_out=self.refs, table_out=self.table) if in_place else {}
        refs, table, src, dst = kda.kda_cache_compact(*self.state, self.page, **kw)
        if not in_place:
            assert all(torch.equal(a, b) for a, b in zip(was, self.state))   # the inputs stay
        self.refs, self.table = refs, table
        s, d = self.plain.compact()
        self.check()
        assert src.tolist() == s and dst.tolist() == d
        return src, dst


@pytest.mark.parametrize("P,N,wide,page", [(1, 1, 1, 8), (7, 3, 4, 16), (300, 20, 40, 16), (5000, 60, 130, 8),
                                           (40000, 1500, 33, 64), (70001, 5, 2000, 8)])
@pytest.mark.parametrize("seed", [1, 2])
def test_bookkeeping(P, N, wide, page, seed):
    """Calls in any order, with too few pages and rows that are too short among them."""
    r = random.Random(seed * 1000 + P)
    c = Both(P, N, wide, page)
    for step in range(14):
        kind = r.choice(["reserve", "reserve", "free", "fork", "compact"]) if step > 1 else "reserve"
        if kind == "reserve":
            most = max(1, int(2.5 * P * page / N / 4))
            c.reserve([r.choice([0, 1, r.randint(0, most), r.randint(-3, 3 * page)]) for _ in range(N)])
        elif kind == "free":
            seqs = [r.randrange(N) for _ in range(r.randint(1, N))]      # some of them twice
            keep = [r.choice([0, -1, r.randint(0, wide * page)]) for _ in seqs] if r.random() < 0.6 else None
            c.free(seqs, keep)
        elif kind == "fork":
            full = [n for n in range(N) if c.plain.lens[n]]
            empty = [n for n in range(N) if not c.plain.lens[n]]
            if full and empty:
                r.shuffle(empty)
                children = empty[:r.randint(1, len(empty))]
                c.fork([r.choice(full) for _ in children], children)
        else:
            c.compact(r.random() < 0.5)
    c.compact(True)
    assert kda.kda_get_last_device_error() == 0


def test_shared_pages_that_grow():
    """Continuations cut back into the page they share: each gets one of its own, and without
    lists for the copies none is served."""
    c = Both(20, 5, 6, 8)
    c.reserve([30, 0, 0, 0, 7])
    c.fork([0, 0], [1, 2])
    c.free([0, 1, 2], [21, 13, 16])
    c.reserve([1, 4, 0, 9, 1])
    c.free([0, 1], [5, 5])                                       # both in the page of tokens 0..7, and 2 has it too
    before = [x.clone() for x in c.state]
    kda.kda_cache_reserve(*c.state, ints([3, 0, 0, 0, 0]), 8)
    assert kda.kda_get_last_device_error() == 1
    assert all(torch.equal(a, b) for a, b in zip(before, c.state))
    kda.kda_cache_reserve(*c.state, ints([0, 0, 3, 0, 0]), 8)    # 2 ends with a full page: nothing to copy
    c.plain.reserve([0, 0, 3, 0, 0])
    c.check()
    c.reserve([3, 3, 0, 0, 0])


def test_aligned_or_not():
    """Counts that do not start on 16 bytes."""
    c = Both(3000, 4, 800, 8)
    c.refs = torch.zeros(3001, dtype=torch.int32, device=DEV)[1:]
    c.reserve([5000, 40, 0, 7])
    c.free([0, 1], [100, 9])
    c.reserve([0, 900, 3000, 0])
    c.compact(False)


def layer(P, page, H, d, dtype, order, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device=DEV).to(dtype)  # noqa: E731
    if order == "NHD":
        return rnd(P, page, H, d), rnd(P, page, H, d)
    if order == "HND":
        return rnd(P, H, page, d).transpose(1, 2), rnd(P, H, page, d).transpose(1, 2)
    both = rnd(P, 2, page, H, d)                     # keys and values of a page side by side
    return both[:, 0], both[:, 1]


@pytest.mark.parametrize("order", ["NHD", "HND", "both"])
@pytest.mark.parametrize("P,page,H,d,dtype", [(5, 8, 1, 64, BF16), (40, 16, 3, 64, F16), (300, 64, 8, 128, BF16),
                                              (9, 1024, 2, 128, F16), (33, 32, 5, 8, BF16)])
def test_copy(P, page, H, d, dtype, order):
    k, v = layer(P, page, H, d, dtype, order, P)
    gen = torch.Generator().manual_seed(P)
    perm = torch.randperm(P, generator=gen)
    m = P // 2
    src, dst = perm[:m].tolist(), perm[m:2 * m].tolist()
    src[::3] = [src[0]] * len(src[::3])              # one page to several
    want_k, want_v = k.clone(), v.clone()
    for a, b in zip(src, dst):
        want_k[b], want_v[b] = k[a], v[a]
    src += [-1, -1]
    dst += [-1, -1]
    kda.kda_cache_copy(k, v, ints(src), ints(dst))
    assert torch.equal(k, want_k) and torch.equal(v, want_v)
    assert kda.kda_get_last_device_error() == 0


@pytest.mark.parametrize("order", ["NHD", "HND", "both"])
@pytest.mark.parametrize("page,H,d,dtype", [(8, 1, 64, BF16), (16, 3, 64, F16), (64, 8, 128, BF16), (128, 2, 24, F16)])
@pytest.mark.parametrize("had,new", [([0], [1]), ([5, 0, 63, 100], [1, 1, 1, 1]), ([0, 7, 130, 64, 9], [300, 0, 1, 64, 0]),
                                     ([0] * 70, [3] * 70)])
def test_append(had, new, page, H, d, dtype, order):
    N = len(had)
    total = [a + b for a, b in zip(had, new)]
    c = Both(sum(-(-t // page) for t in total) + 3, N, max(-(-t // page) for t in total) + 1, page)
    c.reserve(had)
    c.reserve(new)
    assert c.lens.tolist() == total
    k_pages, v_pages = layer(c.plain.P, page, H, d, dtype, order, 3)
    want_k, want_v = k_pages.clone(), v_pages.clone()
    T = sum(new)
    gen = torch.Generator(device=DEV).manual_seed(9)
    rows = torch.randn((T, 2 * H + 1, d), generator=gen, device=DEV).to(dtype)
    k, v = rows[:, :H], rows[:, H + 1:]
    t = 0
    for n in range(N):
        for i in range(had[n], total[n]):
            p = c.plain.table[n][i // page]
            want_k[p, i % page], want_v[p, i % page] = k[t], v[t]
            t += 1
    cu = None
    if len(set(new)) > 1:
        cu = [0]
        for x in new:
            cu.append(cu[-1] + x)
        cu = ints(cu)
    kda.kda_cache_append(k, v, k_pages, v_pages, c.table, c.lens, cu)
    assert torch.equal(k_pages, want_k) and torch.equal(v_pages, want_v)
    assert kda.kda_get_last_device_error() == 0
