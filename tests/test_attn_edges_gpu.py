"""GPU tests of softmax attention and its cache at their edges: strides, rows without
sequences, values that must not be seen, scores that grow, graphs and streams, offsets past 32
bits, bad pages, and a run of all calls together.  Bounds as in attn_reference.py."""
import random

import pytest
import torch

import linear_attention_sequence_gb300 as kda
from attn_reference import U, backward as ref_backward, backward_bounds, rows
from test_attn_gpu import (BF16, DEV, F16, F32, check_backward, check_paged, check_prompts, cu_of, make_cache,
                           prompt_inputs, rnd, starts)

pytestmark = pytest.mark.gpu
INVALID = 1


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.fixture(autouse=True)
def status():
    """No bounded wait gave up, and nothing was out of range (but where a test says so)."""
    kda.kda_get_last_device_error()
    yield
    assert kda.kda_get_last_device_error() == 0


# ------------------------------------------------------------------ layouts

def fused(T, H, Hkv, d, dtype, seed):
    """q, k, v as slices of one projection's rows."""
    x = rnd(seed, dtype, T, H + 2 * Hkv, d)
    return x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]


def by_heads(T, H, Hkv, d, dtype, seed):
    """Heads before tokens."""
    return tuple(rnd(seed + i, dtype, h, T, d).transpose(0, 1) for i, h in enumerate((H, Hkv, Hkv)))


def padded(T, H, Hkv, d, dtype, seed):
    """Rows and heads with gaps, from an address that is a multiple of 16 bytes only."""
    def one(i, h):
        x = rnd(seed + i, dtype, (T + 1) * (h * (d + 8) + 24) + 8)[8:]
        return torch.as_strided(x, (T, h, d), (h * (d + 8) + 24, d + 8, 1), x.storage_offset())
    return one(0, H), one(1, Hkv), one(2, Hkv)


@pytest.mark.parametrize("layout", [fused, by_heads, padded])
@pytest.mark.parametrize("d,dtype", [(128, BF16), (64, F16)])
def test_strides(layout, d, dtype):
    lens, H, Hkv = [130, 0, 77, 300], 6, 2
    q, k, v = layout(sum(lens), H, Hkv, d, dtype, 31)
    dy = layout(sum(lens), H, Hkv, d, dtype, 41)[0]
    cu = cu_of(lens)
    out, lse = kda.kda_attn_prefill(q, k, v, cu, out_dtype=F32, return_lse=True)
    check_prompts(out, lse, q, k, v, lens)
    plain = [x.contiguous() for x in (q, k, v)]
    assert torch.equal(out, kda.kda_attn_prefill(*plain, cu, out_dtype=F32))
    o16 = out.to(dtype)
    g = kda.kda_attn_backward(q, k, v, o16, lse, dy, cu, grad_dtype=F32)
    want = kda.kda_attn_backward(*plain, o16, lse, dy.contiguous(), cu, grad_dtype=F32)
    assert all(torch.equal(g[n], want[n]) for n in g)


@pytest.mark.parametrize("order", ["HND", "both"])
@pytest.mark.parametrize("new,total", [([1, 1, 1], [1, 300, 4000]), ([40, 0, 300], [40, 7, 3000])])
def test_cache_layouts(new, total, order):
    H, Hkv, d, page = 8, 2, 128, 32
    kp, vp, table, lens, ks, vs = make_cache(total, Hkv, d, page, BF16, 51, order="HND" if order == "HND" else "NHD")
    if order == "both":
        both = torch.stack([kp, vp], 1)
        kp, vp = both[:, 0], both[:, 1]
    q = fused(sum(new), H, Hkv, d, BF16, 52)[0]
    out, lse = kda.kda_attn_paged(q, kp, vp, table, lens, cu_of(new), out_dtype=F32, return_lse=True)
    check_paged(out, lse, q, new, total, ks, vs)


@pytest.mark.parametrize("page", [8, 128, 1024])
@pytest.mark.parametrize("H,Hkv,d,dtype", [(300, 1, 64, BF16), (17, 1, 128, F16), (16, 1, 128, BF16), (2, 2, 64, F16)])
def test_groups_and_pages(H, Hkv, d, dtype, page):
    """Groups of more rows than a tile, and of just as many as the kernel of few rows takes."""
    new, total = [1, 2, 30, 1], [1, 1025, 2050, 128]
    kp, vp, table, lens, ks, vs = make_cache(total, Hkv, d, page, dtype, 61)
    q = rnd(62, dtype, sum(new), H, d)
    out, lse = kda.kda_attn_paged(q, kp, vp, table, lens, cu_of(new), out_dtype=F32, return_lse=True)
    check_paged(out, lse, q, new, total, ks, vs)
    T = 40
    q, k, v = prompt_inputs(T, H, Hkv, d, dtype, 63)
    out, lse = kda.kda_attn_prefill(q, k, v, out_dtype=F32, return_lse=True)
    check_prompts(out, lse, q, k, v, [T])


def test_equal_sequences_without_offsets():
    N, L, H, Hkv, d = 5, 150, 4, 2, 64
    q, k, v = prompt_inputs(N * L, H, Hkv, d, BF16, 71)
    dy = rnd(72, BF16, N * L, H, d)
    a = kda.kda_attn_prefill(q, k, v, num_seqs=N, return_lse=True)
    b = kda.kda_attn_prefill(q, k, v, cu_of([L] * N), return_lse=True)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    ga = kda.kda_attn_backward(q, k, v, *a, dy, num_seqs=N)
    gb = kda.kda_attn_backward(q, k, v, *a, dy, cu_of([L] * N))
    assert all(torch.equal(ga[n], gb[n]) for n in ga)


def test_many_sequences():
    """More sequences than a block has threads, most of them short, many empty."""
    r = random.Random(5)
    lens = [r.choice([0, 0, 1, 2, 5]) for _ in range(1500)] + [300] + [1] * 200
    H, Hkv, d = 4, 2, 64
    q, k, v = prompt_inputs(sum(lens), H, Hkv, d, BF16, 81)
    cu = cu_of(lens)
    out, lse = kda.kda_attn_prefill(q, k, v, cu, out_dtype=F32, return_lse=True)
    at = starts(lens)
    some = [n for n in range(len(lens)) if lens[n] and n % 37 == 0] + [1500]
    for n in some:
        part = slice(at[n], at[n + 1])
        check_prompts(out[part], lse[part], q[part], k[part], v[part], [lens[n]])
    dy = rnd(82, BF16, sum(lens), H, d)
    g = kda.kda_attn_backward(q, k, v, out.to(BF16), lse, dy, cu, grad_dtype=F32)
    for n in some:
        part = slice(at[n], at[n + 1])
        check_backward({m: x[part] for m, x in g.items()}, q[part], k[part], v[part], out[part].to(BF16), lse[part], dy[part],
                       [lens[n]])
    # the same as chunks over a cache, lengths of 0 and more than the new tokens among them
    total = [n + r.choice([0, 0, 3, 40]) for n in lens]
    kp, vp, table, kv_lens, ks, vs = make_cache(total, Hkv, d, 16, BF16, 83)
    out, lse = kda.kda_attn_paged(q, kp, vp, table, kv_lens, cu, out_dtype=F32, return_lse=True)
    for n in some:
        part = slice(at[n], at[n + 1])
        check_paged(out[part], lse[part], q[part], [lens[n]], [total[n]], [ks[n]], [vs[n]])


# ------------------------------------------------------------------ rows without sequences

@pytest.mark.parametrize("first,lens", [(0, [40, 0, 100]), (7, [40, 100]), (200, []), (3, [0, 0]), (0, [129])])
def test_rows_without_sequences(first, lens):
    """Rows before the first sequence and behind the last stay as they were, whatever they hold."""
    T, H, Hkv, d = first + sum(lens) + 33, 4, 2, 64
    q, k, v = prompt_inputs(T, H, Hkv, d, BF16, 91)
    dy = rnd(92, BF16, T, H, d)
    used = slice(first, first + sum(lens))
    for x in (q, k, v, dy):
        keep = x[used].clone()
        x.fill_(float("nan"))
        x[used] = keep
    cu = cu_of(lens, first)
    out, lse = torch.full((T, H, d), 7.0, device=DEV), torch.full((T, H), 7.0, device=DEV)
    kda.kda_attn_prefill(q, k, v, cu, out=out, lse=lse, out_dtype=F32)
    check_prompts(out, lse, q, k, v, lens, first)
    grads = {n: torch.full((T, h, d), 7.0, device=DEV) for n, h in (("dq", H), ("dk", Hkv), ("dv", Hkv))}
    o16 = torch.where(torch.arange(T, device=DEV)[:, None, None] < 0, 0.0, out).to(BF16)
    kda.kda_attn_backward(q, k, v, o16, lse, dy, cu, grad_dtype=F32, **grads)
    check_backward(grads, q, k, v, o16, lse, dy, lens, first)
    total = [n + 50 for n in lens]
    kp, vp, table, kv_lens, ks, vs = make_cache(total, Hkv, d, 16, BF16, 93)
    pout, plse = torch.full((T, H, d), 7.0, device=DEV), torch.full((T, H), 7.0, device=DEV)
    if lens:
        kda.kda_attn_paged(q, kp, vp, table, kv_lens, cu, out=pout, lse=plse, out_dtype=F32)
        check_paged(pout, plse, q, lens, total, ks, vs, first)
    for x in (out, lse, pout, plse, *grads.values()):
        rest = torch.cat([x[:used.start].flatten(), x[used.stop:].flatten()])
        assert bool((rest == 7).all())


def test_empty_calls():
    z = torch.zeros(0, 4, 64, device=DEV, dtype=BF16)
    out, lse = kda.kda_attn_prefill(z, z, z, return_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    g = kda.kda_attn_backward(z, z, z, out, lse, z)
    assert g["dq"].shape == (0, 4, 64)
    kp = torch.zeros(3, 16, 2, 64, device=DEV, dtype=BF16)
    assert kda.kda_attn_paged(z, kp, kp.clone(), ints([[0, 1]]), ints([5]), ints([0, 0])).shape == (0, 4, 64)


# ------------------------------------------------------------------ values

@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_other_sequences_are_not_seen(bad):
    """A sequence of infinities or NaN next to others, at places that share tiles with them."""
    lens, H, Hkv, d = [100, 60, 129, 5], 4, 2, 128
    q, k, v = prompt_inputs(sum(lens), H, Hkv, d, BF16, 101)
    dy = rnd(102, BF16, sum(lens), H, d)
    cu, at = cu_of(lens), starts(lens)
    out, lse = kda.kda_attn_prefill(q, k, v, cu, return_lse=True)
    g = kda.kda_attn_backward(q, k, v, out, lse, dy, cu)
    for n in (1, 3):
        for x in (q, k, v, dy):
            x[at[n]:at[n + 1]] = bad
    out2, lse2 = kda.kda_attn_prefill(q, k, v, cu, return_lse=True)
    g2 = kda.kda_attn_backward(q, k, v, out2, lse2, dy, cu)
    for n in (0, 2):
        part = slice(at[n], at[n + 1])
        assert torch.equal(out[part], out2[part]) and torch.equal(lse[part], lse2[part])
        assert all(torch.equal(g[m][part], g2[m][part]) for m in g)
    assert bool(torch.isnan(out2[at[1]:at[2]]).all())


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F16, 64)])
@pytest.mark.parametrize("grow", [1.0, -1.0])
def test_scores_that_grow(grow, dtype, d):
    """Scores from -900 to 900 along the keys, up or down: the maximum moves in every tile, or the
    later weights are nothing."""
    T, H = 600, 2
    q, k, v = prompt_inputs(T, H, 1, d, dtype, 111, std=0.05)
    q[..., 0] = 4.0
    k[..., 0] = (grow * torch.linspace(-225, 225, T, device=DEV)).to(dtype)[:, None]
    out, lse = kda.kda_attn_prefill(q, k, v, scale=1.0, out_dtype=F32, return_lse=True)
    check_prompts(out, lse, q, k, v, [T], scale=1.0)
    page = 64
    kp, vp, table, lens, _, _ = make_cache([T], 1, d, page, dtype, 112)
    for j in range(-(-T // page)):
        p, part = int(table[0, j]), slice(j * page, min((j + 1) * page, T))
        kp[p, :part.stop - part.start], vp[p, :part.stop - part.start] = k[part], v[part]
    for n in (1, 3, 200):
        out, lse = kda.kda_attn_paged(q[-n:], kp, vp, table, lens, scale=1.0, out_dtype=F32, return_lse=True)
        check_paged(out, lse, q[-n:], [n], [T], [k], [v], scale=1.0)


def test_one_value_everywhere():
    """Equal scores: the mean of what is seen, and lse = score + log of how many."""
    T, H, d = 300, 3, 64
    q, k = torch.ones(T, H, d, device=DEV, dtype=BF16), torch.ones(T, 1, d, device=DEV, dtype=BF16)
    v = rnd(121, BF16, T, 1, d)
    out, lse = kda.kda_attn_prefill(q, k, v, scale=0.125, out_dtype=F32, return_lse=True)
    check_prompts(out, lse, q, k, v, [T], scale=0.125)
    want = 8.0 + torch.log(torch.arange(1, T + 1, device=DEV, dtype=torch.float64))
    assert bool(((lse.double() - want[:, None]).abs() <= 64 * U[F32] * want[:, None]).all())


# ------------------------------------------------------------------ gradients against differences

def test_gradients_against_differences():
    """d/dh of sum(w . out) along a direction, from the definition in 64 bits, is what the
    gradients say of it: each within its bound, and within the part of out's own rounding in
    delta (out is the forward's 16-bit result: off by half a step)."""
    lens, H, Hkv, d = [90, 37], 4, 2, 64
    T, scale = sum(lens), 64 ** -0.5
    q, k, v = prompt_inputs(T, H, Hkv, d, BF16, 131)
    w = rnd(134, BF16, T, H, d)
    cu, at = cu_of(lens), starts(lens)
    out, lse = kda.kda_attn_prefill(q, k, v, cu, return_lse=True)
    g = kda.kda_attn_backward(q, k, v, out, lse, w, cu, grad_dtype=F32)

    def loss(q, k, v):
        return sum(float((rows(q[a:b], k[a:b], v[a:b], 0, scale)[0] * w[a:b].double()).sum()) for a, b in zip(at[:-1], at[1:]))

    for i, name in enumerate(("dq", "dk", "dv")):
        x = [q.double(), k.double(), v.double()]
        way = rnd(140 + i, torch.float64, *x[i].shape)
        h = 1e-5
        up, dn = list(x), list(x)
        up[i], dn[i] = x[i] + h * way, x[i] - h * way
        diff = (loss(*up) - loss(*dn)) / (2 * h)
        got, tol = float((g[name].double() * way).sum()), 1e-6 * abs(diff)   # (differences: h^2 and 1e-16 / h)
        for a, b in zip(at[:-1], at[1:]):
            args = (q[a:b], k[a:b], v[a:b], out[a:b], lse[a:b], w[a:b])
            want, mag, err, most = ref_backward(*args, scale)
            bound = backward_bounds(want, mag, err, most, q[a:b], k[a:b], lse[a:b], w[a:b], scale, F32)[name]
            # delta with out off by half a step (and by the forward's own weights' rounding): P delta times k or q
            e = ref_backward(q[a:b], k[a:b], v[a:b], 2 * U[BF16] * out[a:b].double().abs().sign() * out[a:b].double().abs(),
                             lse[a:b], w[a:b].double().abs(), scale)[2][name]
            tol += float(((bound + e) * way[a:b].abs()).sum())
        assert abs(got - diff) <= tol, (name, got, diff, tol)


# ------------------------------------------------------------------ graphs, streams, repetition

def test_graphs_and_streams():
    """Each call captured and replayed, two captures in turn, and on a stream of its own beside
    another call: the bits of the plain call."""
    lens, H, Hkv, d = [300, 1, 77], 8, 2, 128
    cu, T = cu_of(lens), sum(lens)
    sets = []
    for seed in (151, 161):
        q, k, v = prompt_inputs(T, H, Hkv, d, BF16, seed)
        total = [3000, 200, 77]
        cache = make_cache(total, Hkv, d, 64, BF16, seed)[:4]
        sets.append((q, k, v, rnd(seed + 5, BF16, T, H, d), cache))

    def call(s, **kw):
        q, k, v, dy, cache = s
        out, lse = kda.kda_attn_prefill(q, k, v, cu, return_lse=True, **kw)
        g = kda.kda_attn_backward(q, k, v, out, lse, dy, cu, **kw)
        one = kda.kda_attn_paged(q[:3], *cache, **kw)
        return [out, lse, *g.values(), kda.kda_attn_paged(q, *cache, cu, **kw), one]

    want = [call(s) for s in sets]
    graphs, outs = [], []
    for s in sets:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(call(s))
    for i in range(6):
        for x in outs[i % 2]:
            x.fill_(float("nan"))
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs[i % 2], want[i % 2]))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    got = [call(sets[i % 2], stream=streams[i % 2]) for i in range(8)]
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 2])), i


def test_serving_steps_in_a_graph():
    """A decode step (pages, append, attention) captured once and replayed: lengths and tables
    move on the device."""
    N, H, Hkv, d, page, steps = 5, 4, 2, 64, 8, 30
    total = [3, 0, 17, 8, 40]
    P, wide = 60, 12
    refs, table, lens = torch.zeros(P, dtype=torch.int32, device=DEV), torch.full((N, wide), -1, dtype=torch.int32, device=DEV), ints([0] * N)
    kp, vp = (torch.full((P, page, Hkv, d), float("nan"), device=DEV, dtype=BF16) for _ in range(2))
    ks = [[rnd(200 + n, BF16, total[n], Hkv, d)] for n in range(N)]
    vs = [[rnd(300 + n, BF16, total[n], Hkv, d)] for n in range(N)]
    kda.kda_cache_reserve(refs, table, lens, ints(total), page)
    kda.kda_cache_append(torch.cat([x[0] for x in ks]), torch.cat([x[0] for x in vs]), kp, vp, table, lens, cu_of(total))
    one = ints([1] * N)
    q, k, v = (torch.empty(N, h, d, device=DEV, dtype=BF16) for h in (H, Hkv, Hkv))
    out = torch.empty(N, H, d, device=DEV)

    def step():
        kda.kda_cache_reserve(refs, table, lens, one, page)
        kda.kda_cache_append(k, v, kp, vp, table, lens)
        kda.kda_attn_paged(q, kp, vp, table, lens, out=out, out_dtype=F32)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in range(steps):
        for i, x in enumerate((q, k, v)):
            x.copy_(rnd(400 + 3 * t + i, BF16, *x.shape))
        graph.replay()
        for n in range(N):
            ks[n].append(k[n:n + 1].clone()), vs[n].append(v[n:n + 1].clone())
        if t % 7 == 0 or t == steps - 1:
            check_paged(out, None, q, [1] * N, [x + t + 1 for x in total], [torch.cat(x) for x in ks], [torch.cat(x) for x in vs])
    assert lens.tolist() == [x + steps for x in total]


# ------------------------------------------------------------------ large offsets

def test_offsets_past_32_bits():
    """A cache of more than 2^32 elements, and queries of more than 2^31."""
    P, page, Hkv, d = 140000, 64, 4, 128                      # 4.6e9 elements each
    kp, vp = (torch.empty(P, page, Hkv, d, device=DEV, dtype=BF16) for _ in range(2))
    total, new, H = [200, 3000], [1, 40], 8
    need = [-(-n // page) for n in total]
    pages = [P - 1, 3, P - 2, 70001] + [P - 3 - 7 * i for i in range(need[1])]
    table = torch.full((2, need[1]), -1, dtype=torch.int32, device=DEV)
    table[0, :need[0]] = ints(pages[:need[0]])
    table[1] = ints(pages[4:4 + need[1]])
    lens = ints(total)
    ks, vs = [rnd(500 + n, BF16, total[n], Hkv, d) for n in range(2)], [rnd(510 + n, BF16, total[n], Hkv, d) for n in range(2)]
    kda.kda_cache_append(torch.cat(ks), torch.cat(vs), kp, vp, table, lens, cu_of(total))
    q = rnd(520, BF16, sum(new), H, d)
    for _ in range(2):
        out, lse = kda.kda_attn_paged(q, kp, vp, table, lens, cu_of(new), out_dtype=F32, return_lse=True)
        check_paged(out, lse, q, new, total, ks, vs)
        # once more from copies of the first sequence's pages
        src = table[0, :need[0]].clone()
        dst = ints([P - 4, 5, P - 5, P - 6])
        kda.kda_cache_copy(kp, vp, src, dst)
        table[0, :need[0]] = dst
    del kp, vp
    N, L, H = 1100, 128, 128
    q = rnd(530, BF16, N * L, H, 128)                          # 2.3e9 elements
    k, v = (rnd(531 + i, BF16, N * L, 1, 128) for i in range(2))
    out, lse = kda.kda_attn_prefill(q, k, v, num_seqs=N, return_lse=True)
    part = slice((N - 1) * L, N * L)
    check_prompts(out[part], lse[part], q[part], k[part], v[part], [L])
    g = kda.kda_attn_backward(q, k, v, out, lse, q, num_seqs=N)
    check_backward({n: x[part] for n, x in g.items()}, q[part], k[part], v[part], out[part], lse[part], q[part], [L])


# ------------------------------------------------------------------ what is out of range

def test_bad_pages_are_reported():
    """Page numbers outside the cache and lengths past the table: an error status, other sequences
    unharmed, the next call clean."""
    total, new, H, Hkv, d, page = [100, 200, 300], [1, 1, 1], 4, 2, 64, 16
    kp, vp, table, lens, ks, vs = make_cache(total, Hkv, d, page, BF16, 601)
    for q, n in ((rnd(602, BF16, 3, H, d), [1, 1, 1]), (rnd(603, BF16, 90, H, d), [30, 30, 30])):
        for bad in (-1, kp.shape[0], 10 ** 9, -(2 ** 31)):
            t = table.clone()
            t[1, 3] = bad
            out = kda.kda_attn_paged(q, kp, vp, t, lens, out_dtype=F32)
            assert kda.kda_get_last_device_error() == INVALID
            check_paged(torch.cat([out[:n[0]], out[-n[2]:]]), None, torch.cat([q[:n[0]], q[-n[2]:]]), [n[0], n[2]], [100, 300],
                        [ks[0], ks[2]], [vs[0], vs[2]])
        far = lens.clone()
        far[1] = table.shape[1] * page + 1
        kda.kda_attn_paged(q, kp, vp, table, far)
        assert kda.kda_get_last_device_error() == INVALID
        out = kda.kda_attn_paged(q, kp, vp, table, lens, out_dtype=F32)
        check_paged(out, None, q, n, total, ks, vs)
    # the cache's own calls pass such entries by
    was = kp.clone()
    t = table.clone()
    t[1, :] = kp.shape[0]
    x = rnd(604, BF16, 3, Hkv, d)
    kda.kda_cache_append(x, x, kp, vp, t, ints([0, 200, 0]))
    assert kda.kda_get_last_device_error() == INVALID and torch.equal(kp.nan_to_num(7.0), was.nan_to_num(7.0))
    kda.kda_cache_copy(kp, vp, ints([0, 2 ** 30]), ints([kp.shape[0], 1]))
    assert kda.kda_get_last_device_error() == INVALID and torch.equal(kp.nan_to_num(7.0), was.nan_to_num(7.0))
    refs, tab, ln = ints([1, 0]), ints([[0, -1], [-1, -1]]), ints([5, 0])
    state = [z.clone() for z in (refs, tab, ln)]
    kda.kda_cache_free(refs, tab, ln, ints([7, -1]), 16)
    assert kda.kda_get_last_device_error() == INVALID
    kda.kda_cache_fork(refs, tab, ln, ints([0, 9]), ints([0, 1]), 16)
    assert kda.kda_get_last_device_error() == INVALID
    assert all(torch.equal(a, b) for a, b in zip(state, (refs, tab, ln)))


@pytest.mark.parametrize("cu", [[0, 50, 20, 64], [-5, 10, 30, 64], [0, 10, 2 ** 31 - 1, 64], [64, 0, 64, 0], [0, 64, 0, 64]])
def test_malformed_offsets_stay_in_bounds(cu):
    """What is computed is unspecified; nothing outside the buffers is touched and every call ends."""
    T, H, Hkv, d = 64, 4, 2, 64
    guard = torch.full((3 * T, H, d), 7.0, device=DEV, dtype=BF16)
    q, k, v = prompt_inputs(T, H, Hkv, d, BF16, 701)
    c = ints(cu)
    out, lse = kda.kda_attn_prefill(q, k, v, c, out=guard[T:2 * T], return_lse=True)
    kda.kda_attn_backward(q, k, v, out, lse, q, c)
    kp, vp, table, lens, _, _ = make_cache([80, 80, 80], Hkv, d, 16, BF16, 702)
    kda.kda_attn_paged(q, kp, vp, table, lens, c, out=guard[T:2 * T])
    kda.kda_cache_append(k, v, kp, vp, table, lens, c)
    torch.cuda.synchronize()
    assert bool((guard[:T] == 7).all()) and bool((guard[2 * T:] == 7).all())


# ------------------------------------------------------------------ all of it together

@pytest.mark.parametrize("dtype,d,page,order", [(BF16, 128, 16, "NHD"), (F16, 64, 8, "HND")])
def test_serving(dtype, d, page, order):
    """Two layers of a small server: prompts enter the cache, whole or in chunks, are forked, decoded,
    rolled back, freed and compacted; every answer is that of the sequence's whole history."""
    r = random.Random(7)
    N, H, Hkv, P, wide, layers = 12, 6, 2, 200, 40, 2
    shape = (P, page, Hkv, d) if order == "NHD" else (P, Hkv, page, d)
    kp, vp = ([torch.full(shape, float("nan"), device=DEV, dtype=dtype) for _ in range(layers)] for _ in range(2))
    if order == "HND":
        kp, vp = ([x.transpose(1, 2) for x in xs] for xs in (kp, vp))
    refs, table, lens = torch.zeros(P, dtype=torch.int32, device=DEV), torch.full((N, wide), -1, dtype=torch.int32, device=DEV), ints([0] * N)
    past = [[(torch.zeros(0, Hkv, d, device=DEV, dtype=dtype),) * 2] * layers for _ in range(N)]
    seed = 800
    for step in range(24):
        kind = ["prompt", "decode", "fork", "decode", "chunk", "rollback", "free", "compact"][step % 8]
        live = [n for n in range(N) if past[n][0][0].shape[0]]
        if kind in ("prompt", "decode", "chunk"):
            new = [0] * N
            for n in range(N):
                if kind == "prompt" and n not in live and n < N - 3:
                    new[n] = r.choice([1, 5, page, 70])
                elif kind == "decode" and n in live:
                    new[n] = 1
                elif kind == "chunk" and n in live:
                    new[n] = r.choice([0, 1, 3, 40])
            T, seed = sum(new), seed + 10
            src, dst = kda.kda_cache_reserve(refs, table, lens, ints(new), page, return_copies=True)
            cu, at = cu_of(new), starts(new)
            for y in range(layers):
                kda.kda_cache_copy(kp[y], vp[y], src, dst)
                q, k, v = prompt_inputs(T, H, Hkv, d, dtype, seed + 3 * y)
                kda.kda_cache_append(k, v, kp[y], vp[y], table, lens, cu)
                out = kda.kda_attn_paged(q, kp[y], vp[y], table, lens, cu, out_dtype=F32)
                for n in range(N):
                    a, b = at[n], at[n + 1]
                    hist = past[n][y]
                    past[n] = list(past[n])
                    past[n][y] = (torch.cat([hist[0], k[a:b]]), torch.cat([hist[1], v[a:b]]))
                check_paged(out, None, q, new, [past[n][y][0].shape[0] for n in range(N)], [past[n][y][0] for n in range(N)],
                            [past[n][y][1] for n in range(N)])
                if kind == "prompt" and step == 0:
                    # the same prompts without a cache: the same answers, within both bounds
                    direct = kda.kda_attn_prefill(q, k, v, cu, out_dtype=F32)
                    check_prompts(direct, None, q, k, v, new)
        elif kind == "fork":
            empty = [n for n in range(N) if n not in live]
            if empty and live:
                parents = [r.choice(live) for _ in empty]
                src, dst = kda.kda_cache_fork(refs, table, lens, ints(parents), ints(empty), page)
                for y in range(layers):
                    kda.kda_cache_copy(kp[y], vp[y], src, dst)
                for p, c in zip(parents, empty):
                    past[c] = list(past[p])
        elif kind in ("rollback", "free"):
            some = r.sample(live, max(1, len(live) // 2))
            keep = [r.randint(0, past[n][0][0].shape[0]) if kind == "rollback" else 0 for n in some]
            kda.kda_cache_free(refs, table, lens, ints(some), page, keep=ints(keep) if kind == "rollback" else None)
            for n, m in zip(some, keep):
                past[n] = [(k[:m], v[:m]) for k, v in past[n]]
        else:
            _, _, src, dst = kda.kda_cache_compact(refs, table, lens, page, refs_out=refs, table_out=table)
            for y in range(layers):
                kda.kda_cache_copy(kp[y], vp[y], src, dst)
            assert bool((refs[:int((refs > 0).sum())] > 0).all())
        assert lens.tolist() == [x[0][0].shape[0] for x in past]


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F16, 64), (F16, 128), (BF16, 64)])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (8, 2), (12, 1)])
@pytest.mark.parametrize("lens", [[1], [2], [3, 0, 5], [128], [127, 2, 64]])
def test_gradients_of_short_sequences(lens, H, Hkv, d, dtype):
    """Sequences of one tile keep what the rounding of P and dS to 16 bits leaves as a second operand: the
    rest is at most u16 of the value and is itself off by u16 of that, so that u16^2 stands in the
    bound for u16 (the 2^-25 of small fp16 values holds for the rest as for the value).  The sums have
    twice as many products: (2 T H / 16 + 64) u32 of the magnitudes, the half of it counted already."""
    T = sum(lens)
    q, k, v = prompt_inputs(T, H, Hkv, d, dtype, 150 + T)
    dy = rnd(160 + T, dtype, T, H, d)
    out, lse = kda.kda_attn_prefill(q, k, v, cu_of(lens), return_lse=True)
    got = kda.kda_attn_backward(q, k, v, out, lse, dy, cu_of(lens), grad_dtype=F32)
    at = starts(lens)
    for a, b in zip(at[:-1], at[1:]):
        if a == b:
            continue
        x = [t[a:b] for t in (q, k, v, out, lse, dy)]
        want, mag, err, most = ref_backward(*x, d ** -0.5)
        tol = backward_bounds(want, mag, err, most, x[0], x[1], x[4], x[5], d ** -0.5, F32)
        for n in want:
            sums = (b - a) * (H if n != "dq" else 1) / 16 * U[F32]
            bound = tol[n] - (U[dtype] - U[dtype] ** 2 - sums) * mag[n]
            off = (got[n][a:b].double() - want[n]).abs()
            assert bool((off <= bound).all()), f"{n} of {b - a} tokens: off by {float((off / bound).max())} bounds"
    assert kda.kda_get_last_device_error() == 0
