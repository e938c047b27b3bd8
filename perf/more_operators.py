"""Cases of the softmax attention operators and of the paged cache that serves them:
attention over whole prompts (packed, causal, grouped heads), its gradients, attention of
new tokens over a paged cache (chunks and single tokens), and the operations on the pages.

For query head h of Hq, key head h // G of Hkv = Hq / G, token i of a sequence of L tokens
whose last n are new, and scale = d^-1/2:

    s_ij = scale q_i . k_j   for j <= L - n + i (nothing else is seen)
    lse_i = log sum_j exp(s_ij),   out_i = sum_j exp(s_ij - lse_i) v_j
    (a token that sees nothing has out 0 and lse -inf)

and for d_out:  P = exp(s - lse), delta_i = d_out_i . out_i, dP_ij = d_out_i . v_j,
    dS = P (dP - delta),  dq_i = scale sum_j dS_ij k_j,
    dk_j = scale sum_{h of the group, i} dS_ij q_i,  dv_j = sum_{h of the group, i} P_ij d_out_i

The cache: pages [P, page, Hkv, d] for keys and for values, a table [N, most] of page
numbers a sequence (-1: none), lengths [N], and of every page how many table entries name it
(0: free).  Free pages are given out lowest number first, to the sequences in their order.

Sizes: 8192 tokens and 256 single tokens are the sizes of this repository's layer
workloads, heads of 64 and 128 channels its head sizes; 32 query heads on 8 key heads,
pages of 16 to 128 tokens and prompts of 32768 are generic.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one long prompt through a layer
        dict(name="prompt 8k", op="prompt", T=8192, N=1, Hkv=8, G=4, d=128, dtype="bf16"),
        # prompts of different lengths packed into one batch, odd sizes, a group of 3; with the
        # log-sums that a training step keeps
        dict(name="prompt packed", op="prompt", T=5003, N=13, Hkv=4, G=3, d=64, dtype="f16"),
        # a short question: latency
        dict(name="prompt short", op="prompt", T=37, N=1, Hkv=2, G=8, d=128, dtype="bf16"),
        # a training step's gradients of the long prompt
        dict(name="backward 8k", op="backward", T=8192, N=1, Hkv=8, G=4, d=128, dtype="bf16"),
        # and of the packed batch
        dict(name="backward packed", op="backward", T=5003, N=13, Hkv=4, G=3, d=64, dtype="f16"),
        # one decode step of a single long sequence: latency, few rows over a long axis
        dict(name="token 1", op="paged", T=1, N=1, most=32768, fill=1.0, Hkv=8, G=4, d=128, page=64, dtype="bf16"),
        # one decode step of 256 sequences of different lengths: the cache streams through once
        dict(name="token 256", op="paged", T=256, N=256, most=8192, fill=0.5, Hkv=8, G=4, d=128, page=64, dtype="bf16"),
        # a prompt that is fed in pieces: 512 new tokens behind 32k
        dict(name="chunk 512", op="paged", T=512, N=1, most=32768, fill=1.0, Hkv=8, G=4, d=128, page=128, dtype="bf16"),
        # a serving step that mixes pieces of prompts with single tokens
        dict(name="chunks mixed", op="paged", T=1500, N=23, most=6000, fill=0.5, Hkv=2, G=5, d=64, page=16, dtype="f16"),
        # a prompt enters the cache: its pages are taken and its keys and values written
        dict(name="append 8k", op="append", T=8192, N=3, most=9000, Hkv=8, d=128, page=64, dtype="bf16"),
        # sampling several continuations of each of 32 prompts, the last ones given back first
        dict(name="fork 96", op="fork", N=128, M=96, most=8192, Hkv=8, d=128, page=64, dtype="bf16"),
        # half of a cache of small pages is in use: it is moved together
        dict(name="compact", op="compact", N=256, most=1000, P=16384, Hkv=8, d=128, page=16, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "backward", "backward", "paged", "paged", "paged", "append", "fork", "compact"])
    c = dict(op=op, Hkv=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 128]), dtype=rng.choice(["bf16", "f16"]))
    if op in ("prompt", "backward"):
        c.update(T=_log(rng, 1, 8192), N=rng.choice([1, 1, 2, 5, 13]), G=rng.choice([1, 2, 3, 4, 6, 8, 12]))
        while c["Hkv"] * c["G"] * c["d"] > 4096:
            c["Hkv"] //= 2
        return c
    c["page"] = rng.choice([16, 32, 64, 128])
    if op == "paged":
        N = _log(rng, 1, 256)
        c.update(N=N, G=rng.choice([1, 2, 3, 4, 5, 8, 12]), most=_log(rng, 20, 32768), fill=rng.choice([0.5, 1.0]))
        c["T"] = N if rng.random() < 0.4 else min(N * _log(rng, 1, 600), 2048)
        while N * c["most"] > 256 * 4096:
            c["most"] //= 2
        while c["Hkv"] * c["G"] * c["d"] > 4096:
            c["Hkv"] //= 2
        while c["T"] * min(c["most"], 32768) * c["Hkv"] * c["G"] * c["d"] > 512 * 32768 * 4096:
            c["T"] = max(N, c["T"] // 2)
            c["most"] //= 2
        return c
    if op == "append":
        c.update(T=_log(rng, 1, 8192), N=rng.choice([1, 2, 5, 13, 64]), most=9000)
    elif op == "fork":
        N = _log(rng, 2, 128)
        c.update(N=N, M=rng.randint(1, N - 1), most=_log(rng, 20, 8192))
    else:
        c.update(N=_log(rng, 1, 256), most=_log(rng, 20, 1000))
        c["P"] = 2 * c["N"] * (c["most"] // c["page"] + 2)
    return c


# ---------------------------------------------------------------- inputs

def _rng(case):
    return random.Random(sum(ord(ch) * 31 ** i for i, ch in enumerate(repr(sorted(
        (k, v) for k, v in case.items() if k != "name")))) % (1 << 61))


def _cut(r, T, N):
    """N ragged lengths with the sum T, some of them 0."""
    ends = [0] + sorted(r.randint(0, T) for _ in range(N - 1)) + [T]
    return [b - a for a, b in zip(ends[:-1], ends[1:])]


def _starts(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def _ceil(a, b):
    return -(-a // b)


def _lengths(case):
    """(tokens in the cache, new tokens) of every sequence of a call on the cache."""
    r, N = _rng(case), case["N"]
    op = case["op"]
    if op == "paged":
        total = [max(1, int(case["most"] * (1.0 - (1.0 - case["fill"]) * 2 * r.random()))) for _ in range(N)]
        new = [1] * N if case["T"] == N else _cut(r, case["T"], N)
        return [max(t, n) for t, n in zip(total, new)], new
    if op == "append":
        new = _cut(r, case["T"], N)
        return [r.randint(0, case["most"]) + n for n in new], new
    if op == "fork":
        return [_log(r, 1, case["most"]) if n < N - case["M"] else 0 for n in range(N)], None
    return [r.randint(1, case["most"]) for _ in range(N)], None   # compact


def _pages(case):
    """(number of pages, table width) of a case's cache."""
    total, new = _lengths(case)
    page = case["page"]
    wide = max(_ceil(n, page) for n in total) + 1
    if case["op"] == "compact":
        return max(case["P"], sum(_ceil(n, page) for n in total)), wide
    spare = case["M"] + 3 if case["op"] == "fork" else 5
    return sum(_ceil(n, page) for n in total) + spare, wide


def _shared(total, n, page):
    """Every fourth sequence continues the one before it: they share their prefix's whole pages."""
    return min(total[n - 1], total[n]) // page if n % 4 == 3 else 0


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(int(seed) * 2 + 1)
    dt, op = DTYPES[case["dtype"]], case["op"]
    Hkv, d = case["Hkv"], case["d"]

    def rnd(*shape, std=1.0):
        x = torch.randn(shape, generator=gen, device=dev, dtype=dt)
        return x if std == 1.0 else x * std

    s = dict(op=op)
    if op in ("prompt", "backward"):
        T, N, Hq = case["T"], case["N"], Hkv * case["G"]
        lens = [T] if N == 1 else _cut(_rng(case), T, N)
        s["at"] = _starts(lens)
        s["cu"] = None if N == 1 else torch.tensor(s["at"], dtype=torch.int32, device=dev)
        # queries, keys and values are parts of one projection's rows
        rows = rnd(T, Hq + 2 * Hkv, d)
        rows[:, :Hq] *= 1.5
        s["q"], s["k"], s["v"] = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
        s["lse_too"] = N > 1
        if op == "backward":
            s["d_out"] = rnd(T, Hq, d)
            s["out"], s["lse"] = _prompt_plain(s)
        return s
    page, N = case["page"], case["N"]
    total, new = _lengths(case)
    P, wide = _pages(case)
    s.update(page=page, lens_host=total)
    s["k_pages"], s["v_pages"] = rnd(P, page, Hkv, d), rnd(P, page, Hkv, d)
    # the pages of a cache that has been in use for a while lie in no order
    order = torch.randperm(P, generator=gen, device=dev).to(torch.int32)
    table = torch.full((N, wide), -1, dtype=torch.int32, device=dev)
    if op == "paged":
        T, Hq = case["T"], Hkv * case["G"]
        s["at"] = _starts(new)
        s["cu"] = None if T == N else torch.tensor(s["at"], dtype=torch.int32, device=dev)
        s["q"] = rnd(T, Hq, d, std=1.5)
    elif op == "append":
        T = case["T"]
        s["at"] = _starts(new)
        s["cu"] = torch.tensor(s["at"], dtype=torch.int32, device=dev)
        s["k"], s["v"] = rnd(T, Hkv, d), rnd(T, Hkv, d)
        s["new"] = torch.tensor(new, dtype=torch.int32, device=dev)
        s["seqs"] = torch.arange(N, dtype=torch.int32, device=dev)
        total = [a - b for a, b in zip(total, new)]
        s["keep"] = torch.tensor(total, dtype=torch.int32, device=dev)
    elif op == "fork":
        M, r = case["M"], _rng(case)
        s["parents"] = torch.tensor([r.randint(0, N - M - 1) for _ in range(M)], dtype=torch.int32, device=dev)
        s["children"] = torch.arange(N - M, N, dtype=torch.int32, device=dev)
    at = 0
    for n, length in enumerate(total):
        have = _ceil(length, page)
        table[n, :have] = order[at:at + have]
        at += have
        if op == "compact" and n % 4 == 3:
            shared = _shared(total, n, page)
            table[n, :shared] = table[n - 1, :shared]
    s["table"] = table
    s["lens"] = torch.tensor(total, dtype=torch.int32, device=dev)
    used = table[table >= 0].long()
    s["refs"] = torch.zeros(P, dtype=torch.int32, device=dev).index_add_(0, used, torch.ones_like(used, dtype=torch.int32))
    return s


# ---------------------------------------------------------------- plain forms

BLOCK = 1024   # query tokens whose scores are held at once


def _scores(q, k, first, scale):
    """[Hkv, G, t, s] scores of t tokens, the first of which sees `first` + 1 of the s keys."""
    t, Hq, d = q.shape
    n, Hkv = k.shape[:2]
    s = torch.matmul(q.float().view(t, Hkv, Hq // Hkv, d).permute(1, 2, 0, 3).reshape(Hkv, -1, d),
                     k.float().permute(1, 2, 0)).view(Hkv, Hq // Hkv, t, n) * scale
    seen = torch.arange(n, device=q.device) <= (first + torch.arange(t, device=q.device))[:, None]
    return torch.where(seen, s, torch.full_like(s, -math.inf))


def _attend(q, k, v, first):
    """(out [t, Hq, d], lse [t, Hq]) in fp32."""
    t, Hq, d = q.shape
    Hkv = k.shape[1]
    if k.shape[0] == 0:
        return torch.zeros(t, Hq, d, device=q.device), torch.full((t, Hq), -math.inf, device=q.device)
    s = _scores(q, k, first, d ** -0.5)
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(s - m)
    del s
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(Hkv, -1, k.shape[0]), v.float().permute(1, 0, 2)).view(Hkv, -1, t, d)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    lse = (torch.log(total) + m)[..., 0]
    return o.permute(2, 0, 1, 3).reshape(t, Hq, d), lse.permute(2, 0, 1).reshape(t, Hq)


def _prompt_plain(s):
    q, k, v = s["q"], s["k"], s["v"]
    out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    lse = torch.empty(q.shape[:2], device=q.device)
    for a, e in zip(s["at"][:-1], s["at"][1:]):
        for b in range(a, e, BLOCK):
            c = min(b + BLOCK, e)
            out[b:c], lse[b:c] = _attend(q[b:c], k[a:c], v[a:c], b - a)
    return out, lse


def _backward_plain(s):
    q, k, v, out, lse, dy = (s[n] for n in ("q", "k", "v", "out", "lse", "d_out"))
    T, Hq, d = q.shape
    Hkv, scale = k.shape[1], d ** -0.5
    dq = torch.empty((T, Hq, d), dtype=q.dtype, device=q.device)
    dk, dv = (torch.zeros((T, Hkv, d), device=q.device) for _ in range(2))
    delta = (dy.float() * out.float()).sum(-1)

    def grouped(x):   # [t, Hq, ...] -> [Hkv, G t, ...], heads before tokens
        x = x.float().unflatten(1, (Hkv, Hq // Hkv))
        return x.permute(1, 2, 0, *range(3, x.dim())).flatten(1, 2)

    for a, e in zip(s["at"][:-1], s["at"][1:]):
        for b in range(a, e, BLOCK):
            c = min(b + BLOCK, e)
            p = torch.exp(_scores(q[b:c], k[a:c], b - a, scale).flatten(1, 2) - grouped(lse[b:c])[..., None])
            g = grouped(dy[b:c])
            dv[a:c] += torch.matmul(p.transpose(1, 2), g).transpose(0, 1)
            ds = p * (torch.matmul(g, v[a:c].float().permute(1, 2, 0)) - grouped(delta[b:c])[..., None])
            del p
            dk[a:c] += torch.matmul(ds.transpose(1, 2), grouped(q[b:c])).transpose(0, 1) * scale
            x = torch.matmul(ds, k[a:c].float().transpose(0, 1)) * scale
            dq[b:c] = x.view(Hkv, Hq // Hkv, c - b, d).permute(2, 0, 1, 3).reshape(c - b, Hq, d)
    return dict(dq=dq, dk=dk.to(q.dtype), dv=dv.to(q.dtype))


def _paged_plain(s):
    q = s["q"]
    out = torch.empty_like(q)
    for n, (a, e) in enumerate(zip(s["at"][:-1], s["at"][1:])):
        L = s["lens_host"][n]
        pages = s["table"][n, :_ceil(L, s["page"])].long()
        k, v = s["k_pages"][pages].flatten(0, 1)[:L], s["v_pages"][pages].flatten(0, 1)[:L]
        for b in range(a, e, BLOCK):
            c = min(b + BLOCK, e)
            out[b:c] = _attend(q[b:c], k, v, L - (e - b))[0]
    return out


def _ceil_t(x, page):
    return torch.div(x + (page - 1), page, rounding_mode="floor")


def _free_plain(s, seqs, keep):
    table, lens, refs, page = s["table"], s["lens"], s["refs"], s["page"]
    seqs = seqs.long()
    keep = torch.minimum(lens[seqs], keep)
    col = torch.arange(table.shape[1], device=table.device)
    drop = (col >= _ceil_t(keep, page)[:, None]) & (col < _ceil_t(lens[seqs], page)[:, None])
    rows = table[seqs]
    gone = rows[drop].long()
    refs.index_add_(0, gone, torch.full_like(gone, -1, dtype=torch.int32))
    table[seqs] = torch.where(drop, torch.full_like(rows, -1), rows)
    lens[seqs] = keep


def _give(need, refs):
    """(first place in the list of free pages, whether it is served) of each, and the list."""
    free = torch.nonzero(refs == 0)[:, 0]
    upto = torch.cumsum(need, 0)
    return upto - need, (need == 0) | (upto <= free.shape[0]), free


def _reserve_plain(s, new):
    table, lens, refs, page = s["table"], s["lens"], s["refs"], s["page"]
    have, want = _ceil_t(lens, page), _ceil_t(lens + new, page)
    start, served, free = _give((want - have).long(), refs)
    col = torch.arange(table.shape[1], device=table.device)
    here = (col >= have[:, None]) & (col < want[:, None]) & served[:, None]
    took = free[(start[:, None] + col - have[:, None])[here]]
    table[here] = took.to(torch.int32)
    refs[took] = 1
    lens += torch.where(served, new, torch.zeros_like(new))


def _append_plain(s):
    page = s["page"]
    cu, row = s["cu"].long(), torch.arange(s["k"].shape[0], device=s["k"].device)
    seq = torch.searchsorted(cu, row, right=True) - 1
    place = s["lens"].long()[seq] - (cu[1:] - cu[:-1])[seq] + row - cu[seq]
    pages = s["table"][seq, torch.div(place, page, rounding_mode="floor")].long()
    s["k_pages"][pages, place % page] = s["k"]
    s["v_pages"][pages, place % page] = s["v"]


def _copy_plain(s, src, dst):
    ok = src >= 0
    src, dst = src[ok].long(), dst[ok].long()
    s["k_pages"][dst] = s["k_pages"][src]
    s["v_pages"][dst] = s["v_pages"][src]


def _fork_plain(s):
    table, lens, refs, page = s["table"], s["lens"], s["refs"], s["page"]
    parents, children = s["parents"].long(), s["children"].long()
    length = lens[parents]
    part = (length % page != 0)
    start, served, free = _give(part.long(), refs)
    rows = table[parents]
    col = torch.arange(table.shape[1], device=table.device)
    whole = torch.div(length, page, rounding_mode="floor")[:, None]
    none = torch.full_like(rows, -1)
    new = torch.where((col < whole) & served[:, None], rows, none)
    own_page = (col == whole) & (part & served)[:, None]
    took = free[start[part & served]]
    src = torch.full_like(parents, -1, dtype=torch.int32)
    dst = src.clone()
    src[part & served] = rows[own_page]
    dst[part & served] = took.to(torch.int32)
    new[own_page] = took.to(torch.int32)
    kept = new[(col < whole) & served[:, None]].long()
    refs.index_add_(0, kept, torch.ones_like(kept, dtype=torch.int32))
    refs[took] = 1
    table[children] = new
    lens[children] = torch.where(served, length, torch.zeros_like(length))
    return src, dst


def _compact_plain(s):
    table, lens, refs, page = s["table"], s["lens"], s["refs"], s["page"]
    P = refs.shape[0]
    number = torch.arange(P, device=refs.device)
    live = refs > 0
    L = live.sum()
    src_some, dst_some = number[live & (number >= L)], number[~live & (number < L)]
    src = torch.full((P,), -1, dtype=torch.int32, device=refs.device)
    dst = src.clone()
    src[:src_some.shape[0]], dst[:dst_some.shape[0]] = src_some.to(torch.int32), dst_some.to(torch.int32)
    to = number.clone()
    to[src_some] = dst_some
    refs_out = refs.clone()
    refs_out[dst_some] = refs[src_some]
    refs_out[src_some] = 0
    col = torch.arange(table.shape[1], device=table.device)
    mine = col < _ceil_t(lens, page)[:, None]
    table_out = torch.where(mine, to[table.clamp(min=0).long()].to(torch.int32), table)
    return refs_out, table_out, src, dst


# ---------------------------------------------------------------- the framework's calls

def _run_own(s):
    import linear_attention_sequence_gb300 as kda
    op = s["op"]
    if op == "prompt":
        return kda.kda_attn_prefill(s["q"], s["k"], s["v"], s["cu"], return_lse=s["lse_too"])
    if op == "backward":
        return kda.kda_attn_backward(s["q"], s["k"], s["v"], s["out"], s["lse"], s["d_out"], s["cu"])
    if op == "paged":
        return kda.kda_attn_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["cu"])
    page = s["page"]
    if op == "append":
        kda.kda_cache_free(s["refs"], s["table"], s["lens"], s["seqs"], page, keep=s["keep"])
        kda.kda_cache_reserve(s["refs"], s["table"], s["lens"], s["new"], page)
        kda.kda_cache_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["cu"])
        return {n: s[n] for n in ("refs", "table", "lens", "k_pages", "v_pages")}
    if op == "fork":
        kda.kda_cache_free(s["refs"], s["table"], s["lens"], s["children"], page)
        src, dst = kda.kda_cache_fork(s["refs"], s["table"], s["lens"], s["parents"], s["children"], page)
        kda.kda_cache_copy(s["k_pages"], s["v_pages"], src, dst)
        return {n: s[n] for n in ("refs", "table", "lens", "k_pages", "v_pages")}
    refs, table, src, dst = kda.kda_cache_compact(s["refs"], s["table"], s["lens"], page)
    kda.kda_cache_copy(s["k_pages"], s["v_pages"], src, dst)
    return dict(refs=refs, table=table, src=src, dst=dst, k_pages=s["k_pages"], v_pages=s["v_pages"])


def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "prompt":
        out, lse = _prompt_plain(s)
        return (out, lse) if s["lse_too"] else out
    if op == "backward":
        return _backward_plain(s)
    if op == "paged":
        return _paged_plain(s)
    if op == "append":
        _free_plain(s, s["seqs"], s["keep"])
        _reserve_plain(s, s["new"])
        _append_plain(s)
        return {n: s[n] for n in ("refs", "table", "lens", "k_pages", "v_pages")}
    if op == "fork":
        _free_plain(s, s["children"], torch.zeros_like(s["children"]))
        src, dst = _fork_plain(s)
        _copy_plain(s, src, dst)
        return {n: s[n] for n in ("refs", "table", "lens", "k_pages", "v_pages")}
    refs, table, src, dst = _compact_plain(s)
    _copy_plain(s, src, dst)
    return dict(refs=refs, table=table, src=src, dst=dst, k_pages=s["k_pages"], v_pages=s["v_pages"])


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op, Hkv, d = case["op"], case["Hkv"], case["d"]
    row = Hkv * d * 2   # a token's keys, or its values
    if op in ("prompt", "backward"):
        T, N, G = case["T"], case["N"], case["G"]
        lens = [T] if N == 1 else _cut(_rng(case), T, N)
        pairs = sum(n * (n + 1) // 2 for n in lens) * Hkv * G
        one = T * row
        if op == "prompt":
            return dict(bytes=2 * one * G + 2 * one + (T * Hkv * G * 4 if N > 1 else 0), flops=4 * pairs * d)
        # q, out, d_out, dq; k, v, dk, dv; lse
        return dict(bytes=4 * one * G + 4 * one + T * Hkv * G * 4, flops=10 * pairs * d)
    total, new = _lengths(case)
    if op == "paged":
        G = case["G"]
        pairs = sum(n * t - n * (n - 1) // 2 for t, n in zip(total, new)) * Hkv * G
        seen = sum(t for t, n in zip(total, new) if n)
        table = sum(_ceil(t, case["page"]) for t in total) * 4
        return dict(bytes=2 * seen * row + 2 * case["T"] * row * G + table + 8 * case["N"], flops=4 * pairs * d)
    P = _pages(case)[0]
    held = sum(_ceil(n, case["page"]) for n in total)
    if op == "append":
        taken = sum(_ceil(t, case["page"]) - _ceil(t - n, case["page"]) for t, n in zip(total, new))
        return dict(bytes=4 * case["T"] * row + P * 4 + taken * 16, flops=case["T"])
    page = case["page"] * row * 2   # a page's keys and values
    if op == "fork":
        r, M = _rng(case), case["M"]
        parents = [r.randint(0, case["N"] - M - 1) for _ in range(M)]
        moved = sum(1 for p in parents if total[p] % case["page"])
        held = sum(_ceil(total[p], case["page"]) for p in parents)
        return dict(bytes=2 * moved * page + P * 4 + held * 16, flops=M)
    live = held - sum(_shared(total, n, case["page"]) for n in range(case["N"]))
    moved = live * (P - live) // P   # of the live pages, those that lie behind the first `live` numbers
    return dict(bytes=2 * moved * page + 4 * P * 4 + 2 * held * 4, flops=P)


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    op = case["op"]
    if op in ("append", "fork", "compact"):
        return None   # numbers that are moved, and whole numbers
    s = prepare(case, seed)
    if op == "backward":
        return _exact_backward(s)
    if op == "paged":
        out = s["q"].double()
        for n, (a, e) in enumerate(zip(s["at"][:-1], s["at"][1:])):
            L, page = s["lens_host"][n], s["page"]
            if e == a:
                continue
            place = torch.arange(L, device=out.device)
            pages = s["table"][n].long()[place // page]
            k, v = s["k_pages"][pages, place % page].double(), s["v_pages"][pages, place % page].double()
            for b in range(a, e, 256):
                c = min(b + 256, e)
                out[b:c] = _exact_rows(out[b:c], k, v, L - (e - b))[0]
        return out
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=q.dtype, device=q.device)
    for a, e in zip(s["at"][:-1], s["at"][1:]):
        for b in range(a, e, 512):
            c = min(b + 512, e)
            out[b:c], lse[b:c] = _exact_rows(q[b:c], k[a:c], v[a:c], b - a)
    return (out, lse) if s["lse_too"] else out


def _exact_rows(q, k, v, first):
    """Head by head: the probabilities of the rows, and what they average."""
    t, Hq, d = q.shape
    G = Hq // k.shape[1]
    hidden = torch.ones(t, k.shape[0], dtype=torch.bool, device=q.device).triu(first + 1)
    out, lse = torch.empty_like(q), torch.empty((t, Hq), dtype=q.dtype, device=q.device)
    for h in range(Hq):
        s = (q[:, h] @ k[:, h // G].t() / math.sqrt(d)).masked_fill_(hidden, -math.inf)
        lse[:, h] = torch.logsumexp(s, 1)
        out[:, h] = torch.exp(s - lse[:, h:h + 1]) @ v[:, h // G]
    return out, lse


def _exact_backward(s):
    q, k, v, out, lse, dy = (s[n].double() for n in ("q", "k", "v", "out", "lse", "d_out"))
    Hq, d = q.shape[1:]
    G = Hq // k.shape[1]
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for a, e in zip(s["at"][:-1], s["at"][1:]):
        for h in range(Hq):
            g = h // G
            for b in range(a, e, 2048):
                c = min(b + 2048, e)
                hidden = torch.ones(c - b, c - a, dtype=torch.bool, device=q.device).triu(b - a + 1)
                p = torch.exp((q[b:c, h] @ k[a:c, g].t() / math.sqrt(d)).masked_fill_(hidden, -math.inf)
                              - lse[b:c, h:h + 1])
                dv[a:c, g] += p.t() @ dy[b:c, h]
                delta = (dy[b:c, h] * out[b:c, h]).sum(1, keepdim=True)
                ds = p * (dy[b:c, h] @ v[a:c, g].t() - delta) / math.sqrt(d)
                dq[b:c, h] = ds @ k[a:c, g]
                dk[a:c, g] += ds.t() @ q[b:c, h]
    return dict(dq=dq, dk=dk, dv=dv)
