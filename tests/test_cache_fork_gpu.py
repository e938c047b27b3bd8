"""GPU tests of forks at their edges: children that are not empty, lists and caches without entries."""
import pytest
import torch

import linear_attention_sequence_gb300 as kda
from test_cache_gpu import Both, ints

pytestmark = pytest.mark.gpu
INVALID = 1


@pytest.mark.parametrize("wide", [5, 3000])
@pytest.mark.parametrize("M", [4, 40])
def test_children_with_pages_are_passed_by(M, wide):
    """In one launch and in two (by the size of the rows): every third child has pages of its own, which it
    keeps with their counts; the others are served as if those were not in the lists."""
    N = M + 2
    c = Both(3 * N, N, wide, 8)
    taken = list(range(2, N, 3))
    c.reserve([13, 16] + [9 if n in taken else 0 for n in range(2, N)])
    parents, children = [n % 2 for n in range(2, N)], list(range(2, N))
    src, dst = kda.kda_cache_fork(*c.state, ints(parents), ints(children), 8, missing=c.missing)
    assert kda.kda_get_last_device_error() == INVALID
    some = [i for i, n in enumerate(children) if n not in taken]
    s, d, want = c.plain.fork([parents[i] for i in some], [children[i] for i in some])
    c.check()
    assert c.missing.item() == want
    got = list(zip(src.tolist(), dst.tolist()))
    assert [got[i] for i in some] == list(zip(s, d))
    assert all(x == (-1, -1) for i, x in enumerate(got) if i not in some)
    # and once more: now none of them is empty
    before = [x.clone() for x in c.state]
    kda.kda_cache_fork(*c.state, ints(parents), ints(children), 8)
    assert kda.kda_get_last_device_error() == INVALID
    assert all(torch.equal(a, b) for a, b in zip(before, c.state))


def test_no_children_and_no_rows():
    """Results are written where there is nothing to fork, and a cache without rows has no sequence to name."""
    c = Both(9, 2, 4, 8)
    c.reserve([9, 0])
    missing = ints([-7])
    src, dst = kda.kda_cache_fork(*c.state, ints([]), ints([]), 8, missing=missing)
    assert missing.item() == 0 and src.shape == dst.shape == (0,)
    kda.kda_cache_free(*c.state, ints([]), 8)
    c.check()
    assert kda.kda_get_last_device_error() == 0
    for wide in (4, 3000):
        none = (c.refs, torch.empty((0, wide), dtype=torch.int32, device="cuda"), ints([]))
        src, dst, missing = ints([77] * 5), ints([77] * 5), ints([-7])
        kda.kda_cache_fork(*none, ints([0, 1, -1, 2, 0]), ints([1, 0, 5, 3, 0]), 8, src=src, dst=dst, missing=missing)
        assert kda.kda_get_last_device_error() == INVALID
        assert src.tolist() == dst.tolist() == [-1] * 5 and missing.item() == 0
    kda.kda_cache_free(*none, ints([3]), 8)
    assert kda.kda_get_last_device_error() == INVALID
    kda.kda_cache_reserve(*none, ints([]), 8, missing=missing.fill_(-7))
    assert missing.item() == 0 and kda.kda_get_last_device_error() == 0
    c.check()
