"""Host-side checks of what a reservation granted (no GPU): the C calls that take it refuse bad
arguments before anything reaches the device.  Every pointer here is made up and never read."""
import pytest

from test_attn_host import INVALID, L, OK, R, UNSUPPORTED, at, cache, dims, heads, pages  # noqa: F401


def reserve(L, granted, c=None, **kw):
    a = dict(N=5, refs=at(1), table=at(2), lens=at(3), new=at(4), src=at(6), dst=at(7), missing=None, granted=granted,
             ws=at(5), size=1 << 20)
    a.update(kw)
    return L.kda_cache_reserve_granted(R(c or cache()), *a.values(), None)


def append(L, granted, c=None, **kw):
    a = dict(N=5, T=20)
    a.update(kw)
    return L.kda_cache_append_granted(R(c or cache()), a["N"], a["T"], 2, 128, R(heads(1, 2)), R(heads(2, 2)), R(pages(3)),
                                      R(pages(4)), at(5), at(6), None, granted, None)


def paged(L, granted, d=None, c=None):
    return L.kda_attn_paged_granted(R(d or dims()), R(c or cache()), R(heads(1)), R(pages(2)), R(pages(3)), at(4), at(5), None,
                                    granted, at(10), None, at(11), 1 << 30, None)


@pytest.mark.parametrize("granted", [at(1) + 4, at(2), at(3) + 8, at(4), at(5) + 16, at(6), at(7) + 4, at(8) + 2])
def test_reserve_refuses(L, granted):  # noqa: F811
    assert reserve(L, granted) == INVALID


@pytest.mark.parametrize("granted", [at(3), at(4) + 64, at(8) + 2])
def test_append_refuses(L, granted):  # noqa: F811
    assert append(L, granted) == INVALID


@pytest.mark.parametrize("granted", [at(10), at(11) + 4096, at(8) + 1])
def test_paged_refuses(L, granted):  # noqa: F811
    assert paged(L, granted) == INVALID


def test_other_checks_are_the_same(L):  # noqa: F811
    bad = cache(page_size=24)
    assert reserve(L, at(8), bad) == append(L, at(8), bad) == paged(L, at(8), c=bad) == UNSUPPORTED
    assert reserve(L, at(8), missing=at(8) + 4) == INVALID
    assert reserve(L, None, N=0, table=None, lens=None, new=None) == append(L, None, T=0) == OK
