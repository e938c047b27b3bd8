"""Host-side checks (no GPU) of how the state space kernels find their way through a
batch's lengths.  The functions are those of csrc/kda_ssm_common.cuh, compiled for the
host."""
import ctypes
import itertools
import random
import subprocess

import pytest

from linear_attention_sequence_gb300 import _build

SOURCE = """
#include "kda_ssm_common.cuh"
extern "C" int find(const int32_t *cu, int N, int64_t total, int64_t seq_len, int64_t t, int *n, int64_t *sa, int64_t *sb) {
    return kda::find_seq(cu, N, total, seq_len, t, *n, *sa, *sb);
}
extern "C" void cut(int N, int T, int ragged, int across, int places, int64_t *rows_cut_most) {
    kda::SsmProblem P{};
    P.N = N;
    P.T = T;
    const kda::Parts p = kda::cut_parts(P, ragged, across, {1.6, 0.5, 2.0, 0.1, 1.0, places});
    rows_cut_most[0] = p.rows;
    rows_cut_most[1] = p.cut;
    rows_cut_most[2] = p.most;
}
"""


@pytest.fixture(scope="module")
def H(tmp_path_factory):
    d = tmp_path_factory.mktemp("lengths")
    (d / "lengths.cu").write_text(SOURCE)
    r = subprocess.run([_build.nvcc(), "-shared", "-o", str(d / "lengths.so"), str(d / "lengths.cu"), "-I", _build.CSRC,
                        "-cudart", "shared"] + _build.cflags(), capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return ctypes.CDLL(str(d / "lengths.so"))


def walk(H, cu, total, t0=0):
    """The pieces [a, b) of sequences n that a kernel's run from t0 to the batch's end
    takes, as the kernels walk: to the end of the sequence found, or to where the search says."""
    arr = (ctypes.c_int32 * len(cu))(*cu)
    n, sa, sb = ctypes.c_int(), ctypes.c_int64(), ctypes.c_int64()
    N, t, got = len(cu) - 1, t0, []
    for _ in range(2 * len(cu) + 2):
        if t >= total:
            return got
        if H.find(arr, N, ctypes.c_int64(total), ctypes.c_int64(0), ctypes.c_int64(t), ctypes.byref(n), ctypes.byref(sa),
                  ctypes.byref(sb)):
            assert 0 <= n.value < N and 0 <= sa.value <= t < sb.value <= total
            got.append((n.value, t, sb.value))
            t = sb.value
        else:
            assert t < sa.value <= total, f"the search at {t} of {cu} leads to {sa.value}"
            t = sa.value
    raise AssertionError(f"no end in {cu}")


def test_search_passes_rows_of_an_empty_batch(H):
    for first in (-3, 0, 2, 9, 10, 50):
        for t0 in (0, 2, 9):
            assert walk(H, [first], 10, t0) == []


def test_search_finds_every_sequence(H):
    rng = random.Random(3)
    for _ in range(300):
        lens = [rng.choice([0, 0, 1, 2, 7, 30]) for _ in range(rng.randint(1, 9))]
        cu = [rng.choice([0, 0, 4])]
        for x in lens:
            cu.append(cu[-1] + x)
        total = cu[-1] + rng.choice([0, 0, 5])
        assert walk(H, cu, total) == [(n, a, b) for n, (a, b) in enumerate(zip(cu, cu[1:])) if b > a]
        for t0 in range(total):
            want = [(n, max(a, t0), b) for n, (a, b) in enumerate(zip(cu, cu[1:])) if b > max(a, t0)]
            assert walk(H, cu, total, t0) == want


def test_search_moves_on_in_malformed_lengths(H):
    for cu in itertools.product([-5, 0, 3, 4, 10, 11, 1 << 30], repeat=3):
        for t0 in range(10):
            walk(H, list(cu), 10, t0)


def test_no_runs_without_sequences():
    """The convolution's gradient walks no rows of a batch without sequences: its runs'
    shares, W + 1 rows of channels each, need no room."""
    _build.build()
    from linear_attention_sequence_gb300 import _ssm, lib
    size = lambda N: lib().kda_ssm_conv_backward_workspace(_ssm._DIMS.pack(N, 200, 40, 4, 0, 0))  # noqa: E731
    assert size(0) == 0 and size(1) > 0


def test_no_parts_without_sequences(H):
    """A batch without sequences has no parts, however many rows: sums over its parts are
    sums over nothing."""
    got = (ctypes.c_int64 * 3)()
    for T in (0, 1, 32, 33, 200, 2000, 100000):
        for ragged in (0, 1):
            for across in (1, 2, 64, 500):
                H.cut(0, T, ragged, across, 304, got)
                assert list(got) == [0, 0, 0], (T, ragged, across)
                H.cut(1, T, ragged, across, 304, got)
                assert got[2] == 1 + got[0]
