"""GPU tests of which kernel computes a call of attention over the 4-bit cache: the kernel is read from
the launch, so that a test of a way of computing it cannot pass by another."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import recv_fifo_plane_amd as xf  # noqa: E402
from launches import launches  # noqa: E402
from mxcache_cases import check_attend  # noqa: E402
from test_mxcache_attend_gpu import DIMS, TYPES  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture
def kernels(monkeypatch):
    """Names of the kernels that the calls of attend launch, those of each call a list."""
    got, attend = [], xf.PagedCache.attend

    def recorded(self, *args, **kw):
        got.append([name for name, _ in launches(lambda: attend(self, *args, **kw))])
        return attend(self, *args, **kw)

    monkeypatch.setattr(xf.PagedCache, "attend", recorded)
    return got


def are(call, *kernels):
    """Whether a call's kernels are these: (kernel, core), the core of a join None."""
    return len(call) == len(kernels) and all(
        name in have and (core is None or core in have) for have, (name, core) in zip(call, kernels))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", DIMS)
def test_numbered_tiles_of_many_rows(D, dtype, kernels):
    """Two requests with many rows among many with few, whose largest number is not known."""
    rng = np.random.default_rng(D)
    rows = rng.integers(0, 5, 90).tolist()
    rows[40], rows[70] = 190, 150
    lens = [max(0, r + int(rng.integers(-3, 40))) for r in rows]
    check_attend(lens, rows, 16, 16, 8, D, dtype, seed=D, many=1216, shared=False, hints=False, behind=3)
    assert are(kernels[0], ("attend_packed_kernel", "4Wide")), kernels


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", DIMS)
def test_tiles_and_shares_of_many_rows(D, dtype, kernels):
    H = 32 if D <= 128 else 16
    check_attend([190, 200, 0, 33], [190, 199, 1, 17], 16, H, 4, D, dtype, seed=D, many=1216, shared=False)
    check_attend([300, 129, 1, 64], [300, 129, 1, 64], 16, 1, 2, D, dtype, seed=D, many=0, shared=True)
    assert are(kernels[0], ("attend_kernel", "4Wide")), kernels[0]
    assert are(kernels[1], ("attend_wide_kernel", "4Wide"), ("join_kernel", None)), kernels[1]


@pytest.mark.parametrize("dtype", TYPES)
def test_few_rows(dtype, kernels):
    rng = np.random.default_rng(0)
    rows = rng.integers(0, 5, 300).tolist()
    rows[40] = 100
    lens = [max(0, r + int(rng.integers(-3, 40))) for r in rows]
    check_attend([40, 8, 90], [2, 1, 3], 16, 2, 4, 128, dtype)
    check_attend([1700, 9], [1, 2], 16, 2, 4, 128, dtype)
    check_attend(lens, rows, 16, 4, 4, 128, dtype, hints=False, width=4)
    assert are(kernels[0], ("attend_kernel", "5Core4")), kernels[0]
    assert are(kernels[1], ("attend_flat_kernel", "5Core4"), ("join_kernel", None)), kernels[1]
    assert are(kernels[2], ("attend_packed_kernel", "5Core4")), kernels[2]


@pytest.mark.parametrize("D", DIMS)
def test_requests_of_half_a_tile(D, kernels):
    """However long, 64 rows of a request (32 of wide heads) are few; one more are many."""
    most = 64 if D <= 128 else 32
    for rows in (most, most + 1):
        check_attend([300], [rows], 16, 2, 1, D, seed=D, many=0)
    assert "5Core4" in kernels[0][0] and "4Wide" in kernels[1][0], kernels
