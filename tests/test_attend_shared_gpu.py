"""GPU tests of attention whose tokens are shared out over workgroups (calls with
a workspace): every head size and type, one and two tiles of rows, and the
inputs where a tile that several workgroups share can go wrong."""
import math

import numpy as np
import pytest

import cache_ref as R
from attend_bounds import two_part_bounds
from test_attend_weights_gpu import is_shared
from test_cache_gpu import check_attend

pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DIMS = [64, 96, 128, 192, 256]
TYPES = ["bf16", "fp16"]


@pytest.fixture(autouse=True)
def bounds(monkeypatch):
    monkeypatch.setattr(R, "attend_bounds", two_part_bounds)


def check(lens, rows, T, H, group, D, dtype="bf16", tokens=None, **kw):
    """check_attend() of a call that is shared; tokens: of the table's width."""
    n = kw.get("before", 0) + sum(rows) + kw.get("behind", 0)
    hints = tokens is None
    width = max(-(-x // T) for x in lens) + 1 if hints else -(-tokens // T)
    assert is_shared(len(lens), n, T, H, group, D, dtype, width, max(rows) if hints else 0,
                     max(lens) if hints else 0)
    return check_attend(lens, rows, T, H, group, D, dtype, width=width, hints=hints, **kw)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("T", [16, 32, 64])
def test_shapes(T, D, dtype):
    check([1700, 33, 1, T, 650, 1537], [1] * 6, T, 2, 4, D, dtype, seed=T + D)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", DIMS)
def test_many_rows(D, dtype):
    check([1700, 3, 500, 1600], [40, 3, 0, 17], 16, 2, 3, D, dtype, seed=D)
    check([1550, 700, 1], [1, 90, 1], 64, 1, 2, D, dtype, seed=D + 1, tokens=1601)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H,group", [(1, 1), (3, 1), (5, 7), (1, 17), (2, 40), (7, 3)])
def test_groups(H, group, dtype):
    check([1601, 77, 900], [1, 1, 2], 16, H, group, 128, dtype, seed=group)
    check([1601, 77, 900], [1, 1, 2], 32, H, group, 64, dtype, seed=H)


def test_more_heads_than_shares_fit():
    """300 heads leave two shares a head."""
    check([1600, 70], [1, 1], 16, 300, 1, 64, tokens=4200, seed=4)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", DIMS)
def test_bad_pages(D, dtype):
    check([1700, 500, 64, 1], [1, 4, 1, 1], 16, 2, 4, D, dtype, seed=D, bad_pages=40)
    check([1700, 500, 64, 1], [30, 4, 1, 1], 64, 2, 2, D, dtype, seed=D + 1, bad_pages=8)
    got, lse = check([1600, 1700], [1, 9], 16, 1, 2, D, dtype, seed=D, edit=lambda q, c, t: t.fill(-1))
    assert np.all(got == 0) and np.all(np.isneginf(lse))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", DIMS)
def test_rows_that_see_nothing(D, dtype):
    """No tokens, fewer tokens than rows, negative lengths, requests without rows,
    rows of no request."""
    lens, rows = [0, 3, 1700, 20, -5, 1, 900], [2, 9, 0, 1, 1, 40, 3]
    got, lse = check(lens, rows, 16, 2, 2, D, dtype, seed=D, before=3, behind=6)
    assert np.all(got[3:5] == 0) and np.all(np.isneginf(lse[3:5]))
    check([0, 0, -1], [1, 1, 5], 16, 2, 2, D, dtype, tokens=1600)
    check([5, 5], [0, 0], 16, 2, 2, D, dtype, tokens=1600, behind=7)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", DIMS)
def test_nans(D, dtype):
    """NaN codes and queries in tiles that are shared; those of tokens that some
    rows of a tile do not see."""
    def edit(q, c, t):
        c.k[t[0, 50], 0, 3, 5] = 127
        c.v[t[1, 70], 1, 7, 9] = 255
        c.v[t[1, 2], 0, 15, 0] = 127
        c.v[t[2, 88], 1, 9, 33] = 255     # token 1417 of 1430, whose rows are tokens 1401 .. 1429
        c.k[t[2, 89], 0, 1, 3] = 127      # token 1425
        q[0, 3, 0] = math.nan
    got, lse = check([1700, 1500, 1430], [1, 1, 29], 16, 2, 2, D, dtype, seed=D, edit=edit)
    assert np.isnan(got[0, :2]).all() and np.isnan(got[0, 3]).all() and not np.isnan(got[0, 2]).any()
    assert np.isnan(got[1]).sum() == 4 and np.isnan(got[1, 2:, 9]).all() and np.isnan(got[1, :2, 0]).all()
    assert not np.isnan(got[2:18, 2:]).any() and np.isnan(got[18:, 2:, 33]).all()
    assert not np.isnan(got[2:26, :2]).any() and np.isnan(got[26:, :2]).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", DIMS)
def test_strides(D, dtype):
    check([1700, 37, 640], [1, 5, 2], 16, 2, 4, D, dtype, strides=True, seed=D)
    check([1700, 37, 64], [1, 50, 2], 64, 3, 2, D, dtype, strides=True, seed=D + 1)


@pytest.mark.parametrize("batch", [256, 257, 513, 700])
def test_many_requests(batch):
    """More requests than threads of a workgroup, most of them short, a few long."""
    rng = np.random.default_rng(batch)
    lens, rows = (rng.integers(a, b, batch).tolist() for a, b in ((-2, 30), (0, 3)))
    for i, n in zip((0, batch // 2, batch - 1), (4100, 3000, 2222)):
        lens[i], rows[i] = n, 2
    check(lens, rows, 16, 3, 2, 64, seed=batch)
    check(lens, rows, 64, 1, 20, 128, "fp16", seed=batch, behind=2)


@pytest.mark.parametrize("dtype", TYPES)
def test_loud_scores(dtype):
    check([1600, 1700], [1, 3], 16, 2, 4, 128, dtype, seed=5, mag=20.0)
    check([1600, 1700], [1, 30], 16, 2, 4, 256, dtype, seed=5, mag=20.0)
    check([1600, 1700], [1, 3], 16, 2, 4, 96, dtype, seed=6, scale=1e-6)
