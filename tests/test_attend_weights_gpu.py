"""GPU test that attention multiplies the values by weights in two bfloat16
numbers, for both types of queries, in every form of the kernel."""
import ctypes as C

import pytest

import cache_ref as R
from attend_bounds import cancelling_pairs, two_part_bounds
from test_cache_gpu import check_attend

pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def bounds(monkeypatch):
    monkeypatch.setattr(R, "attend_bounds", two_part_bounds)


def pairs(q, cache, table):
    q *= 0.3
    cancelling_pairs(cache)


def is_shared(batch, rows, T, H, group, D, dtype, width, max_query=0, max_length=0):
    """Whether a call shares its tokens out over workgroups (it then has a workspace)."""
    from recv_fifo_plane_amd import xfer as X
    p = 1 << 40
    a = X.xfer_attend(p, p, None, p, p, p, None, 0, H * group * D, D, H * group * D, D, width, batch, rows,
                      H * group, width, 0 if dtype == "bf16" else 1, 1.0, max_query, max_length)
    n = C.c_size_t()
    assert X.lib().xfer_cache_attend_workspace(C.byref(X.xfer_cache_shape(T, H, D, 10)), C.byref(a),
                                               C.byref(n)) == 0
    return n.value > 0


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("T", [16, 64])
def test_single_rows(T, D, dtype):
    lens = [2, 8, 14, 30, 64, 150]
    check_attend(lens, [1] * 6, T, 2, 4, D, dtype, seed=T + D, nan_tail=False, edit=pairs)
    # a table of 1600 tokens, of which the requests use few
    assert is_shared(6, 6, T, 2, 4, D, dtype, 1600 // T)
    check_attend(lens, [1] * 6, T, 2, 4, D, dtype, seed=T + D, nan_tail=False, edit=pairs,
                 width=1600 // T, hints=False)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
def test_many_rows(D, dtype):
    lens, rows = [40, 8, 90], [33, 5, 20]
    check_attend(lens, rows, 16, 2, 3, D, dtype, seed=D, nan_tail=False, edit=pairs)
    check_attend(lens, rows, 16, 2, 3, D, dtype, seed=D, nan_tail=False, edit=pairs, width=100, hints=False)
