"""GPU tests of how tiles of many rows hold the weights of attention over the 4-bit cache: as two
numbers, as tiles of few rows do, whatever shape a call has."""
import math

import pytest

torch = pytest.importorskip("torch")
import mxcache_cases  # noqa: E402
from attend_bounds import two_part_bounds  # noqa: E402
from mxcache_cases import check_attend, gpu_cache, ints, new_pool  # noqa: E402
from test_mxcache_attend_gpu import DIMS, TYPES, pairs  # noqa: E402

pytestmark = pytest.mark.gpu


def two_numbers(want, tokens, D, dtype, wide):
    """As mxcache_cases.bounds, but every weight is off by 2^-16 at most, and 2^-32 of the row's
    largest: of a weight w, a float16 number leaves 2^-11 w or 2^-25, and a second one 2^-11 of that or
    2^-25, the reference being such that the row's largest is 2^7 or more."""
    tol, tol_lse = two_part_bounds(want[:4], tokens, D if dtype == "bf16" else 2 * D,
                                   2.0 ** -8 if dtype == "bf16" else 2.0 ** -11)
    return tol + 1.01 * 2.0 ** -32 * want[4] * 1.01, tol_lse


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", DIMS)
def test_weights_are_two_numbers(D, dtype, monkeypatch):
    """Outputs that are small beside the weights times the values: in shares, by tiles, and where
    the scales ask for bfloat16 numbers."""
    monkeypatch.setattr(mxcache_cases, "bounds", two_numbers)

    def far(q, cache, table):
        pairs(q, cache, table)
        cache.s[:, :, 1] += 20  # beyond float16's

    for edit in (pairs, far) if dtype == "bf16" else (pairs,):
        check_attend([40, 8, 90, 200], [33, 5, 20, 180], 16, 2, 3, D, dtype, seed=D, nan_tail=False, edit=edit, many=0)
        H = 32 if D <= 128 else 16
        check_attend([190, 200, 0, 33], [190, 199, 1, 17], 16, H, 4, D, dtype, seed=D, nan_tail=False, edit=edit,
                     many=1216, shared=False)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shift", [7, -19])
def test_weights_at_the_ends_of_float16_values(shift, dtype, monkeypatch):
    """Values with scales of 130 .. 135 and of 104 .. 109, the ends of those that float16 numbers can hold
    (-19: the values are below its normal numbers)."""
    monkeypatch.setattr(mxcache_cases, "bounds", two_numbers)

    def edit(q, cache, table):
        pairs(q, cache, table)
        cache.s[:, :, 1] += shift % 256
        assert cache.s[:, :, 1].min() >= 104 and cache.s[:, :, 1].max() <= 135

    for D in DIMS:
        check_attend([40, 8, 90, 200], [33, 5, 20, 180], 16, 2, 3, D, dtype, seed=D, nan_tail=False, edit=edit, many=0)
        check_attend([300, 160], [70, 160], 32, 2, 4, D, dtype, seed=4, nan_tail=False, edit=edit, many=0)


@pytest.mark.parametrize("many", [False, True])
def test_weights_that_grow_beside_large_values(many):
    """Values near the largest of the documented range (values times tokens below 2^119) where
    the later chunks' scores are the larger ones: weights reach 2^7.5 of the first chunk's."""
    T, H, D, group, length = 16, 32 if many else 1, 128, 4, 400
    rows = 400 if many else 8
    c = new_pool(26, T, H, D, 1)
    c.k[:], c.v[:] = 0, 7
    c.s[:, :, 0], c.s[:, :, 1] = 127, 127 + 107
    for t in range(67, length, 16):
        c.k[t // T, :, t % T, 0] = 7
    q = torch.zeros(rows, H * group, D, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1
    table = torch.full((1, 76), -1, dtype=torch.int32, device="cuda")
    table[0, :26] = torch.arange(26)
    out = gpu_cache(c).attend(q, table, ints([length]), ints([0, rows]), scale=7.5 * math.log(2.0) / 6)
    assert torch.all(out.double() == 6 * 2.0 ** 107)  # (all values are that, and bfloat16 holds it)
