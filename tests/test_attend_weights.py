"""CPU test of the bounds that attention's outputs are held to: weights in two
bfloat16 numbers are within them, weights rounded to one are far outside."""
import math

import numpy as np
import pytest
import torch

import cache_ref as R
from attend_bounds import cancelling_pairs, rounded_attend, to_bfloat16, two_part_bounds
from test_cache_gpu import new_pool


def test_rounding_is_torchs():
    x = torch.randn(5000, generator=torch.Generator().manual_seed(1))
    x[:3] = torch.tensor([1.0, 1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8])
    want = x.to(torch.bfloat16).double().numpy()
    assert np.array_equal(to_bfloat16(x.double().numpy()), want)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("T,D", [(16, 64), (64, 128), (32, 256)])
def test_bounds_tell_one_part_from_two(T, D, dtype):
    H, group, lens = 2, 4, [2, 8, 14, 30, 64, 150]
    ref = new_pool(40, T, H, D, seed=T)
    cancelling_pairs(ref)
    table = np.random.default_rng(T).integers(0, 40, (6, -(-150 // T)))
    dt = getattr(torch, dtype)
    q = (0.3 * torch.randn(6, H * group, D, generator=torch.Generator().manual_seed(D))).to(dt).double().numpy()
    want = R.attend(ref, q, table, lens, list(range(7)), 1 / math.sqrt(D))
    eps = torch.finfo(dt).eps / 2
    tol, _ = two_part_bounds(want, max(lens), D, eps)
    off = [np.abs(rounded_attend(ref, q, table, lens, 1 / math.sqrt(D), parts) - want[0]) for parts in (1, 2)]
    # (the output's own rounding is in the bound and not in what is compared)
    assert (off[1] <= tol - eps * np.abs(want[0])).all()
    assert [(o > tol).any() for o in off] == [True, False]
    assert (off[0] > 4 * tol).mean() > 0.01
