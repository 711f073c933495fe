"""GPU tests of attention at the ends of its types' ranges."""
import numpy as np
import pytest

import cache_ref as R
from attend_bounds import two_part_bounds
from test_cache_gpu import check_attend

pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def bounds(monkeypatch):
    monkeypatch.setattr(R, "attend_bounds", two_part_bounds)


def scaled(keys, values):
    def edit(q, cache, table):
        cache.s[:, :, 0] *= np.float32(keys)
        cache.s[:, :, 1] *= np.float32(values)
    return edit


@pytest.mark.parametrize("lens,rows", [([300, 40, 65], [1, 3, 30]), ([1700, 9], [1, 2])])
@pytest.mark.parametrize("dtype,mag,scale,keys", [
    ("fp16", 1e-6, 1e5, 1.0),            # queries below float16's normal numbers
    ("fp16", 6e4, 1e-6, 1.0),            # and near its largest
    ("fp16", 1.0, 2.0 ** -60, 2.0 ** 58),
    ("bf16", 2.0 ** -100, 2.0 ** 97, 1.0),
    ("bf16", 2.0 ** 100, 2.0 ** -103, 1.0),
    ("bf16", 2.0 ** -60, 0.1, 2.0 ** 60),
    ("bf16", 2.0 ** 60, 0.1, 2.0 ** -60),
])
def test_scores(lens, rows, dtype, mag, scale, keys):
    check_attend(lens, rows, 16, 2, 4, 128, dtype, seed=3, mag=mag, scale=scale, edit=scaled(keys, 1.0))


@pytest.mark.parametrize("lens,rows", [([300, 40, 65], [1, 3, 30]), ([1700, 9], [1, 2])])
@pytest.mark.parametrize("values", [2.0 ** 100, 2.0 ** -60, 2.0 ** 60])
def test_values(lens, rows, values):
    check_attend(lens, rows, 16, 2, 4, 128, "bf16", seed=4, edit=scaled(1.0, values))
    check_attend(lens, rows, 64, 1, 8, 256, "bf16", seed=4, edit=scaled(1.0, values))
