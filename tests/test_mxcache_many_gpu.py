"""GPU tests of attention over the 4-bit cache where calls are large enough for tiles of many
rows: in shares of all work, by tiles, and by numbered tiles."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import mxcache_ref as R  # noqa: E402
from mxcache_cases import (bounds, check_attend, gpu_cache, ints, many_length, new_pool, starts_of,  # noqa: E402
                           table_of)
from test_mxcache_attend_gpu import DIMS, TYPES, pairs, scaled  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("T", [16, 64])
def test_shapes(T, D, dtype):
    check_attend([2, 40, 70, 65], [2, 11, 70, 33], T, 2, 3, D, dtype, seed=T + D, many=0, shared=True)
    check_attend([1700, 3, 500, 1600], [40, 3, 0, 17], T, 2, 3, D, dtype, seed=D, many=0, shared=True)
    check_attend([300, 129, 1, 64], [300, 129, 1, 64], T, 1, 2, D, dtype, seed=D, many=0, shared=True)


@pytest.mark.parametrize("rows", [[2, 1, 25], [7, 64, 33], [0, 33, 0, 0, 1], [130, 1, 16, 17], [129, 128, 127]])
def test_many_rows(rows):
    rng = np.random.default_rng(len(rows))
    lens = [r + int(rng.integers(0, 200)) for r in rows]
    check_attend(lens, rows, 16, 2, 3, 128, seed=1, many=0, shared=True)
    check_attend(lens, rows, 32, 1, 4, 64, "fp16", seed=2, hints=False, many=0, shared=True)
    check_attend(lens, rows, 64, 1, 2, 256, seed=3, many=0, shared=True)
    check_attend(lens, rows, 16, 1, 4, 192, "fp16", seed=4, many=0, before=3, behind=6)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", DIMS)
def test_by_tiles(D, dtype):
    """Short requests with many rows and heads: a workgroup for each tile, no shares."""
    H, group = (32, 4) if D <= 128 else (16, 4)
    check_attend([190, 200, 0, 33], [190, 199, 1, 17], 16, H, group, D, dtype, seed=D, many=1216, shared=False,
                 before=1, behind=2)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 128, 192])
def test_by_numbered_tiles(D, dtype):
    """The same among many requests, whose largest number of rows is not known."""
    rng = np.random.default_rng(D)
    rows = rng.integers(0, 5, 90).tolist()
    rows[40] = 190
    lens = [max(0, r + int(rng.integers(-3, 40))) for r in rows]
    check_attend(lens, rows, 16, 16, 8, D, dtype, seed=D, many=1216, shared=False, hints=False, behind=3)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", DIMS)
def test_rows_that_see_nothing(D, dtype):
    got, lse = check_attend([0, 3, 0, 20, -5, 1], [2, 9, 0, 1, 1, 40], 16, 2, 2, D, dtype, seed=3, many=0)
    assert np.all(got[:2] == 0) and np.all(np.isneginf(lse[:2]))
    assert np.all(np.isneginf(lse[2:8])) and np.all(np.isfinite(lse[8:11]))
    check_attend([0, 50, -1], [1, 140, 5], 16, 2, 2, D, dtype, hints=False, many=0)
    got, lse = check_attend([0, 0], [40, 70], 16, 2, 2, D, dtype, many=0)
    assert np.all(got == 0) and np.all(np.isneginf(lse))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", DIMS)
def test_bad_pages(D, dtype):
    for T in (16, 64):
        check_attend([200, 500, 64, 1], [40, 40, 64, 1], T, 2, 2, D, dtype, seed=T, bad_pages=6, many=0)
    got, lse = check_attend([64, 300], [40, 50], 64, 1, 2, D, dtype, seed=1, edit=lambda q, c, t: t.fill(-1), many=0)
    assert np.all(got == 0) and np.all(np.isneginf(lse))


@pytest.mark.parametrize("D", DIMS)
def test_strides(D):
    check_attend([100, 37, 64], [60, 37, 2], 64, 3, 2, D, "fp16", strides=True, many=0)
    check_attend([1700, 37, 64], [90, 37, 2], 64, 1, 2, D, strides=True, many=0)


@pytest.mark.parametrize("batch", [256, 300])
def test_many_requests(batch):
    """More requests than threads of a workgroup, most of them short, one with many rows."""
    rng = np.random.default_rng(batch)
    lens, rows = (rng.integers(a, b, batch).tolist() for a, b in ((-2, 30), (0, 3)))
    lens[batch // 2], rows[batch // 2] = 1200, 170
    check_attend(lens, rows, 16, 3, 2, 64, seed=batch, many=0, shared=True)
    check_attend(lens, rows, 64, 1, 20, 128, "fp16", seed=batch, behind=2, many=0, hints=False)


@pytest.mark.parametrize("dtype", TYPES)
def test_loud_scores(dtype):
    def spread(q, c, t):
        rng = np.random.default_rng(1)
        c.s[:, :, 0] = rng.integers(100, 129, c.s[:, :, 0].shape)
        c.s[:, :, 1] = rng.integers(107, 147, c.s[:, :, 1].shape)
    for lens, rows in (([300, 140], [20, 130]), ([1600, 1700], [1, 60])):
        check_attend(lens, rows, 16, 2, 4, 128, dtype, seed=5, mag=20.0, many=0)
        check_attend(lens, rows, 16, 2, 4, 96, dtype, seed=6, scale=1e-6, many=0)
        check_attend(lens, rows, 16, 2, 4, 128, dtype, seed=7, edit=spread, nan_tail=False, many=0)
        check_attend(lens, rows, 32, 2, 2, 192, dtype, seed=7, edit=spread, nan_tail=False, many=0)


@pytest.mark.parametrize("dtype,mag,scale,keys", [
    ("fp16", 1e-6, 1e5, 0), ("fp16", 6e4, 1e-6, 0), ("fp16", 1.0, 2.0 ** -60, 58), ("fp16", 1.0, 2.0 ** 60, -62),
    ("bf16", 2.0 ** -100, 2.0 ** 97, 0), ("bf16", 2.0 ** 100, 2.0 ** -103, 0), ("bf16", 2.0 ** -60, 0.1, 60),
    ("bf16", 2.0 ** 60, 0.1, -60)])
def test_ranges_of_scores(dtype, mag, scale, keys):
    for D in (128, 256):
        check_attend([300, 160], [70, 160], 16, 2, 4, D, dtype, seed=3, mag=mag, scale=scale,
                     edit=scaled(keys, 0), nan_tail=False, many=0)


@pytest.mark.parametrize("values", [100, -60, 60, 16, -23, 8, 9, -24])
def test_ranges_of_values(values):
    for D in (64, 128, 256):
        check_attend([300, 160], [70, 160], 16, 2, 4, D, "bf16", seed=4, edit=scaled(0, values), nan_tail=False, many=0)
        if -60 <= values <= 16:
            check_attend([300, 160], [70, 160], 64, 1, 8, D, "fp16", seed=4, edit=scaled(0, values), nan_tail=False,
                         many=0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", DIMS)
def test_weights_that_cancel(D, dtype):
    check_attend([40, 8, 90, 200], [33, 5, 20, 180], 16, 2, 3, D, dtype, seed=D, nan_tail=False, edit=pairs, many=0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", DIMS)
def test_nan_of_unseen_tokens(D, dtype):
    """A NaN stored for a token reaches the rows that see it, not the earlier ones of its tile."""
    last = D // 32 - 1

    def edit(q, c, t):
        c.s[t[0, 1], 0, 1, 0, 9] = 255       # token 25 of 40, whose rows are tokens 20 .. 39
        c.s[t[0, 2], 1, 0, last, 1] = 255    # token 33
        c.s[t[1, 6], 1, 1, last, 0] = 255    # token 96 of 130
    for rows in ([20, 60], [20, 130]):
        got, lse = check_attend([40, 130], rows, 16, 2, 3, D, dtype, seed=8, edit=edit, many=0)
        assert not np.isnan(got[:5, :3]).any() and np.isnan(got[5:20, :3, :32]).all()
        assert not np.isnan(got[:13, 3:]).any() and np.isnan(got[13:20, 3:]).all()
        first = 20 + rows[1] - 130 + 96
        assert np.isnan(got[first:, 3:, -32:]).all() and not np.isnan(got[20:first]).any()


@pytest.mark.parametrize("D", [128, 256])
def test_wrong_hints(D):
    """Hints that are too small only shape the launch."""
    T, H = 16, 1
    ref = new_pool(300, T, H, D, 1)
    gpu = gpu_cache(ref)
    lens, rows = [1900, 700], [90, 3]
    told = many_length(93, H, 4, D)
    table = np.full((2, told // T), -1)
    table[:, :120] = np.arange(240).reshape(2, 120)
    q = torch.randn(93, 4, D, device="cuda").to(torch.bfloat16)
    want = R.attend(ref, q.double().cpu().numpy(), table.tolist(), lens, starts_of(rows), 1 / math.sqrt(D))
    tol, tol_lse = bounds(want, 1900, D, "bf16", True)
    for mq, ml in ((0, 0), (9, 0), (20, told), (93, told), (5000, 1 << 30)):
        got, lse = gpu.attend(q, table_of(table), ints(lens), ints(starts_of(rows)), max_query=mq,
                              max_length=ml, lse=True)
        assert np.all(np.abs(got.double().cpu().numpy() - want[0]) <= tol), (mq, ml)
        assert np.all(np.abs(lse.double().cpu().numpy() - want[1]) <= tol_lse), (mq, ml)


def test_same_twice():
    """The same call gives the same bits."""
    gpu = gpu_cache(new_pool(400, 16, 2, 128, 1))
    t = torch.full((3, 30000), -1, dtype=torch.int32, device="cuda")
    t[:, :130] = ints(np.arange(390)).reshape(3, 130)
    q = torch.randn(269, 8, 128, device="cuda").to(torch.bfloat16)
    a = [gpu.attend(q, t, ints([2000, 1999, 70]), ints(starts_of([60, 200, 9])), lse=True) for _ in range(5)]
    for x in a[1:]:
        assert torch.equal(x[0], a[0][0]) and torch.equal(x[1], a[0][1])
