"""GPU tests of attention over the 4-bit cache against its plain form in 64 bits: types,
head sizes, groups, lengths, masks that leave nothing, and the ways in which a
call's work is shared."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import mxcache_ref as R  # noqa: E402
from mxcache_cases import (bounds, check_attend, gpu_cache, ints, is_shared, new_pool, starts_of,  # noqa: E402
                           table_of)

pytestmark = pytest.mark.gpu

DIMS = [64, 96, 128, 192, 256]
TYPES = ["bf16", "fp16"]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("T", [16, 32, 64])
def test_shapes(T, D, dtype):
    check_attend([1, T - 1, T, T + 1, 150, 333], [1] * 6, T, 2, 4, D, dtype, seed=T + D)
    check_attend([2, 40, 70, 65], [2, 11, 70, 33], T, 2, 3, D, dtype, seed=T + D)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("T", [16, 32, 64])
def test_shared_shapes(T, D, dtype):
    check_attend([1700, 33, 1, T, 650, 1537], [1] * 6, T, 2, 4, D, dtype, seed=T + D, shared=True)


@pytest.mark.parametrize("H,group", [(1, 1), (3, 1), (1, 2), (2, 3), (1, 5), (5, 7), (2, 8), (1, 15),
                                     (1, 16), (2, 17), (1, 40), (8, 1)])
def test_groups(H, group):
    check_attend([77, 1, 260], [1, 1, 1], 16, H, group, 128, seed=group)
    check_attend([77, 3, 130], [3, 2, 1], 32, H, group, 64, "fp16", seed=group)
    check_attend([1601, 77], [1, 2], 32, H, group, 96, seed=group)


@pytest.mark.parametrize("rows", [[2, 1, 5], [7, 64, 33], [0, 3, 0, 0, 1], [130, 1, 16, 17]])
@pytest.mark.parametrize("T", [16, 64])
def test_many_rows(rows, T):
    rng = np.random.default_rng(len(rows) * T)
    lens = [r + int(rng.integers(0, 200)) for r in rows]
    check_attend(lens, rows, T, 2, 3, 128, seed=T)
    check_attend(lens, rows, T, 1, 4, 64, "fp16", seed=T + 1, hints=False)
    check_attend(lens, rows, T, 1, 2, 256, seed=T + 2)
    check_attend(lens, rows, T, 1, 4, 192, "fp16", seed=T + 2)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", DIMS)
def test_whole_prompts(D, dtype):
    check_attend([300, 129, 1, 64], [300, 129, 1, 64], 16, 1, 2, D, dtype, seed=D)
    check_attend([200, 33], [200, 33], 64, 2, 1, D, dtype, seed=D, hints=False, before=2, behind=3)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", DIMS)
def test_shared_rows(D, dtype):
    check_attend([1700, 3, 500, 1600], [40, 3, 0, 17], 16, 2, 3, D, dtype, seed=D)
    check_attend([1550, 700, 1], [1, 90, 1], 64, 1, 2, D, dtype, seed=D + 1, hints=False, width=26)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", DIMS)
def test_rows_that_see_nothing(D, dtype):
    """No tokens, fewer tokens than rows, a negative length: 0 and -infinity."""
    got, lse = check_attend([0, 3, 0, 20, -5, 1], [2, 9, 0, 1, 1, 40], 16, 2, 2, D, dtype, seed=3)
    assert np.all(got[:2] == 0) and np.all(np.isneginf(lse[:2]))
    assert np.all(np.isneginf(lse[2:8])) and np.all(np.isfinite(lse[8:11]))
    got, lse = check_attend([0, 3, 1700, 20, -5, 1, 900], [2, 9, 0, 1, 1, 40, 3], 16, 2, 2, D, dtype,
                            seed=D, before=3, behind=6)
    assert np.all(got[3:5] == 0) and np.all(np.isneginf(lse[3:5]))
    check_attend([0, 0, -1], [1, 1, 5], 16, 2, 2, D, dtype, hints=False, width=100)
    check_attend([5, 5], [0, 0], 16, 2, 2, D, dtype, hints=False, width=100, behind=7)


def test_rows_of_no_request():
    check_attend([50, 9], [2, 1], 16, 2, 4, 128, before=3, behind=6)
    check_attend([50, 9, 300], [20, 1, 70], 32, 1, 3, 64, before=1, behind=17, hints=False)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", DIMS)
def test_bad_pages(D, dtype):
    """Table entries outside the cache leave their tokens out."""
    for T in (16, 64):
        check_attend([200, 500, 64, 1], [1, 4, 1, 1], T, 2, 4, D, dtype, seed=T, bad_pages=6)
        check_attend([200, 500, 64, 1], [40, 4, 64, 1], T, 2, 2, D, dtype, seed=T, bad_pages=6)
    check_attend([1700, 500, 64, 1], [1, 4, 1, 1], 16, 2, 4, D, dtype, seed=D, bad_pages=40)
    got, lse = check_attend([64, 1700], [1, 1], 64, 1, 2, D, dtype, seed=1, edit=lambda q, c, t: t.fill(-1))
    assert np.all(got == 0) and np.all(np.isneginf(lse))


def test_narrow_table():
    """Tokens past the table's width are left out."""
    check_attend([100, 500, 40], [1, 2, 1], 16, 2, 2, 128, width=4)
    check_attend([100, 500, 40], [100, 70, 40], 16, 2, 2, 128, width=4)
    check_attend([100, 5], [1, 2], 16, 2, 2, 128, width=0)


@pytest.mark.parametrize("D", DIMS)
def test_strides(D):
    check_attend([100, 37, 64], [1, 5, 2], 16, 2, 4, D, strides=True)
    check_attend([100, 37, 64], [1, 37, 2], 64, 3, 2, D, "fp16", strides=True)
    check_attend([1700, 37, 64], [1, 37, 2], 64, 1, 2, D, strides=True)


@pytest.mark.parametrize("hints", [True, False])
def test_long(hints):
    check_attend([9000, 33], [1, 1], 16, 1, 4, 128, seed=1, hints=hints)
    check_attend([7001, 5000], [3, 1], 64, 2, 2, 64, "fp16", seed=2, hints=hints)


@pytest.mark.parametrize("batch", [256, 257, 700])
def test_many_requests(batch):
    """More requests than threads of a workgroup, most of them short, a few long."""
    rng = np.random.default_rng(batch)
    lens, rows = (rng.integers(a, b, batch).tolist() for a, b in ((-2, 30), (0, 3)))
    for i, n in zip((0, batch // 2, batch - 1), (4100, 2900, 2222)):
        lens[i], rows[i] = n, 2
    check_attend(lens, rows, 16, 3, 2, 64, seed=batch)
    check_attend(lens, rows, 64, 1, 20, 128, "fp16", seed=batch, behind=2)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", DIMS)
def test_numbered_tiles(D, dtype):
    """Many requests whose largest number of rows is not known: tiles are numbered
    through the packed rows."""
    rng = np.random.default_rng(D)
    rows = rng.integers(0, 9, 90).tolist()
    lens = [max(0, r + int(rng.integers(-3, 120))) for r in rows]
    rows[40], lens[40] = 70, 200
    check_attend(lens, rows, 16, 2, 16, D, dtype, seed=D, hints=False)
    check_attend(lens, rows, 64, 2, 16, D, dtype, seed=D, bad_pages=9, before=5, behind=9, hints=False)


@pytest.mark.parametrize("dtype", TYPES)
def test_loud_scores(dtype):
    """One token far above the others, scores far below zero, values of all sizes."""
    for lens, rows in (([300, 40], [1, 3]), ([300, 140], [1, 130]), ([1600, 1700], [1, 30])):
        check_attend(lens, rows, 16, 2, 4, 128, dtype, seed=5, mag=20.0)
        check_attend(lens, rows, 16, 2, 4, 96, dtype, seed=6, scale=1e-6)

    def spread(q, c, t):
        rng = np.random.default_rng(1)
        c.s[:, :, 0] = rng.integers(100, 129, c.s[:, :, 0].shape)
        c.s[:, :, 1] = rng.integers(107, 147, c.s[:, :, 1].shape)
    for lens, rows in (([300, 700], [1, 3]), ([300, 170], [90, 130])):
        check_attend(lens, rows, 16, 2, 4, 128, dtype, seed=7, edit=spread, nan_tail=False)
        check_attend(lens, rows, 32, 2, 2, 192, dtype, seed=7, edit=spread, nan_tail=False)


def scaled(keys, values):
    def edit(q, cache, table):
        cache.s[:, :, 0] += np.uint8(keys % 256)
        cache.s[:, :, 1] += np.uint8(values % 256)
    return edit


@pytest.mark.parametrize("lens,rows", [([300, 40, 65], [1, 3, 30]), ([1700, 9], [1, 2]), ([160], [160])])
@pytest.mark.parametrize("dtype,mag,scale,keys", [
    ("fp16", 1e-6, 1e5, 0),            # queries below float16's normal numbers
    ("fp16", 6e4, 1e-6, 0),            # and near its largest
    ("fp16", 1.0, 2.0 ** -60, 58),
    ("fp16", 1.0, 2.0 ** 60, -62),
    ("bf16", 2.0 ** -100, 2.0 ** 97, 0),
    ("bf16", 2.0 ** 100, 2.0 ** -103, 0),
    ("bf16", 2.0 ** -60, 0.1, 60),
    ("bf16", 2.0 ** 60, 0.1, -60),
])
def test_ranges_of_scores(lens, rows, dtype, mag, scale, keys):
    check_attend(lens, rows, 16, 2, 4, 128, dtype, seed=3, mag=mag, scale=scale, edit=scaled(keys, 0),
                 nan_tail=False)


@pytest.mark.parametrize("lens,rows", [([300, 40, 65], [1, 3, 30]), ([1700, 9], [1, 2]), ([160], [160])])
@pytest.mark.parametrize("values", [100, -60, 60, 16])
def test_ranges_of_values(lens, rows, values):
    check_attend(lens, rows, 16, 2, 4, 128, "bf16", seed=4, edit=scaled(0, values), nan_tail=False)
    check_attend(lens, rows, 64, 1, 8, 256, "bf16", seed=4, edit=scaled(0, values), nan_tail=False)
    if values in (16, -60):
        check_attend(lens, rows, 64, 1, 8, 128, "fp16", seed=4, edit=scaled(0, min(values, 16)), nan_tail=False)


def pairs(q, cache, table):
    """Tokens 2i and 2i + 1 get nearly the same keys and opposite values: outputs are small
    beside the weights times the values, and show how weights are held."""
    q *= 0.3
    cache.k[:, :, 1::2] = cache.k[:, :, 0::2]
    cache.k[:, :, 1::2, :4] ^= 1
    cache.s[:, :, :, :, 1::2] = cache.s[:, :, :, :, 0::2]
    cache.v[:, :, 1::2] = cache.v[:, :, 0::2] ^ 8


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", DIMS)
def test_weights_that_cancel(D, dtype):
    lens = [2, 8, 14, 30, 64, 150]
    check_attend(lens, [1] * 6, 16, 2, 4, D, dtype, seed=D, nan_tail=False, edit=pairs)
    check_attend(lens, [1] * 6, 64, 2, 4, D, dtype, seed=D, nan_tail=False, edit=pairs, width=100, hints=False)
    check_attend([40, 8, 90, 200], [33, 5, 20, 180], 16, 2, 3, D, dtype, seed=D, nan_tail=False, edit=pairs)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", DIMS)
def test_not_finite(D, dtype):
    """A NaN that a row sees makes that row and head NaN: all of it where a key has it, its 32
    dims where a value has it; and no other row."""
    def edit(q, c, t):
        c.s[t[0, 2], 0, 0, 1, 3] = 255
        c.s[t[1, 1], 1, 1, 0, 7] = 255
        q[2, 3, 0] = math.nan
    got, lse = check_attend([100, 90, 80], [1, 1, 1], 16, 2, 2, D, dtype, seed=8, edit=edit)
    assert np.isnan(got[0, :2]).all() and not np.isnan(got[0, 2:]).any()
    assert np.isnan(got[1, 2:, :32]).all() and np.isnan(got[1]).sum() == 64


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
        got, lse = check_attend([40, 130], rows, 16, 2, 3, D, dtype, seed=8, edit=edit)
        assert not np.isnan(got[:5, :3]).any() and np.isnan(got[5:20, :3, :32]).all()
        assert not np.isnan(got[:13, 3:]).any() and np.isnan(got[13:20, 3:]).all()
        first = 20 + rows[1] - 130 + 96
        assert np.isnan(got[first:, 3:, -32:]).all() and not np.isnan(got[20:first]).any()
    got, lse = check_attend([1700, 1500, 1430], [1, 1, 29], 16, 2, 2, D, dtype, seed=D, edit=lambda q, c, t:
                            c.s[t[2, 88], 1, 1, 0].__setitem__((9,), 255) or c.s[t[0, 50], 0, 0, last].__setitem__((3,), 255))
    assert np.isnan(got[0, :2]).all() and not np.isnan(got[0, 2:]).any()
    assert not np.isnan(got[1]).any() and not np.isnan(got[2:18]).any()
    assert np.isnan(got[18:, 2:, :32]).all()


def test_wrong_hints():
    """Hints that are too small only shape the launch."""
    T, H, D = 16, 1, 128
    ref = new_pool(300, T, H, D, 1)
    gpu = gpu_cache(ref)
    lens, rows = [1900, 700], [90, 3]
    table = np.arange(240).reshape(2, 120)
    q = torch.randn(93, 4, D, device="cuda").to(torch.bfloat16)
    want = R.attend(ref, q.double().cpu().numpy(), table.tolist(), lens, starts_of(rows), 1 / math.sqrt(D))
    tol, tol_lse = bounds(want, 1900, D, "bf16", False)
    for mq, ml in ((0, 0), (1, 1), (1, 0), (0, 5), (20, 64), (93, 1900), (5000, 1 << 30)):
        got, lse = gpu.attend(q, table_of(table), ints(lens), ints(starts_of(rows)), max_query=mq,
                              max_length=ml, lse=True)
        assert np.all(np.abs(got.double().cpu().numpy() - want[0]) <= tol), (mq, ml)
        assert np.all(np.abs(lse.double().cpu().numpy() - want[1]) <= tol_lse), (mq, ml)


def test_same_twice():
    """The same call gives the same bits."""
    gpu = gpu_cache(new_pool(400, 16, 2, 128, 1))
    t = ints(np.arange(390)).reshape(3, 130)
    for rows in ([1, 1, 1], [60, 200, 9]):
        q = torch.randn(sum(rows), 8, 128, device="cuda").to(torch.bfloat16)
        a = [gpu.attend(q, t, ints([2000, 1999, 70]), ints(starts_of(rows)), lse=True) for _ in range(5)]
        for x in a[1:]:
            assert torch.equal(x[0], a[0][0]) and torch.equal(x[1], a[0][1])


def test_nothing():
    gpu = gpu_cache(new_pool(4, 16, 2, 64, 1))
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    o, l = gpu.attend(q, ints([]).reshape(0, 3), ints([]), ints([0]), lse=True)
    assert o.shape == (0, 4, 64) and l.shape == (0, 4)
    q = torch.full((3, 4, 64), 2.0, dtype=torch.bfloat16, device="cuda")
    o = torch.full((3, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    gpu.attend(q, ints([]).reshape(0, 3), ints([]), ints([0]), out=o)
    gpu.attend(q, ints([0] * 6).reshape(2, 3), ints([0, 0]), ints([0, 0, 0]), out=o)
    torch.cuda.synchronize()
    assert torch.all(o == 5.0)


def test_rows_are_aligned_to_their_elements():
    T, H, group, D = 16, 2, 3, 96
    c = gpu_cache(new_pool(40, T, H, D, 3))
    n, heads = 5, H * group
    table, lens, starts = ints(range(36)).reshape(3, 12), ints([150, 33, 190]), ints([0, 1, 3, 5])
    for dtype in (torch.bfloat16, torch.float16):
        q = torch.randn(n, heads, D, device="cuda").to(dtype)
        want = c.attend(q, table, lens, starts)
        flat = torch.zeros(n * (heads * (D + 3) + 5) + 9, dtype=dtype, device="cuda")
        odd = flat[1:].as_strided((n, heads, D), (heads * (D + 3) + 5, D + 3, 1))
        odd.copy_(q)
        out = torch.full((n * heads * (D + 1) + 9,), 7.0, dtype=dtype, device="cuda")
        got = out[3:].as_strided((n, heads, D), (heads * (D + 1), D + 1, 1))
        c.attend(odd, table, lens, starts, out=got)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.all(out[:3] == 7.0) and torch.all(out[3 + D::D + 1] == 7.0)


def test_shared_is_told():
    assert is_shared(2, 2, 16, 2, 4, 128, "bf16", 500) and not is_shared(2, 2, 16, 2, 4, 128, "bf16", 10)
