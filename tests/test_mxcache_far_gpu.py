"""GPU tests of attention over the 4-bit cache where scores are far from 0: a row's largest one
still decides, however coarse a float is there."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from mxcache_cases import DT, gpu_cache, ints, many_length, new_pool, starts_of, table_of  # noqa: E402
from test_mxcache_attend_gpu import DIMS, TYPES  # noqa: E402

pytestmark = pytest.mark.gpu


def far_scores(D, dtype, power, many, values=0, first=5):
    """Rows whose queries have one number, a, and a cache whose keys have one, c, so a score is
    a * c * 2^power exactly.  c is 2, 3 or 4, but 6 for two tokens and 0.5 for two others: of
    a row with a > 0 the first two have all weight but exp(-2^(power - 1)) of it, of one with a < 0 the
    others.  They have the same score, so half of it each (of rows that see both)."""
    T, H, group, lens, rows = 16, 2, 2, [200, 150], [100, 66]
    rng = np.random.default_rng(D + power)
    n, heads, pages = sum(rows), H * group, 13
    ref = new_pool(2 * pages, T, H, D, D + power)
    ref.s[:, :, 0] = 127
    ref.s[:, :, 1] += np.uint8(values % 256)
    table = rng.permutation(2 * pages).reshape(2, pages)
    ref.k[:] = 0
    ref.k[..., 1] = rng.choice([4, 5, 6], ref.k[..., 1].shape)
    peaks = {1: (first, first + 67), -1: (first + 3, first + 64)}
    for b in range(2):
        for sign, code in ((1, 7), (-1, 1)):
            for t in peaks[sign]:
                ref.k[table[b, t // T], :, t % T, 1] = code
    a = rng.choice([-1, 1], (n, heads)) * (1 + rng.integers(0, 128, (n, heads)) / 128)
    q = np.zeros((n, heads, D))
    q[..., 1] = a
    starts = starts_of(rows)
    width = -(-many_length(n, H, group, D) // T) if many else pages
    wide = np.full((2, width), -1)
    wide[:, :pages] = table
    out, lse = gpu_cache(ref).attend(torch.tensor(q).to(DT[dtype]).cuda(), table_of(wide), ints(lens), ints(starts),
                                     scale=2.0 ** power, lse=True, max_query=max(rows))
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for i in range(n):
        b = int(i >= rows[0])
        for g in range(heads):
            sign = 1 if a[i, g] > 0 else -1
            last = lens[b] - rows[b] + i - starts[b]
            v = [ref.tokens(1, [table[b, t // T]], g // group, [t % T])[0] for t in peaks[sign] if t <= last]
            # Of the same score, so of the same weight, held in 11 bits at worst (2^-11); 12 roundings of a
            # sum of two; then the output's own.
            want, mag = sum(v) / len(v), sum(np.abs(x) for x in v) / len(v)
            eps = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
            tol = 1.01 * (eps * np.abs(want) + (2.0 ** -11 + 12 * 2.0 ** -24) * mag)
            if dtype == "fp16":
                tol = tol + 2.0 ** -25  # half a step below its normal numbers
            assert np.all(np.abs(out[i, g] - want) <= tol), (i, g, a[i, g])
            # roundings of: scale times log2(e), two; the score times it; maximum and sum's logarithm
            # joined; ln 2; the product; what the logarithm is off by, in units of its argument's rounding
            x = a[i, g] * (6.0 if sign > 0 else 0.5) * 2.0 ** power + np.log(len(v))
            assert abs(lse[i, g] - x) <= 8 * 2.0 ** -24 * abs(x), (i, g, lse[i, g], x)


@pytest.mark.parametrize("power", [12, 18, 20, 24, 27, 29, 33, 60, 100])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("many", [False, True])
def test_far_scores(many, dtype, power):
    far_scores(128, dtype, power, many)
    far_scores(64, dtype, power, many, first=66)  # (the second chunk's)


@pytest.mark.parametrize("power", [14, 31, 47])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", DIMS)
def test_far_scores_of_all_dims(D, dtype, power):
    far_scores(D, dtype, power, True)
    # values that no float16 number is
    far_scores(D, dtype, power, True, values=-27 if dtype == "fp16" else 30, first=20)
