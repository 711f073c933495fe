"""CPU tests of the 4-bit cache's plain forms, which the GPU tests compare with."""
import numpy as np
import pytest

import mxcache_ref as R


def test_codes():
    assert R.CODES[:8].tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert np.array_equal(R.CODES[8:], -R.CODES[:8])
    assert R.to_codes(R.CODES[1:]).tolist() == list(range(1, 16))  # (-0 is code 8)
    ties = {0.25: 0, 0.75: 1, 1.25: 1, 1.75: 2, 2.5: 2, 3.5: 4, 5: 4, 7: 6, 8: 6}
    for x, want in ties.items():
        assert R.CODES[R.to_codes(x)] == want and R.CODES[R.to_codes(-x)] == -want
        below, above = (R.CODES[R.to_codes(np.nextafter(x, to))] for to in (0, 9))
        assert below <= want <= above and (below < above or x >= 6)


def test_scales():
    """Up to 7 times the scale a number is off by at most the scale; that is half of the
    largest codes' distance."""
    for e in (-118, -3, 0, 125):
        assert R.exponent_of(7 * 2.0 ** e) == e
        assert R.exponent_of(np.nextafter(7 * 2.0 ** e, np.inf)) == min(e + 1, 125)
    assert R.exponent_of(0.0) == -118
    x = np.linspace(0, 7, 10001)
    assert np.abs(R.CODES[R.to_codes(x)] - x).max() <= 1.0


@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("T", [16, 32, 64])
def test_records(T, D):
    """The arrays hold every byte of a record, and a byte's place is the documented one."""
    H = 3
    raw = np.random.default_rng(T + D).integers(0, 256, (4, R.block_bytes(T, H, D)), dtype=np.uint8)
    c = R.Cache(raw, T, H, D)
    assert np.array_equal(c.raw(), raw) and raw.shape[1] % 128 == 0
    for b, h, t, d in np.random.default_rng(1).integers(0, (4, H, T, D), (200, 4)):
        shift = 4 * (d % 2)
        assert c.k[b, h, t, d] == raw[b, h * T * D + t * (D // 2) + d // 2] >> shift & 15
        at = 0
        for P in R.PARTS[D]:
            if at <= d < at + P:
                break
            at += P
        wide = P // 32
        u, n, k = 16 // wide, (d - at) // (2 * wide), (d - at) % (2 * wide) // 2
        byte = h * T * D + T * D // 2 + T * at // 2 + (t // u * 16 + n) * 16 + t % u * wide + k
        assert c.v[b, h, t, d] == raw[b, byte] >> shift & 15
        for side in range(2):
            s = raw[b, H * T * D + ((h * 2 + side) * (D // 32) + d // 32) * T + t]
            assert c.s[b, h, side, d // 32, t] == s


def test_store_and_load():
    T, H, D = 16, 2, 64
    c = R.Cache(np.zeros((3, R.block_bytes(T, H, D)), np.uint8), T, H, D)
    rng = np.random.default_rng(0)
    key, value = rng.normal(size=(2, 20, H, D))
    key[3, 1, 40] = np.nan
    slots = [32 + i for i in range(16)] + [0, 1, -1, 2]
    R.store(c, key, value, slots)
    k, v, real = R.load(c, [[2, 0]], [19], [0, 19], 20)
    assert real.tolist() == [True] * 19 + [False]
    order = list(range(18)) + [19]
    assert np.isnan(k[3, 1, 32:]).all() and np.isnan(k).sum() == 32
    for got, x in ((k, key), (v, value)):
        near = np.abs(got[:19] - x[order]).reshape(19, H, 2, 32)
        far = np.abs(x[order]).reshape(19, H, 2, 32).max(-1, keepdims=True)
        assert np.nanmax(near / far) <= 1 / 3.5      # off by the scale, which is over far / 7 / 2
    back = R.load(c, [[2, 0]], [2], [0, 5], 5)[0]    # three rows before the first token
    assert np.all(back[:3] == 0) and np.array_equal(back[3:], k[:2])
