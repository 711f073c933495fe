"""Plain forms of the 4-bit cache's operators, and of reading either cache back, for
the tests: loops over rows and requests, in 64 bits, on the CPU."""
from __future__ import annotations

import math

import numpy as np

# The value of each of the 16 codes: 1 sign, 2 exponent (bias 1), 1 mantissa bit.
CODES = np.array([(-1.0) ** (c >> 3) * ((c & 1) / 2 if (c >> 1 & 3) == 0
                                        else (1 + (c & 1) / 2) * 2.0 ** ((c >> 1 & 3) - 1))
                  for c in range(16)])
PARTS = {64: (64,), 96: (64, 32), 128: (128,), 192: (128, 64), 256: (128, 128)}


def block_bytes(T, H, D):
    return H * T * D + (H * T * D // 16 + 127) // 128 * 128


def to_codes(x):
    """Nearest codes of float64 numbers, ties to the even one; beyond 6, 6."""
    x = np.asarray(x, dtype=np.float64)
    far = np.abs(np.abs(x)[..., None] - CODES[:8])
    near = np.min(far, -1, keepdims=True)
    hit = far == near
    even = hit & (np.arange(8) % 2 == 0)
    pick = np.where(hit.sum(-1) > 1, even.argmax(-1), hit.argmax(-1))
    return (pick | np.where(np.signbit(x), 8, 0)).astype(np.uint8)


def exponent_of(amax):
    """The smallest e, -118 at least and 125 at most, with amax <= 7 * 2^e."""
    e = -118
    while e < 125 and amax > 7 * 2.0 ** e:
        e += 1
    return e


class Cache:
    """A pool as arrays: codes of keys and values [blocks, H, T, D], bytes of scale
    [blocks, H, 2, D / 32, T]."""

    def __init__(self, raw, T, H, D):
        n = raw.shape[0]
        assert raw.shape[1] == block_bytes(T, H, D)
        self.T, self.H, self.D, self.blocks = T, H, D, n
        body = raw[:, :H * T * D].reshape(n, H, 2, T * D // 2)
        self.k = self._split(body[:, :, 0].reshape(n, H, T, D // 2))
        cols, at = [], 0
        for P in PARTS[D]:
            b = P // 32
            part = body[:, :, 1, at:at + T * P // 2].reshape(n, H, b * T // 16, 16, 16 // b, b)
            cols.append(part.transpose(0, 1, 2, 4, 3, 5).reshape(n, H, T, P // 2))
            at += T * P // 2
        self.v = self._split(np.concatenate(cols, -1))
        scales = H * T * D // 16
        self.s = raw[:, H * T * D:H * T * D + scales].reshape(n, H, 2, D // 32, T).copy()
        self.pad = raw[:, H * T * D + scales:].copy()

    @staticmethod
    def _split(x):
        return np.stack([x & 15, x >> 4], -1).reshape(x.shape[:-1] + (-1,))

    def raw(self):
        n, H, T, D = self.blocks, self.H, self.T, self.D
        k, v = (x[..., 0::2] | x[..., 1::2] << 4 for x in (self.k, self.v))
        cols, at = [], 0
        for P in PARTS[D]:
            b = P // 32
            part = v[..., at // 2:(at + P) // 2].reshape(n, H, b * T // 16, 16 // b, 16, b)
            cols.append(part.transpose(0, 1, 2, 4, 3, 5).reshape(n, H, -1))
            at += P
        body = np.concatenate([k.reshape(n, H, -1)] + cols, 2)
        return np.concatenate([body.reshape(n, -1), self.s.reshape(n, -1), self.pad], 1)

    def tokens(self, side, ids, h, places):
        """float64 [len(ids), D] of one head at some blocks and places."""
        codes = (self.v if side else self.k)[ids, h, places]
        s = self.s[ids, h, side, :, places].astype(np.float64)
        power = np.where(s == 255, np.nan, 2.0 ** (np.minimum(s, 254) - 127))
        return CODES[codes] * np.repeat(power, 32, -1)


class Eight:
    """As Cache.tokens, of a pool of 8 bits (a cache_ref.Cache)."""

    def __init__(self, c):
        import cache_ref as R
        self.c, self.values = c, R.VALUES
        self.T, self.H, self.D, self.blocks = c.T, c.H, c.D, c.blocks

    def tokens(self, side, ids, h, places):
        codes = (self.c.v if side else self.c.k)[ids, h, places]
        return self.values[codes] * self.c.s[ids, h, side].astype(np.float64)[:, None]


def store(cache, key, value, slots):
    """Stores float64 rows [rows, H, D] into `cache`."""
    for n, slot in enumerate(slots):
        if slot < 0 or slot // cache.T >= cache.blocks:
            continue
        b, t = slot // cache.T, slot % cache.T
        for side, (codes, x) in enumerate(((cache.k, key), (cache.v, value))):
            for h in range(cache.H):
                for g in range(cache.D // 32):
                    new = x[n, h, 32 * g:32 * g + 32]
                    if not np.isfinite(new).all():
                        codes[b, h, t, 32 * g:32 * g + 32] = 0
                        cache.s[b, h, side, g, t] = 255
                        continue
                    e = exponent_of(np.abs(new).max())
                    codes[b, h, t, 32 * g:32 * g + 32] = to_codes(new / 2.0 ** e)
                    cache.s[b, h, side, g, t] = e + 127


def _places(cache, table_row, positions):
    """Blocks and places of positions, and which of them the table has."""
    ids = np.full(len(positions), -1, dtype=np.int64)
    for i, p in enumerate(positions):
        if p >= 0 and p // cache.T < len(table_row):
            ids[i] = table_row[p // cache.T]
    ok = (ids >= 0) & (ids < cache.blocks)
    return np.where(ok, ids, 0), np.maximum(positions, 0) % cache.T, ok


def load(cache, table, lengths, starts, rows):
    """float64 keys and values [rows, H, D], and which rows are of a request."""
    out = np.zeros((2, rows, cache.H, cache.D))
    real = np.zeros(rows, bool)
    for b, length in enumerate(lengths):
        r0, r1 = starts[b], min(starts[b + 1], rows)
        if r0 < 0 or r1 <= r0:
            continue
        pos = length - (starts[b + 1] - r0) + np.arange(r1 - r0)
        ids, places, ok = _places(cache, table[b], pos)
        real[r0:r1] = True
        for side in range(2):
            for h in range(cache.H):
                out[side, r0:r1, h] = np.where(ok[:, None], cache.tokens(side, ids, h, places), 0.0)
    return out[0], out[1], real


def attend(cache, query, table, lengths, starts, scale):
    """float64 (out, lse, bound of |weights| times |values|, bound of scores, sum of the
    |values| seen) for query rows [rows, heads, D]; rows of no request are NaN."""
    rows, heads, D = query.shape
    group = heads // cache.H
    out = np.full((rows, heads, D), np.nan)
    lse = np.full((rows, heads), np.nan)
    mag = np.zeros((rows, heads, D))
    big = np.zeros((rows, heads))
    far = np.zeros((rows, heads, D))
    for b, length in enumerate(lengths):
        r0, r1 = starts[b], min(starts[b + 1], rows)
        t = np.arange(max(0, min(length, len(table[b]) * cache.T)))
        ids, places, ok = _places(cache, table[b], t)
        for h in range(cache.H):
            k, v = (cache.tokens(side, ids, h, places) for side in range(2))
            for n in range(r0, r1):
                see = ok & (t <= length - (starts[b + 1] - starts[b]) + n - starts[b])
                for g in range(h * group, (h + 1) * group):
                    if not see.any():
                        out[n, g], lse[n, g] = 0.0, -np.inf
                        continue
                    q = query[n, g]
                    with np.errstate(invalid="ignore", over="ignore"):
                        x = (k[see] @ q) * scale
                        m = x.max()
                        p = np.exp(x - m)
                        l = p.sum()
                        out[n, g] = (p @ v[see]) / l
                        lse[n, g] = m + math.log(l) if np.isfinite(l) else np.nan
                        mag[n, g] = (p @ np.abs(v[see])) / l
                        big[n, g] = (np.abs(k[see]) @ np.abs(q)).max() * scale
                        far[n, g] = np.abs(v[see]).sum(0)
    return out, lse, mag, big, far
