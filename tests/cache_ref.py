"""Plain forms of the paged cache's operators for the tests: loops over
requests and blocks, in 64 bits, on the CPU."""
from __future__ import annotations

import math

import numpy as np


def block_bytes(T, H, D):
    return 2 * H * T * D + (8 * H + 127) // 128 * 128


# ---------------------------------------------------------------------- e4m3
def e4m3_values():
    """The value of each of the 256 codes: 1 sign, 4 exponent (bias 7), 3 mantissa bits."""
    v = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = (m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = math.nan if (c & 127) == 127 else (-x if c & 128 else x)
    return v


VALUES = e4m3_values()


def to_codes(x):
    """Nearest codes of float64 numbers (ties to the even one; at most 448); others NaN."""
    x = np.asarray(x, dtype=np.float64)
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    assert a.max(initial=0.0) <= 448.0
    _, e = np.frexp(np.maximum(a, 2.0 ** -40))
    e = np.maximum(e - 1, -6)
    q = np.rint(a / 2.0 ** (e - 3))            # 8 .. 16 for normal numbers, 0 .. 8 below
    up = q == 16
    e = np.where(up, e + 1, e)
    q = np.where(up, 8, q)
    code = np.where(q >= 8, ((e + 7) * 8 + (q - 8)), q).astype(np.int64)
    code = code | np.where(np.signbit(x), 128, 0)
    return np.where(np.isfinite(x), code, 127).astype(np.uint8)


def scale_of(amax):
    """The smallest power of two, 2^-118 at least, that brings amax to 448 or below."""
    e = -118
    while amax > 448 * 2.0 ** e:
        e += 1
    return 2.0 ** e


class Cache:
    """A pool as arrays: codes of keys and values [blocks, H, T, D], scales [blocks, H, 2]."""

    def __init__(self, raw, T, H, D):
        n = raw.shape[0]
        assert raw.shape[1] == block_bytes(T, H, D)
        body = raw[:, :2 * H * T * D].reshape(n, H, 2, T * D)
        self.T, self.H, self.D, self.blocks = T, H, D, n
        self.k = body[:, :, 0].reshape(n, H, T, D).copy()
        self.v = body[:, :, 1].reshape(n, H, D, T).transpose(0, 1, 3, 2).copy()
        self.s = raw[:, 2 * H * T * D:2 * H * T * D + 8 * H].copy().view(np.float32).reshape(n, H, 2)
        self.pad = raw[:, 2 * H * T * D + 8 * H:].copy()

    def raw(self):
        n, H, T, D = self.blocks, self.H, self.T, self.D
        body = np.concatenate([self.k.reshape(n, H, 1, T * D),
                               self.v.transpose(0, 1, 3, 2).reshape(n, H, 1, T * D)], 2)
        s = np.ascontiguousarray(self.s).reshape(n, -1).view(np.uint8)
        return np.concatenate([body.reshape(n, -1), s, self.pad], 1)


# ----------------------------------------------------------------------- plan
def plan(cached, added, table, free, T, rows):
    """(slots, positions, starts, lengths, counts, table) as lists."""
    table = [list(r) for r in table]
    slots, positions, starts, taken, lost = [], [], [0], 0, 0
    lengths = []
    for i, (c, a) in enumerate(zip(cached, added)):
        c, a = max(c, 0), max(a, 0)
        held = -(-c // T)
        reach = min(len(table[i]), held + max(0, len(free) - taken))
        for p in range(held, -(-(c + a) // T)):
            if p < len(table[i]) and taken < len(free):
                table[i][p] = free[taken]
            taken += 1
        for p in range(c, c + a):
            block = table[i][p // T] if p // T < reach else -1
            slots.append(block * T + p % T if block >= 0 else -1)
            positions.append(p)
        lost += max(0, c + a - max(c, reach * T))
        starts.append(starts[-1] + a)
        lengths.append(c + a)
    pad = [-1] * max(0, rows - len(slots))
    return ((slots + pad)[:rows], (positions + pad)[:rows], starts, lengths, [taken, lost], table)


# ---------------------------------------------------------------------- store
def store(cache, key, value, slots):
    """Stores float64 rows [rows, H, D] into `cache`, run by run."""
    T, n = cache.T, 0
    while n < len(slots):
        slot = slots[n]
        if slot < 0 or slot // T >= cache.blocks:
            n += 1
            continue
        cnt = 1
        while n + cnt < len(slots) and slots[n + cnt] == slot + cnt and (slot + cnt) % T:
            cnt += 1
        b, off = slot // T, slot % T
        for h in range(cache.H):
            for side, (codes, x) in enumerate(((cache.k, key), (cache.v, value))):
                new = x[n:n + cnt, h]
                s = scale_of(np.where(np.isfinite(new), np.abs(new), 0.0).max())
                if off:
                    was = float(cache.s[b, h, side])
                    s = max(s, was)
                    if s > was:
                        codes[b, h, :off] = to_codes(VALUES[codes[b, h, :off]] * (was / s))
                codes[b, h, off:off + cnt] = to_codes(new / s)
                cache.s[b, h, side] = s
        n += cnt


# --------------------------------------------------------------------- attend
def attend(cache, query, table, lengths, starts, scale):
    """float64 (out, lse, bound of |weights| times |values|, bound of scores) for
    query rows [rows, heads, D]; rows of no request are NaN."""
    rows, heads, D = query.shape
    T, group = cache.T, heads // cache.H
    out = np.full((rows, heads, D), np.nan)
    lse = np.full((rows, heads), np.nan)
    mag = np.zeros((rows, heads, D))
    big = np.zeros((rows, heads))
    for b, length in enumerate(lengths):
        r0, r1 = max(starts[b], 0), min(starts[b + 1], rows)
        length_seen = max(0, min(length, len(table[b]) * T))
        t = np.arange(length_seen)
        ids = np.array([table[b][p] for p in t // T], dtype=np.int64)
        ok = (ids >= 0) & (ids < cache.blocks)
        ids = np.where(ok, ids, 0)
        for h in range(cache.H):
            k = VALUES[cache.k[ids, h, t % T]] * cache.s[ids, h, 0].astype(np.float64)[:, None]
            v = VALUES[cache.v[ids, h, t % T]] * cache.s[ids, h, 1].astype(np.float64)[:, None]
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
                        lse[n, g] = m + np.log(l)
                        mag[n, g] = (p @ np.abs(v[see])) / l
                        big[n, g] = (np.abs(k[see]) @ np.abs(q)).max() * scale
    return out, lse, mag, big


def attend_bounds(ref, tokens, D, out_eps):
    """How far out and lse may be from attend()'s, elementwise.

    u = 2^-24 rounds a float.  A score is a sum of D products that are exact in
    float, in any order, and three multiplications: off by at most (D + 3) u
    times the sum of the products' magnitudes, `big`.  Its exponential is taken
    in base 2 from a difference of magnitude at most 2 log2(e) big, rounded
    twice, by a function good to 2 steps: p is off by at most
    eta = 1.01 ((D + 3) u big + 6 u big + 4 u) relative to its value, and the
    maximum cancels.  A weight is rounded to bfloat16 (2^-8), each of `tokens`
    additions and rescalings by u; sums of magnitudes bound the rest."""
    out, lse, mag, big = ref
    u = 2.0 ** -24
    eta = 1.01 * ((D + 9) * u * big + 4 * u)
    n = 2 * tokens + 64
    tol_out = out_eps * np.abs(out) + (2.0 ** -8 * 1.01 + 2 * eta[..., None] + 2 * n * u) * mag
    tol_lse = eta + n * u + 4 * u * (1 + np.abs(np.where(np.isfinite(lse), lse, 0.0)))
    return tol_out * 1.01 + 1e-30, tol_lse
