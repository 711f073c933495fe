"""How far attention may be off where its weights are held as the sum of two
bfloat16 numbers, and inputs that tell such weights from rounded ones."""
import numpy as np

import cache_ref as R

WEIGHT = 2.0 ** -16  # what two bfloat16 numbers leave of a weight


def two_part_bounds(ref, tokens, D, out_eps):
    """Bounds of out and lse, elementwise, from R.attend()'s result.

    As R.attend_bounds, but for the weights: bfloat16 holds 8 significant bits,
    so the first number is off by 2^-8 of the weight at most; what is left is
    exact in float (a difference of close numbers), and the second number is off
    by 2^-8 of it: 2^-16 of the weight.

    An output below the type's normal numbers is rounded to a step that does not
    shrink with it: float16's numbers below 2^-14 are 2^-24 apart, so half a
    step is 2^-25 there, which 2^-11 of the output is less than (of -1.2148e-6,
    nearest float16 number -1.1921e-6: off by 2.27e-8, 2^-11 of it 5.9e-10).
    bfloat16's are 2^-133 apart, far below the 1e-30 allowed in any case."""
    out, lse, mag, big = ref
    u = 2.0 ** -24
    eta = 1.01 * ((D + 9) * u * big + 4 * u)
    n = 2 * tokens + 64
    tol_out = out_eps * np.abs(out) + (WEIGHT * 1.01 + 2 * eta[..., None] + 2 * n * u) * mag
    tol_lse = eta + n * u + 4 * u * (1 + np.abs(np.where(np.isfinite(lse), lse, 0.0)))
    return tol_out * 1.01 + (2.0 ** -25 if out_eps == 2.0 ** -11 else 1e-30), tol_lse


def cancelling_pairs(cache):
    """Tokens 2i and 2i + 1 get nearly the same keys and opposite values: outputs
    are small beside the weights times the values, so the output's own rounding
    does not hide that of the weights."""
    k, v = cache.k, cache.v
    k[:, :, 1::2] = k[:, :, 0::2]
    k[:, :, :, :4] &= 0xFE
    k[:, :, 1::2, :4] ^= 2
    v[:, :, 1::2] = v[:, :, 0::2] ^ 128
    assert not ((k & 127) == 127).any() and not ((v & 127) == 127).any()


def to_bfloat16(x):
    """Nearest numbers of 8 significant bits, ties to the even one (float64)."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(m * 256), e - 8)


def rounded_attend(cache, query, table, lengths, scale, parts):
    """Attention of one query row per request in 64 bits, but for its weights, which
    are held as `parts` bfloat16 numbers; their sum is that of the weights."""
    out = np.zeros(query.shape)
    group = query.shape[1] // cache.H
    for b, n in enumerate(lengths):
        t = np.arange(n)
        ids = np.asarray(table[b])[t // cache.T]
        for g in range(query.shape[1]):
            h = g // group
            k = R.VALUES[cache.k[ids, h, t % cache.T]] * cache.s[ids, h, 0].astype(float)[:, None]
            v = R.VALUES[cache.v[ids, h, t % cache.T]] * cache.s[ids, h, 1].astype(float)[:, None]
            x = (k @ query[b, g]) * scale
            p = np.exp(x - x.max())
            held, rest = np.zeros_like(p), p
            for _ in range(parts):
                held = held + to_bfloat16(rest)
                rest = p - held
            out[b, g] = (held @ v) / p.sum()
    return out
