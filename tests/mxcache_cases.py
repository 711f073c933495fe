"""What the GPU tests of the 4-bit cache share: pools, and one call of each operator
checked against its plain form."""
import math

import numpy as np
import torch

import mxcache_ref as R
from attend_bounds import two_part_bounds

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def xf():
    import recv_fifo_plane_amd
    return recv_fifo_plane_amd


def dev(a):
    return torch.as_tensor(np.ascontiguousarray(a)).to("cuda")


def ints(a):
    return torch.tensor(np.asarray(a, dtype=np.int32).tolist(), dtype=torch.int32, device="cuda")


def table_of(rows, pad=2, fill=2 ** 31 - 1):
    """A table [batch, width] whose rows lie `pad` entries apart."""
    rows = np.asarray(rows, dtype=np.int64)
    wide = np.full((rows.shape[0], rows.shape[1] + pad), fill)
    wide[:, :rows.shape[1]] = rows
    return ints(wide.reshape(-1)).reshape(wide.shape)[:, :rows.shape[1]]


def starts_of(rows, before=0):
    s = [before]
    for r in rows:
        s.append(s[-1] + r)
    return s


def new_pool(n, T, H, D, seed, low=-4, high=1):
    """Any codes, scales of 2^low to 2^high."""
    rng = np.random.default_rng(seed)
    c = R.Cache(rng.integers(0, 256, (n, R.block_bytes(T, H, D)), dtype=np.uint8), T, H, D)
    c.s[:] = rng.integers(127 + low, 128 + high, c.s.shape)
    return c


def gpu_cache(c):
    return xf().PagedCache(c.blocks, c.T, c.H, c.D, buffer=dev(c.raw()), bits=4)


def as_type(x, dtype):
    return torch.tensor(x, dtype=torch.float64).to(DT[dtype]).cuda()


def blocks_of(lens, T, blocks, width, rng, bad_pages=0):
    """A table whose requests hold their tokens in blocks taken in a mixed order."""
    used = [-(-max(x, 0) // T) for x in lens]
    order = rng.permutation(blocks)
    table, at = np.full((len(lens), width), -1), 0
    for b, n in enumerate(used):
        n = min(n, width)
        table[b, :n] = order[at:at + n]
        at += n
    for _ in range(bad_pages):
        b = int(rng.integers(0, len(lens)))
        if used[b]:
            table[b, int(rng.integers(0, min(used[b], width)))] = rng.choice(
                [-1, blocks, 2 ** 31 - 1, -2 ** 31])
    return table, used


def check_store(T, H, D, dtype, slots, seed, blocks=30, edit=None, strides=False):
    """Every byte of the pool is that of the plain form."""
    ref = new_pool(blocks, T, H, D, seed)
    gpu = gpu_cache(ref)
    rng = np.random.default_rng(seed + 1)
    n = len(slots)
    rows = [as_type(rng.normal(0, 1, (n, H, D)) * 2.0 ** rng.integers(-6, 9, (n, H, 1)), dtype)
            for _ in range(2)]
    if edit is not None:
        edit(*rows)
    key, value = rows
    if strides:  # one fused row per token for the keys, heads before rows for the values
        fused = torch.zeros(n, 2 * H + 1, D + 3, dtype=key.dtype, device="cuda")
        fused[:, 1:H + 1, 3:] = key
        key = fused[:, 1:H + 1, 3:]
        value = value.transpose(0, 1).contiguous().transpose(0, 1)
    gpu.store(key, value, ints(slots))
    torch.cuda.synchronize()
    R.store(ref, key.double().cpu().numpy(), value.double().cpu().numpy(), slots)
    got = R.Cache(gpu.buffer.cpu().numpy(), T, H, D)
    for name in ("s", "k", "v", "pad"):
        g, w = getattr(got, name), getattr(ref, name)
        assert np.array_equal(g, w), (name, np.argwhere(g != w)[:5])
    return ref, gpu


def check_load(cache, lens, rows, dtype, seed=0, before=0, behind=0, strides=False, width=None,
               bad_pages=0, cut=0, new=False):
    """cache: (plain, on the GPU).  Every number is the plain form's, rounded."""
    ref, gpu = cache
    T, H, D = ref.T, ref.H, ref.D
    rng = np.random.default_rng(seed)
    width = max([-(-max(x, 0) // T) for x in lens] + [0]) + 1 if width is None else width
    table, _ = blocks_of(lens, T, ref.blocks, width, rng, bad_pages)
    starts = starts_of(rows, before)
    n = max(0, starts[-1] + behind - cut)
    outs = [torch.full((n, H, D), 7.0, dtype=DT[dtype], device="cuda") for _ in range(2)]
    if strides:
        outs = [torch.full((n, H + 2, D + 5), 7.0, dtype=DT[dtype], device="cuda")[:, 1:-1, 2:-3],
                torch.full((H, n, D + 1), 7.0, dtype=DT[dtype], device="cuda").transpose(0, 1)[:, :, 1:]]
    args = (table_of(table), ints(lens), ints(starts), n)
    if new:
        got = gpu.load(*args, dtype=DT[dtype])
        assert all(x.dtype == DT[dtype] and x.shape == (n, H, D) for x in got)
    else:
        got = gpu.load(*args, out=outs)
        assert got[0] is outs[0] and got[1] is outs[1]
    torch.cuda.synchronize()
    want = R.load(ref, table.tolist(), lens, starts, n)
    for g, w in zip(got, want[:2]):
        w = torch.tensor(w).to(DT[dtype])
        g = g.cpu()
        real = torch.tensor(want[2])
        assert torch.equal(torch.isnan(g[real]), torch.isnan(w[real]))
        assert torch.equal(torch.nan_to_num(g[real], 3.0, 1e30, -1e30),
                           torch.nan_to_num(w[real], 3.0, 1e30, -1e30))
        if not new:
            assert torch.all(g[~real] == 7.0)


def is_shared(batch, rows, T, H, group, D, dtype, width, max_query=0, max_length=0):
    """Whether a call shares its tokens out over workgroups (it then has a workspace)."""
    import ctypes as C
    from recv_fifo_plane_amd import xfer as X
    p = 1 << 40
    a = X.xfer_attend(p, p, None, p, p, p, None, 0, H * group * D, D, H * group * D, D, width, batch, rows,
                      H * group, width, 0 if dtype == "bf16" else 1, 1.0, max_query, max_length)
    n = C.c_size_t()
    assert X.lib().xfer_mxcache_attend_workspace(C.byref(X.xfer_cache_shape(T, H, D, 10)), C.byref(a),
                                                 C.byref(n)) == 0
    return n.value > 0


def bounds(want, tokens, D, dtype, wide):
    """How far out and lse may be from R.attend()'s, elementwise.

    Those of two_part_bounds; a bfloat16 query's products are those of D dims, a float16
    query may go in two bfloat16 numbers, exactly, which makes 2 D products of a
    score's sum.  wide: a call of many rows, whose weights may multiply the values as
    float16 numbers.  Theirs are 11 significant bits: one of them is off by 2^-11 of the
    weight at most, the sum of two (float16 queries) by 2^-22, which two_part_bounds
    covers.  Below 2^-14 float16's numbers are 2^-24 apart, so what is left of
    a weight is at least off by 2^-25 there; weights are taken relative to a reference
    that leaves the largest of a row's at 2^7 or more, so that is 2^-32 of the row's
    sum of weights, for each of the values that it sees."""
    out_eps = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
    tol, tol_lse = two_part_bounds(want[:4], tokens, D if dtype == "bf16" else 2 * D, out_eps)
    if wide:
        tol = tol + 1.01 * 2.0 ** -32 * want[4] * 1.01
        if dtype == "bf16":
            tol = tol + 1.01 * 2.0 ** -11 * want[2] * 1.01
    return tol, tol_lse


def many_length(n, H, group, D):
    """A length from which tiles of many rows compute n rows."""
    return 64 * ((57344 if D <= 128 else 24576) // (n * group // 16 * H) + 1)


def check_attend(lens, rows, T, H, group, D, dtype="bf16", seed=0, width=None, bad_pages=0,
                 nan_tail=True, before=0, behind=0, hints=True, strides=False, scale=None, mag=1.0,
                 edit=None, shared=None, many=None):
    """out and lse against the plain form's.  many: the length that the call is told (0: a wide
    table and no hint), so that tiles of many rows compute it."""
    rng = np.random.default_rng(seed)
    width = max([-(-max(x, 0) // T) for x in lens] + [0]) + 1 if width is None else width
    blocks = sum(-(-max(x, 0) // T) for x in lens) + 3
    ref = new_pool(blocks, T, H, D, seed)
    table, used = blocks_of(lens, T, blocks, width, rng)
    for b, n in enumerate(used):
        if nan_tail and lens[b] > 0 and lens[b] % T and n <= width:
            ref.s[table[b, n - 1], :, :, :, lens[b] % T:] = 255  # what stands behind the last token
    for _ in range(bad_pages):
        b = int(rng.integers(0, len(lens)))
        if used[b]:
            table[b, int(rng.integers(0, min(used[b], width)))] = rng.choice(
                [-1, blocks, 2 ** 31 - 1, -2 ** 31])
    heads = H * group
    starts = starts_of(rows, before)
    n = starts[-1] + behind
    q = torch.randn(n, heads, D, generator=torch.Generator().manual_seed(seed)) * mag
    q = q.to(DT[dtype])
    if edit is not None:
        edit(q, ref, table)
    gpu = gpu_cache(ref)
    qd = q.cuda()
    out = torch.full((n, heads, D), 7.0, dtype=q.dtype, device="cuda")
    if strides:
        wide = torch.zeros(n, heads + 2, D + 8, dtype=q.dtype, device="cuda")
        wide[:, 1:-1, :D] = qd
        qd = wide[:, 1:-1, :D]
        out = torch.full((heads, n, D + 8), 7.0, dtype=q.dtype, device="cuda").transpose(0, 1)[:, :, 8:]
    lse = torch.full((n, heads), 7.0, device="cuda")
    more = dict(max_query=max(rows + [0]), max_length=max(lens + [0, 0])) if hints else {}
    if many is not None:
        told = many or many_length(n, H, group, D)
        width = max(width, -(-told // T))
        table = np.pad(table, ((0, 0), (0, width - table.shape[1])), constant_values=-1)
        if hints:
            more["max_length"] = told
    if shared is not None:
        assert is_shared(len(lens), n, T, H, group, D, dtype, width, *more.values()) == shared
    gpu.attend(qd, table_of(table), ints(lens), ints(starts), scale=scale, out=out, lse=lse, **more)
    torch.cuda.synchronize()
    sc = 1 / math.sqrt(D) if scale is None else scale
    want = R.attend(ref, q.double().numpy(), table.tolist(), lens, starts, sc)
    tol, tol_lse = bounds(want, max(lens + [1]), D, dtype, many is not None)
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    real = np.zeros(n, bool)
    real[starts[0]:starts[-1]] = True
    assert np.all(got[~real] == 7.0) and np.all(got_lse[~real] == 7.0)
    for g, w, e, what in ((got, want[0], tol, "out"), (got_lse, want[1], tol_lse, "lse")):
        g, w, e = g[real], w[real], e[real]
        if what == "out" and dtype == "fp16":
            # float16 ends at 65504: what is 65520 (its last half step) or more rounds to infinity
            with np.errstate(invalid="ignore"):
                over, near = np.abs(w) - e >= 65520, np.abs(w) + e >= 65520
            w = np.where(over | (near & np.isinf(g)), np.copysign(np.inf, w), w)
        assert np.array_equal(np.isnan(g), np.isnan(w)), what
        fin = np.isfinite(w)
        assert np.array_equal(g[~fin & ~np.isnan(w)], w[~fin & ~np.isnan(w)]), what
        off = np.abs(g[fin] - w[fin]) / e[fin]
        assert off.size == 0 or off.max() <= 1.0, (what, off.max(), np.argwhere(off > 1)[:4])
    return got, got_lse
