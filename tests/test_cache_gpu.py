"""GPU tests of the paged cache: plans, stores, block transfers and attention
against plain forms in 64 bits, at the sizes and masks where they can go wrong."""
import math

import numpy as np
import pytest

import cache_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def xf():
    import recv_fifo_plane_amd
    return recv_fifo_plane_amd


def dev(a, dtype=None):
    return torch.as_tensor(np.ascontiguousarray(a), device="cuda" if dtype is None else None,
                           dtype=dtype).to("cuda")


def ints(a):
    return torch.tensor(np.asarray(a, dtype=np.int32).tolist(), dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------ plan
def check_plan(cached, added, width, nfree, T, rows, seed=0, pad_columns=0, out=None):
    rng = np.random.default_rng(seed)
    B = len(cached)
    ids = rng.permutation(5 * (B + 1) * (width + 1) + nfree).astype(np.int64)
    free = ids[:nfree].tolist()
    table = rng.permutation(B * width).reshape(B, width) + 100000
    for i, c in enumerate(cached):  # behind the held blocks: anything
        table[i, -(-max(c, 0) // T):] = -7
    full = np.full((B, width + pad_columns), -9)
    full[:, :width] = table
    t = ints(full.reshape(-1)).reshape(B, width + pad_columns)
    plan = xf().plan_blocks(ints(cached), ints(added), t[:, :width], ints(free), T, rows, out=out)
    torch.cuda.synchronize()
    slots, positions, starts, lengths, counts, want = R.plan(cached, added, table.tolist(), free, T,
                                                             rows)
    assert plan.starts.tolist() == starts
    assert plan.lengths.tolist() == lengths
    assert plan.counts.tolist() == counts
    assert plan.positions.tolist() == positions
    assert plan.slots.tolist() == slots
    got = t.cpu().numpy()
    assert np.array_equal(got[:, :width], np.array(want, dtype=np.int64).reshape(B, width))
    assert np.all(got[:, width:] == -9)
    return plan


@pytest.mark.parametrize("B", [0, 1, 2, 63, 64, 65, 255, 1023, 1024, 1025, 2049, 3001])
def test_plan_batches(B):
    rng = np.random.default_rng(B)
    cached = rng.integers(0, 70, B).tolist()
    added = (rng.integers(0, 40, B) * (rng.random(B) > 0.2)).tolist()
    check_plan(cached, added, 8, 20 * (B + 1), 16, sum(added) + 3, seed=B)


@pytest.mark.parametrize("T", [16, 32, 64])
@pytest.mark.parametrize("cached,added", [
    ([0], [0]), ([0], [1]), ([15], [1]), ([16], [1]), ([17], [0]), ([64], [64]), ([63], [2]),
    ([0, 0, 0], [0, 5, 0]), ([5, 0, 9], [0, 0, 0]), ([-3, 4], [7, -2]), ([1000], [3001]),
    ([0] * 5, [1] * 5), ([31, 32, 33], [1, 1, 1])])
def test_plan_edges(T, cached, added):
    check_plan(cached, added, 260, 300, T, max(0, sum(added)) + 2, seed=T, pad_columns=3)


@pytest.mark.parametrize("nfree", [0, 1, 7, 20])
def test_plan_without_room(nfree):
    """A free list that ends, and a table that is too narrow: tokens without a slot are counted."""
    cached, added = [10, 0, 40, 0, 16], [30, 100, 0, 17, 16]
    p = check_plan(cached, added, 4, nfree, 16, 180)
    assert p.counts.tolist()[1] > 0
    check_plan(cached, added, 0, 3, 16, 180)


@pytest.mark.parametrize("rows", [0, 1, 50, 4095])
def test_plan_rows_cut(rows):
    check_plan([3, 50, 0, 7], [1000, 60, 1500, 4000], 300, 600, 32, rows)


def test_plan_long_prompts():
    check_plan([0, 100001, 5], [120000, 1, 70001], 8000, 20000, 16, 200000)


# ----------------------------------------------------------------------- store
def new_pool(n, T, H, D, seed, full=True):
    rng = np.random.default_rng(seed)
    raw = rng.integers(0, 256, (n, R.block_bytes(T, H, D)), dtype=np.uint8)
    c = R.Cache(raw, T, H, D)
    if full:
        c.k, c.v = (R.to_codes(rng.normal(0, 90, x.shape).clip(-448, 448)) for x in (c.k, c.v))
    c.s[:] = 2.0 ** rng.integers(-9, -3, c.s.shape)
    return c


def gpu_cache(c):
    return xf().PagedCache(c.blocks, c.T, c.H, c.D, buffer=dev(c.raw()))


def check_pool(gpu, ref, what=""):
    got = R.Cache(gpu.buffer.cpu().numpy(), ref.T, ref.H, ref.D)
    assert np.array_equal(got.s, ref.s), what
    for g, w, n in ((got.k, ref.k, "key"), (got.v, ref.v, "value")):
        gn, wn = (g & 127) == 127, (w & 127) == 127
        assert np.array_equal(gn, wn), (what, n)
        assert np.array_equal(g[~gn], w[~wn]), (what, n, np.argwhere((g != w) & ~gn)[:5])
    assert np.array_equal(got.pad, ref.pad), what


DT = {"bf16": "bfloat16", "fp16": "float16", "fp32": "float32"}


def as_type(x, dtype):
    return torch.tensor(x, dtype=torch.float64).to(getattr(torch, DT[dtype])).cuda()


def runs_of(rng, blocks, T, runs, one=False):
    """Slots of `runs` runs in blocks of their own."""
    slots = []
    for b in rng.permutation(blocks)[:runs]:
        off = int(rng.integers(0, T))
        if rng.random() < 0.3:
            off = 0
        cnt = 1 if one else int(rng.integers(1, T - off + 1))
        slots += [int(b) * T + off + i for i in range(cnt)]
    return slots


def check_store(T, H, D, dtype, slots, seed, blocks=None, mag=None, edit=None, strides=False):
    blocks = blocks or 40
    ref = new_pool(blocks, T, H, D, seed)
    gpu = gpu_cache(ref)
    rng = np.random.default_rng(seed + 1)
    n = len(slots)
    key, value = (rng.normal(0, 1, (n, H, D)) * 2.0 ** rng.integers(-6, 9, (n, 1, 1))
                  for _ in range(2))
    if mag is not None:
        key, value = key * mag, value * mag
    if edit is not None:
        edit(key, value)
    if strides:  # rows of a wider fused tensor, heads apart
        wide = torch.zeros(n + 1, 2 * H + 3, D + 8, dtype=getattr(torch, DT[dtype]), device="cuda")
        kt, vt = wide[1:, 1:H + 1, 8:], wide[:n, H + 2:2 * H + 2, :D]
        kt.copy_(as_type(key, dtype))
        k_in = kt.clone()
        vt.copy_(as_type(value, dtype))  # the two views do not overlap
        assert torch.equal(k_in.nan_to_num(7), kt.nan_to_num(7))
    else:
        kt, vt = as_type(key, dtype), as_type(value, dtype)
    gpu.store(kt, vt, ints(slots))
    torch.cuda.synchronize()
    R.store(ref, kt.double().cpu().numpy(), vt.double().cpu().numpy(), slots)
    check_pool(gpu, ref, (T, H, D, dtype))
    return gpu, ref


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T", [16, 32, 64])
@pytest.mark.parametrize("H,D", [(1, 64), (2, 96), (3, 128), (8, 128), (1, 192), (2, 256), (17, 64)])
def test_store_runs(T, H, D, dtype):
    rng = np.random.default_rng(T * D + H)
    check_store(T, H, D, dtype, runs_of(rng, 40, T, 9), seed=T + D)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T", [16, 32, 64])
def test_store_single_tokens(T, dtype):
    rng = np.random.default_rng(T)
    check_store(T, 4, 128, dtype, runs_of(rng, 60, T, 50, one=True), seed=T, blocks=60)


@pytest.mark.parametrize("T,D", [(16, 128), (64, 256), (32, 96)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_store_whole_prompt(T, D, dtype):
    """Full blocks in a row, whose ids are consecutive: runs end at a block's end."""
    slots = list(range(3 * T + 5, 11 * T - 2))
    check_store(T, 2, D, dtype, slots, seed=T)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_store_strides_and_padding(dtype):
    T = 16
    rng = np.random.default_rng(4)
    slots = runs_of(rng, 30, T, 6)
    slots = [-1, -1] + slots[:5] + [-1] + runs_of(rng, 0, T, 0) + [40 * T, 40 * T + 3, 2 ** 31 - 1, -5]
    check_store(T, 3, 128, dtype, slots, seed=5, strides=True)


def test_store_odd_strides():
    """Rows whose addresses are aligned to their elements only."""
    T, H, D, n = 32, 2, 96, 45
    ref = new_pool(6, T, H, D, 3)
    gpu = gpu_cache(ref)
    flat = torch.randn(n * (2 * H * D + 7) + 20, device="cuda").to(torch.float16)
    kt = flat[1:].as_strided((n, H, D), (2 * H * D + 7, D + 1, 1))
    vt = flat[3 + H * D:].as_strided((n, H, D), (2 * H * D + 7, D - 3, 1))
    slots = list(range(T + 7, T + 7 + n))
    gpu.store(kt, vt, ints(slots))
    R.store(ref, kt.double().cpu().numpy(), vt.double().cpu().numpy(), slots)
    check_pool(gpu, ref)


def test_store_every_rounding():
    """Every bfloat16 and float16 number, in frames whose scale is 1 and others."""
    for dtype, np_bits in (("bf16", torch.bfloat16), ("fp16", torch.float16)):
        x = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(np_bits).double().numpy()
        for e in (0, -4, 7):
            y = x[np.isfinite(x) & (np.abs(x) <= 448.0 * 2.0 ** e)]
            y = np.concatenate([y, np.zeros(-len(y) % (64 * 15))]).reshape(-1, 15, 64)
            pin = np.full((len(y), 1, 64), 448.0 * 2.0 ** e)  # settles the scale
            rows = np.concatenate([pin, y], 1).reshape(-1, 1, 64)
            check_store(16, 1, 64, dtype, list(range(len(rows))), seed=1, blocks=len(rows) // 16 + 1,
                        edit=lambda k, v: (np.copyto(k, rows), np.copyto(v, -rows)))


@pytest.mark.parametrize("amax", [0.0, 2.0 ** -140, 2.0 ** -111, 447.9, 448.0, 448.1, 511.0, 512.0,
                                  3.3e38, 2.0 ** 127])
def test_store_scale_borders(amax):
    def edit(k, v):
        k[:] = 0
        v[:] = 0
        k[::3, :, 5] = amax
        v[::2, :, 1] = -amax
        v[:, :, 2] = amax / 3
    check_store(16, 2, 64, "fp32", list(range(16, 48)) + [100, 101], seed=2, edit=edit)


def test_store_not_finite():
    def edit(k, v):
        k[0, 0, 0], k[3, 1, 7], k[5, 0, 9] = np.nan, np.inf, -np.inf
        v[1, 1, 3], v[2, 0, 2] = np.inf, np.nan
        k[8:12] = np.nan  # a whole run of them
        v[8:12] = -np.inf
    check_store(16, 2, 128, "bf16", list(range(35, 43)) + list(range(64, 68)) + [5], seed=3, edit=edit)


def test_store_grows_and_keeps_scales():
    """Token by token into the same blocks: the earlier codes follow the scale."""
    T, H, D = 16, 2, 128
    ref = new_pool(4, T, H, D, 9)
    gpu = gpu_cache(ref)
    rng = np.random.default_rng(9)
    for i in range(T):
        key, value = (rng.normal(0, 1, (2, H, D)) * 2.0 ** rng.integers(-12, 12, (2, 1, 1)) for _ in "kv")
        kt, vt = as_type(key, "bf16"), as_type(value, "bf16")
        slots = [T + i, 3 * T + i]
        gpu.store(kt, vt, ints(slots))
        R.store(ref, kt.double().cpu().numpy(), vt.double().cpu().numpy(), slots)
        check_pool(gpu, ref, i)


def test_store_nothing():
    ref = new_pool(4, 16, 2, 64, 1)
    gpu = gpu_cache(ref)
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    gpu.store(e, e, ints([]))
    check_pool(gpu, ref)


# ---------------------------------------------------------------------- attend
def packed(rows, before=0):
    s = [before]
    for r in rows:
        s.append(s[-1] + r)
    return s


def check_attend(lens, rows, T, H, group, D, dtype="bf16", seed=0, width=None, bad_pages=0, nan_tail=True,
                 before=0, behind=0, hints=True, strides=False, scale=None, mag=1.0, blocks=None,
                 edit=None):
    rng = np.random.default_rng(seed)
    used = [-(-max(x, 0) // T) for x in lens]
    width = max(used + [0]) + 1 if width is None else width
    blocks = blocks or sum(used) + 3
    ref = new_pool(blocks, T, H, D, seed)
    order = rng.permutation(blocks)
    table = np.full((len(lens), width), -1)
    at = 0
    for b, n in enumerate(used):
        n = min(n, width)
        table[b, :n] = order[at:at + n]
        at += n
        if nan_tail and lens[b] > 0 and lens[b] % T and n == used[b]:
            last = table[b, n - 1]
            ref.k[last, :, lens[b] % T:] = 127  # what stands behind the last token is not a number
            ref.v[last, :, lens[b] % T:] = 255
    for _ in range(bad_pages):
        b = int(rng.integers(0, len(lens)))
        if used[b]:
            table[b, int(rng.integers(0, min(used[b], width)))] = rng.choice([-1, blocks, 2 ** 31 - 1, -2 ** 31])
    heads = H * group
    starts = packed(rows, before)
    n = starts[-1] + behind
    q = torch.randn(n, heads, D, generator=torch.Generator().manual_seed(seed)) * mag
    q = q.to(getattr(torch, DT[dtype]))
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
    wide_table = np.full((len(lens), width + 2), 2 ** 31 - 1)
    wide_table[:, :width] = table
    t = ints(wide_table.reshape(-1)).reshape(len(lens), width + 2)[:, :width]
    more = dict(max_query=max(rows + [0]), max_length=max(lens + [0])) if hints else {}
    gpu.attend(qd, t, ints(lens), ints(starts), scale=scale, out=out, lse=lse, **more)
    torch.cuda.synchronize()
    sc = 1 / math.sqrt(D) if scale is None else scale
    want = R.attend(ref, q.double().numpy(), table, lens, starts, sc)
    tol, tol_lse = R.attend_bounds(want, max(lens + [1]), D, 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11)
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


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("T", [16, 32, 64])
def test_attend_shapes(T, D, dtype):
    check_attend([1, T - 1, T, T + 1, 150, 333], [1] * 6, T, 2, 4, D, dtype, seed=T + D)


@pytest.mark.parametrize("H,group", [(1, 1), (3, 1), (1, 2), (2, 3), (1, 5), (5, 7), (2, 8), (1, 15),
                                     (1, 16), (2, 17), (1, 40), (8, 1)])
def test_attend_groups(H, group):
    check_attend([77, 1, 260], [1, 1, 1], 16, H, group, 128, seed=group)
    check_attend([77, 3, 130], [3, 2, 1], 32, H, group, 64, "fp16", seed=group)


@pytest.mark.parametrize("rows", [[2, 1, 5], [7, 64, 33], [0, 3, 0, 0, 1], [130, 1, 16, 17]])
@pytest.mark.parametrize("T", [16, 64])
def test_attend_many_rows(rows, T):
    rng = np.random.default_rng(len(rows) * T)
    lens = [r + int(rng.integers(0, 200)) for r in rows]
    check_attend(lens, rows, T, 2, 3, 128, seed=T)
    check_attend(lens, rows, T, 1, 4, 64, "fp16", seed=T + 1, hints=False)
    check_attend(lens, rows, T, 1, 2, 256, seed=T + 2)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T", [16, 64])
def test_attend_wide_heads_of_many_tiles(T, dtype):
    """Heads of 256 in more than 1024 tiles of 16 rows, 32 of them to a workgroup."""
    rng = np.random.default_rng(T)
    rows = [int(x) for x in rng.integers(0, 17, 63)] + [17]
    lens = [int(x) for x in rng.integers(-3, 200, 63)] + [1700]
    lens[:4], rows[:4] = [0, 5, -5, 64], [3, 9, 1, 16]
    check_attend(lens, rows, T, 4, 4, 256, dtype, seed=T)
    check_attend(lens, rows, T, 4, 4, 256, dtype, seed=T + 1, bad_pages=5)


def test_attend_rows_that_see_nothing():
    """No tokens, fewer tokens than rows, a negative length: 0 and -infinity."""
    got, lse = check_attend([0, 3, 0, 20, -5, 1], [2, 9, 0, 1, 1, 40], 16, 2, 2, 128, seed=3)
    assert np.all(got[:2] == 0) and np.all(np.isneginf(lse[:2]))
    assert np.all(np.isneginf(lse[2:8])) and np.all(np.isfinite(lse[8:11]))


def test_attend_rows_of_no_request():
    check_attend([50, 9], [2, 1], 16, 2, 4, 128, before=3, behind=6)
    check_attend([50, 9, 300], [20, 1, 70], 32, 1, 3, 64, before=1, behind=17, hints=False)


@pytest.mark.parametrize("T", [16, 32, 64])
def test_attend_bad_pages(T):
    """Table entries outside the cache leave their tokens out."""
    check_attend([200, 500, 64, 1], [1, 4, 1, 1], T, 2, 4, 128, seed=T, bad_pages=6)
    got, lse = check_attend([T, T], [1, 1], T, 1, 2, 64, seed=T, edit=lambda q, c, t: t.fill(-1))
    assert np.all(got == 0) and np.all(np.isneginf(lse))


def test_attend_narrow_table():
    """Tokens past the table's width are left out."""
    check_attend([100, 500, 40], [1, 2, 1], 16, 2, 2, 128, width=4)
    check_attend([100, 5], [1, 2], 16, 2, 2, 128, width=0)


def test_attend_strides():
    check_attend([100, 37, 64], [1, 5, 2], 16, 2, 4, 128, strides=True)
    check_attend([100, 37, 64], [1, 50, 2], 64, 3, 2, 96, "fp16", strides=True)


@pytest.mark.parametrize("hints", [True, False])
def test_attend_long(hints):
    check_attend([9000, 33], [1, 1], 16, 1, 4, 128, seed=1, hints=hints)
    check_attend([7001, 5000], [3, 1], 64, 2, 2, 64, "fp16", seed=2, hints=hints)


def test_attend_wrong_hints():
    """Hints that are too small only shape the launch."""
    T, H, D = 16, 1, 128
    ref = new_pool(300, T, H, D, 1)
    gpu = gpu_cache(ref)
    lens, rows = [1900, 700], [90, 3]
    table = np.arange(240).reshape(2, 120)
    q = torch.randn(93, 4, D, device="cuda").to(torch.bfloat16)
    want = gpu.attend(q, ints(table.reshape(-1)).reshape(2, 120), ints(lens), ints(packed(rows)))
    ref_out = R.attend(ref, q.double().cpu().numpy(), table, lens, packed(rows), 1 / math.sqrt(D))
    for mq, ml in ((1, 1), (1, 0), (0, 5), (93, 1900), (5000, 1 << 30)):
        got, lse = gpu.attend(q, ints(table.reshape(-1)).reshape(2, 120), ints(lens),
                              ints(packed(rows)), max_query=mq, max_length=ml, lse=True)
        tol, tol_lse = R.attend_bounds(ref_out, 1900, D, 2.0 ** -8)
        assert np.all(np.abs(got.double().cpu().numpy() - ref_out[0]) <= tol), (mq, ml)
        assert np.all(np.abs(lse.double().cpu().numpy() - ref_out[1]) <= tol_lse), (mq, ml)
    assert want.shape == q.shape


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_attend_loud_scores(dtype):
    """One token far above the others, and scores far below zero."""
    check_attend([300, 40], [1, 3], 16, 2, 4, 128, dtype, seed=5, mag=20.0)
    check_attend([300, 40], [1, 3], 16, 2, 4, 128, dtype, seed=6, scale=1e-6)

    def spike(q, c, t):
        c.s[:, :, 1] = 2.0 ** np.random.default_rng(1).integers(-20, 20, c.s[:, :, 1].shape)
    check_attend([300, 700], [1, 3], 16, 2, 4, 128, dtype, seed=7, edit=spike)


def test_attend_not_finite():
    """A NaN code that a row sees makes that row and head NaN, and no other."""
    def edit(q, c, t):
        c.k[t[0, 2], 0, 3, 5] = 127
        c.v[t[1, 1], 1, 7, 9] = 255
        q[2, 3, 0] = math.nan
    got, lse = check_attend([100, 90, 80], [1, 1, 1], 16, 2, 2, 128, seed=8, edit=edit)
    assert np.isnan(got[0, :2]).all() and not np.isnan(got[0, 2:]).any()
    assert np.isnan(got[1, 2:, 9]).all() and np.isnan(got[1]).sum() == 2


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_attend_nan_of_unseen_tokens(dtype):
    """A NaN stored for a token reaches the rows that see it, not the earlier ones of its tile."""
    def edit(q, c, t):
        c.v[t[0, 1], 0, 9, 5] = 127       # token 25 of 40, whose rows are tokens 20 .. 39
        c.k[t[0, 2], 1, 1, 3] = 255       # token 33
        c.v[t[1, 6], 1, 0, 100] = 255     # token 96 of 130
    got, lse = check_attend([40, 130], [20, 60], 16, 2, 3, 128, dtype, seed=8, edit=edit)
    assert not np.isnan(got[:5, :3]).any() and np.isnan(got[5:20, :3, 5]).all()
    assert not np.isnan(got[:13, 3:]).any() and np.isnan(got[13:20, 3:]).all()
    assert np.isnan(got[46:, 3:, 100]).all() and not np.isnan(got[20:46]).any()


def test_attend_nothing():
    ref = new_pool(4, 16, 2, 64, 1)
    gpu = gpu_cache(ref)
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    o, l = gpu.attend(q, ints([]).reshape(0, 3), ints([]), ints([0]), lse=True)
    assert o.shape == (0, 4, 64) and l.shape == (0, 4)
    q = torch.full((3, 4, 64), 2.0, dtype=torch.bfloat16, device="cuda")
    o = torch.full((3, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    gpu.attend(q, ints([]).reshape(0, 3), ints([]), ints([0]), out=o)
    gpu.attend(q, ints([0] * 6).reshape(2, 3), ints([0, 0]), ints([0, 0, 0]), out=o)
    torch.cuda.synchronize()
    assert torch.all(o == 5.0)


def test_attend_same_twice():
    """The same call gives the same bits."""
    ref = new_pool(400, 16, 2, 128, 1)
    gpu = gpu_cache(ref)
    q = torch.randn(3, 8, 128, device="cuda").to(torch.bfloat16)
    t, lens, starts = ints(np.arange(390)).reshape(3, 130), ints([2000, 1999, 70]), ints([0, 1, 2, 3])
    a = [gpu.attend(q, t, lens, starts, lse=True) for _ in range(5)]
    for x in a[1:]:
        assert torch.equal(x[0], a[0][0]) and torch.equal(x[1], a[0][1])
