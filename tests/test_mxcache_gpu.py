"""GPU tests of the 4-bit cache's stores and of reading either cache back, against
plain forms in 64 bits: every byte, every rounded number."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import cache_ref  # noqa: E402
import mxcache_ref as R  # noqa: E402
from mxcache_cases import check_load, check_store, gpu_cache, ints, new_pool, xf  # noqa: E402

pytestmark = pytest.mark.gpu

DIMS = [64, 96, 128, 192, 256]
TYPES = ["bf16", "fp16", "fp32"]


# ----------------------------------------------------------------------- store
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("T", [16, 32, 64])
def test_store_runs(T, D, dtype):
    slots = [3 * T + i for i in range(T)] + [5 * T + 3, 5 * T + 4] + [T - 1] + [7 * T + i for i in range(2, 9)]
    check_store(T, 2, D, dtype, slots, T + D)


@pytest.mark.parametrize("H,n", [(1, 1), (1, 3), (3, 1), (5, 7), (8, 33), (17, 4), (2, 300)])
def test_store_sizes(H, n):
    rng = np.random.default_rng(n)
    check_store(16, H, 64, "bf16", rng.permutation(30 * 16)[:n].tolist(), n)
    check_store(64, H, 96, "fp16", rng.permutation(30 * 64)[:n].tolist(), n + 1)


@pytest.mark.parametrize("dtype", TYPES)
def test_store_any_order(dtype):
    """Tokens of one block in any order, blocks in turn: none touches another."""
    rng = np.random.default_rng(1)
    for D in DIMS:
        check_store(16, 2, D, dtype, rng.permutation(64).tolist(), D, blocks=4)
        check_store(32, 1, D, dtype, list(range(63, 20, -1)), D, blocks=2)


@pytest.mark.parametrize("T", [16, 64])
def test_store_slots_outside(T):
    """Padded rows and slots outside the cache are passed over."""
    n = 6 * T
    slots = [-1, 0, n, n - 1, n + 5, -7, T, 2 ** 31 - 1, -2 ** 31, 2 * T + 1]
    check_store(T, 3, 128, "bf16", slots, 2, blocks=6)
    check_store(T, 3, 192, "fp32", [-1] * 9, 2, blocks=6)


@pytest.mark.parametrize("dtype", TYPES)
def test_store_strides(dtype):
    for D in DIMS:
        check_store(16, 3, D, dtype, list(range(40, 75)), D, strides=True)


@pytest.mark.parametrize("dtype", TYPES)
def test_store_ties_and_ends(dtype):
    """Numbers half way between codes and next to that, and magnitudes around 7 times a scale."""
    def edit(key, value):
        ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0], dtype=torch.float64)
        step = torch.finfo(key.dtype).eps
        near = torch.cat([ties, ties * (1 - step), ties * (1 + step), -ties]).cuda()
        key[:, :, :32] = near.to(key.dtype)
        key[:, :, 31] = 7.0 if key.dtype == torch.float32 else -7.0
        for i in range(key.shape[0]):
            value[i] = (near.repeat(4) * 2.0 ** (i - 8)).to(value.dtype)
            value[i, 0, 64:96] = near.flip(0).to(value.dtype)
    check_store(16, 2, 128, dtype, list(range(16)), 4, edit=edit)


@pytest.mark.parametrize("dtype", TYPES)
def test_store_ranges(dtype):
    """Zeros of both signs, the smallest and the largest numbers of the type."""
    def edit(key, value):
        info = torch.finfo(key.dtype)
        key[0] = 0.0
        key[1] = -0.0
        key[2] = info.tiny
        key[3] = -info.tiny * info.eps                       # the smallest below the normal ones
        key[4, :, ::2] = info.max
        key[5, :, ::32] = -info.max
        key[6] *= info.tiny
        value[0, :, 5] = info.max
        value[1] = info.max * 0.9
        for i in range(2, 16):
            value[i] = value[i].float() * 2.0 ** (9 * i - 130 if key.dtype != torch.float16 else i - 24)
        value[9, :, 64:] = 0.0
    check_store(16, 2, 128, dtype, list(range(16)), 5, edit=edit)


@pytest.mark.parametrize("dtype", TYPES)
def test_store_not_finite(dtype):
    """Infinities and NaN make their 32 dims NaN and no others; storing over them heals."""
    def edit(key, value):
        key[0, 0, 5] = math.nan
        key[1, 1, 33] = math.inf
        key[2, 0, 127] = -math.inf
        value[0, 1, 0] = math.inf
        value[3, :, 96:] = math.nan
        value[4] = -math.nan
    ref, gpu = check_store(16, 2, 128, dtype, list(range(16)), 6, edit=edit)
    assert (ref.s[0, :, 0, :, :3] == 255).sum() == 3 and (ref.s[0, :, 1, :, 4] == 255).all()
    rows = torch.ones(16, 2, 128, device="cuda").to(torch.bfloat16)
    gpu.store(rows, rows, ints(range(16)))
    torch.cuda.synchronize()
    R.store(ref, np.ones((16, 2, 128)), np.ones((16, 2, 128)), range(16))
    assert np.array_equal(gpu.buffer.cpu().numpy(), ref.raw())


def test_store_nothing():
    ref = new_pool(3, 16, 2, 64, 1)
    gpu = gpu_cache(ref)
    empty = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    gpu.store(empty, empty, ints([]))
    torch.cuda.synchronize()
    assert np.array_equal(gpu.buffer.cpu().numpy(), ref.raw())


@pytest.mark.parametrize("n,H,D", [(3000, 8, 128), (2500, 3, 96), (1111, 5, 256)])
def test_store_many_rows(n, H, D):
    """Prompts of many rows, every byte against the plain form in torch."""
    T = 32
    c = xf().PagedCache(n // T + 2, T, H, D, bits=4)
    g = torch.Generator(device="cuda").manual_seed(n)
    kv = torch.randn(n, 2 * H, D, generator=g, device="cuda").to(torch.bfloat16)
    slots = torch.arange(n, device="cuda", dtype=torch.int32) + 5
    c.store(kv[:, :H], kv[:, H:], slots)
    got = R.Cache(c.buffer.cpu().numpy(), T, H, D)
    table = np.arange(c.blocks)
    for side in range(2):
        x = kv[:, side * H:(side + 1) * H].double().cpu().numpy().reshape(n, H, D // 32, 32)
        amax = np.abs(x).max(-1)
        e = np.clip(np.ceil(np.log2(amax / 7)), -118, 125)
        e += amax > 7 * 2.0 ** e
        want = (R.CODES[R.to_codes(x / 2.0 ** e[..., None])] * 2.0 ** e[..., None]).reshape(n, H, D)
        pos = np.arange(n) + 5
        for h in range(H):
            assert np.array_equal(got.tokens(side, table[pos // T], h, pos % T), want[:, h])
    assert (got.s[0, :, :, :, :5] == 0).all() and (got.k[0, :, :5] == 0).all() and (got.v[0, :, :5] == 0).all()


# ------------------------------------------------------------------------ load
def pair(bits, blocks, T, H, D, seed, extremes=False):
    """A plain cache and the same one on the GPU."""
    if bits == 4:
        ref = new_pool(blocks, T, H, D, seed)
        if extremes:
            rng = np.random.default_rng(seed)
            ref.s[:] = rng.integers(9, 253, ref.s.shape)
            ref.s[rng.random(ref.s.shape) < 0.05] = 255
        return ref, gpu_cache(ref)
    import test_cache_gpu as G
    ref = G.new_pool(blocks, T, H, D, seed, full=not extremes)
    if extremes:
        ref.s[:] = 2.0 ** np.random.default_rng(seed).integers(-118, 119, ref.s.shape)
    return R.Eight(ref), G.gpu_cache(ref)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("T", [16, 32, 64])
def test_load_shapes(T, D, dtype, bits):
    cache = pair(bits, 60, T, 2, D, T + D)
    check_load(cache, [1, T - 1, T, T + 1, 150, 5], [1, T - 1, T, 3, 131, 0], dtype, seed=D)
    check_load(cache, [1, 15, 16, 17, 33, 64], [1] * 6, dtype, seed=D, new=True)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("H", [1, 3, 5, 16, 33])
def test_load_heads(H, bits):
    check_load(pair(bits, 20, 16, H, 64, H), [70, 3, 40], [70, 2, 39], "bf16", seed=H)
    check_load(pair(bits, 20, 32, H, 96, H), [70, 3, 40], [1, 2, 39], "fp16", seed=H, strides=True)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", TYPES)
def test_load_ranges(dtype, bits):
    """Scales from 2^-118 up, NaN; what float16 cannot hold becomes infinite or is rounded."""
    for D in (96, 128):
        check_load(pair(bits, 30, 16, 2, D, 3, extremes=True), [200, 100], [200, 77], dtype)


@pytest.mark.parametrize("bits", [4, 8])
def test_load_rows_of_no_request(bits):
    cache = pair(bits, 40, 16, 2, 128, 4)
    check_load(cache, [50, 9, 0, 30], [20, 9, 0, 1], "bf16", before=3, behind=40)
    check_load(cache, [50, 9, 0, 30], [20, 9, 0, 1], "fp32", before=37, behind=5, strides=True)
    check_load(cache, [200, 90], [150, 90], "bf16", cut=100)       # rows that are not there
    check_load(cache, [200, 90], [150, 90], "bf16", cut=17, before=1)


@pytest.mark.parametrize("bits", [4, 8])
def test_load_missing_tokens(bits):
    """Rows before the first token, entries outside the cache, a narrow table: 0."""
    cache = pair(bits, 40, 16, 2, 128, 5)
    check_load(cache, [3, 0, -5, 20, 100], [9, 4, 2, 40, 133], "bf16")
    check_load(cache, [200, 64, 130], [200, 64, 100], "fp16", bad_pages=12)
    check_load(cache, [200, 64, 130], [200, 64, 130], "fp32", width=4)
    check_load(cache, [20, 6], [20, 6], "bf16", width=0)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("B", [2, 63, 64, 65, 129, 1000, 4097])
def test_load_batches(B, bits):
    """Steps of the search for a row's request, requests without rows among them."""
    rng = np.random.default_rng(B)
    lens = rng.integers(-2, 40, B)
    rows = np.where(rng.random(B) < min(1.0, 300 / B), rng.integers(0, 30, B), 0)
    cache = pair(bits, int(np.ceil(np.maximum(lens, 0) / 16).sum()) + 1, 16, 1, 64, B)
    check_load(cache, lens.tolist(), rows.tolist(), "bf16", seed=B, before=B % 19)


@pytest.mark.parametrize("bits", [4, 8])
def test_load_nothing(bits):
    _, gpu = pair(bits, 4, 16, 2, 64, 1)
    k, v = gpu.load(ints([]).reshape(0, 3), ints([]), ints([0]), 0)
    assert k.shape == v.shape == (0, 2, 64) and k.dtype == torch.bfloat16
    out = [torch.full((3, 2, 64), 5.0, device="cuda") for _ in range(2)]
    gpu.load(ints([]).reshape(0, 3), ints([]), ints([0]), 3, out=out)
    gpu.load(ints([0] * 6).reshape(2, 3), ints([9, 9]), ints([0, 0, 0]), 3, out=out)
    torch.cuda.synchronize()
    assert all(torch.all(x == 5.0) for x in out)


def test_load_gives_what_was_stored():
    """What a 4-bit cache holds, stored again, is held unchanged."""
    T, H, D = 16, 3, 192
    rng = np.random.default_rng(0)
    ref, gpu = pair(4, 20, T, H, D, 7)
    table, n = ints(rng.permutation(20)[:12]).reshape(1, 12), 12 * T
    for dtype in (torch.bfloat16, torch.float32):
        k, v = gpu.load(table, ints([n]), ints([0, n]), n, dtype=dtype)
        other = xf().PagedCache(12, T, H, D, bits=4)
        other.store(k, v, ints(range(n)))
        k2, v2 = other.load(ints(range(12)).reshape(1, 12), ints([n]), ints([0, n]), n, dtype=dtype)
        torch.cuda.synchronize()
        assert torch.equal(k, k2) and torch.equal(v, v2)


def test_cache_ref_is_of_8_bits():
    assert cache_ref.block_bytes(16, 2, 64) > R.block_bytes(16, 2, 64)
