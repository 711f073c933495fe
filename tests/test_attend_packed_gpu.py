"""GPU tests of attention over many requests whose largest number of rows is not
known, or is far above the others': tiles are then numbered through the packed
rows, and requests found by a search."""
import numpy as np
import pytest

import cache_ref as R
from attend_bounds import two_part_bounds
from test_attend_weights_gpu import is_shared
from test_cache_gpu import check_attend, ints

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

EMPTY = 16384  # workgroups without work from which on the rows are packed


@pytest.fixture(autouse=True)
def bounds(monkeypatch):
    monkeypatch.setattr(R, "attend_bounds", two_part_bounds)


def check(lens, rows, T, H, group, D, dtype="bf16", **kw):
    n = kw.get("before", 0) + sum(rows) + kw.get("behind", 0)
    most = max(rows) if kw.get("hints", False) else n
    tiles = -(-most * group // 32)  # at least
    assert len(lens) * H * tiles > (n * group // 16 + len(lens)) * H + EMPTY
    width = max(-(-x // T) for x in lens) + 1
    assert not is_shared(len(lens), n, T, H, group, D, dtype, width)
    check_attend(lens, rows, T, H, group, D, dtype, **dict(dict(hints=False), **kw))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
def test_shapes(D, dtype):
    rng = np.random.default_rng(D)
    rows = rng.integers(0, 9, 90).tolist()
    lens = [max(0, r + int(rng.integers(-3, 120))) for r in rows]
    rows[40], lens[40] = 70, 200
    check(lens, rows, 16, 2, 16, D, dtype, seed=D)
    check(lens, rows, 64, 2, 16, D, dtype, seed=D, bad_pages=9, before=5, behind=9)
    check(lens, rows, 32, 2, 16, D, dtype, seed=D, strides=True)


@pytest.mark.parametrize("B", [30, 63, 64, 65, 127, 129, 1000, 4095, 4097, 4200])
def test_searches(B):
    """Steps of the search, requests without rows among them, one that has most."""
    rng = np.random.default_rng(B)
    rows = (rng.integers(0, 3, B) * (rng.random(B) < 150 / B)).tolist()
    big = int(rng.integers(0, B))
    rows[big] = 60 if B > 30 else 150
    rows[-1] = 1
    lens = [int(rng.integers(0, 40)) if r else 1 for r in rows]
    lens[big] = rows[big] + 30
    check(lens, rows, 16, 8, 16, 64, "fp16", seed=B, before=B % 7, behind=B % 5)


def test_hints_of_a_skewed_batch():
    check([5] * 300 + [200], [1] * 300 + [150], 16, 2, 8, 64, seed=1, hints=True)


def test_rows_that_are_cut():
    """Requests that begin or end behind the rows there are."""
    H, group, D, T, B = 2, 32, 64, 16, 100
    from test_cache_gpu import gpu_cache, new_pool
    ref = new_pool(20, T, H, D, 1)
    c = gpu_cache(ref)
    starts = list(range(0, 3 * B + 1, 3))
    lens = [7 + i % 20 for i in range(B)]
    table = [[i % 20, (i + 3) % 20] for i in range(B)]
    for rows in (200, 203, 130):
        q = torch.randn(rows, H * group, D, device="cuda").to(torch.bfloat16)
        out, lse = c.attend(q, ints(table), ints(lens), ints(starts), lse=True)
        torch.cuda.synchronize()
        want = R.attend(ref, q.double().cpu().numpy(), table, lens, starts, D ** -0.5)
        tol, tol_lse = two_part_bounds(want, 30, D, 2.0 ** -8)
        assert np.all(np.abs(out.double().cpu().numpy() - want[0]) <= tol)
        assert np.all(np.abs(lse.double().cpu().numpy() - want[1]) <= tol_lse)


def test_more_numbers_than_a_grid_holds():
    """16 million requests, a 16th of them with a row of 64 heads."""
    T, D, B, every = 16, 64, (1 << 24) - 1, 16
    from test_cache_gpu import gpu_cache, new_pool
    ref = new_pool(3, T, 1, D, 1)
    c = gpu_cache(ref)
    has = (torch.arange(B, device="cuda") % every == 3).to(torch.int32)
    starts = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    starts[1:] = has.cumsum(0)
    n = int(starts[-1])
    assert n * 2 + B > (1 << 24)
    q = torch.randn(1, 64, D, device="cuda").to(torch.bfloat16).expand(n, 64, D)
    block = (torch.arange(B, device="cuda", dtype=torch.int32) // every % 3).reshape(B, 1).contiguous()
    out = torch.full((n, 64, D), 7.0, dtype=torch.bfloat16, device="cuda")
    c.attend(q, block, torch.ones(B, dtype=torch.int32, device="cuda"), starts, out=out)
    torch.cuda.synchronize()
    # each row sees one token and is its value
    value = torch.tensor(R.VALUES[ref.v[:, 0, 0]] * ref.s[:, 0, 1].astype(np.float64)[:, None]).to(torch.bfloat16)
    want = value.cuda()[torch.arange(n, device="cuda") % 3]
    for at in range(0, n, 1 << 17):
        assert torch.equal(out[at:at + (1 << 17)], want[at:at + (1 << 17), None].expand(-1, 64, -1)), at


def test_hints_are_not_needed():
    """Without hints a batch takes about what it takes with them (a grid of every
    request by all rows took 30 times as long)."""
    import recv_fifo_plane_amd as xf
    B, per, H, group, D, T, n = 1024, 16, 8, 4, 128, 16, 64
    c = xf.PagedCache(B * n // T, T, H, D)
    table = ints(np.arange(B * n // T)).reshape(B, -1)
    q = torch.randn(B * per, H * group, D, device="cuda").to(torch.bfloat16)
    lens, starts, out = ints([n] * B), ints(np.arange(B + 1) * per), torch.empty_like(q)
    times = {}
    for kw in (dict(max_query=per, max_length=n), dict()):
        took = []
        for _ in range(6):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(3):
                c.attend(q, table, lens, starts, out=out, **kw)
            b.record()
            torch.cuda.synchronize()
            took.append(a.elapsed_time(b))
        times[bool(kw)] = min(took)
    assert times[False] < 4 * times[True], times
