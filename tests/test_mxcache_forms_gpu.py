"""GPU tests of attention over the 4-bit cache in tiles of many rows for float16 queries: each run of
64 tokens is multiplied in the form that its own scales ask for."""
import pytest

torch = pytest.importorskip("torch")
import numpy as np  # noqa: E402
from mxcache_cases import gpu_cache, ints, is_shared, many_length, new_pool, table_of  # noqa: E402
from test_mxcache_attend_gpu import DIMS, pairs  # noqa: E402

pytestmark = pytest.mark.gpu

SHORT, LONG = 130, 600  # tokens: the first request's, all of them new, and the second's, half of them


def one_call(D, edit, shared, scale, seed=1, dtype=torch.float16):
    """out and lse of a call of queries whose first dim is 1, with values that cancel;
    edit(pool, table)."""
    T, (H, group) = 16, ((2, 3) if shared else (32, 4) if D <= 128 else (16, 4))
    rows = [SHORT, LONG // 2]
    c = new_pool(50, T, H, D, seed)
    table = np.full((2, 76), -1)
    order = np.random.default_rng(seed).permutation(50)
    table[0, :9], table[1, :38] = order[:9], order[9:47]
    q = torch.randn(sum(rows), H * group, D, generator=torch.Generator().manual_seed(seed))
    pairs(q, c, table)
    q[..., 0] = 1
    q = q.to(dtype)
    edit(c, table)
    hints = {}
    if shared:
        width = -(-many_length(sum(rows), H, group, D) // T)
        table = np.pad(table, ((0, 0), (0, width - 76)), constant_values=-1)
    else:
        hints["max_length"] = 1216
    assert is_shared(2, sum(rows), T, H, group, D, "fp16" if dtype == torch.float16 else "bf16",
                     table.shape[1], max(rows), **hints) == shared
    return gpu_cache(c).attend(q.cuda(), table_of(table), ints([SHORT, LONG]), ints([0, rows[0], sum(rows)]),
                               lse=True, max_query=max(rows), scale=scale, **hints)


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("D", DIMS)
def test_one_run_does_not_decide_for_the_next(D, shared):
    """Of each request 64 tokens have scores so far down (-192 of about 1) that they add nothing to any row that sees
    another: weights of exactly 0, or what they add up to multiplied by 0 later.  Their
    keys are the same numbers with a scale byte that float16 numbers allow (135) and one that they do
    not (136, half the code).  So outputs are the same in every bit if the other runs are taken
    in the same form."""
    def far(byte, code):
        def edit(c, table):
            for b, chunk in ((0, 0), (1, 2)):
                for page in table[b, 4 * chunk:4 * chunk + 4]:
                    c.k[page, :, :, :32] = 0
                    c.k[page, :, :, 0] = code
                    c.s[page, :, 0, 0] = byte
        return edit

    scale = 1 / 8
    want, got = (one_call(D, far(*x), shared, scale) for x in ((135, 15), (136, 13)))
    for x, y in zip(want, got):
        assert torch.isfinite(x).all()
        assert torch.equal(x[64:], y[64:])  # (the first request's first 64 rows see nothing else)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("D", DIMS)
def test_no_block_stands_in_for_one_that_is_missing(D, shared, dtype):
    """Where a table names no block of the cache, outputs do not depend on what any other block holds."""
    def missing(byte, code):
        def edit(c, table):
            table[table == 0] = 49 if 49 not in table else max(set(range(1, 49)) - set(table.ravel().tolist()))
            for b, page, bad in ((0, 1, -1), (1, 0, 50), (1, 13, 2 ** 31 - 1), (1, 20, -2 ** 31)):
                table[b, page] = bad
            c.k[0], c.v[0], c.s[0] = code, code, byte
        return edit

    want = one_call(D, missing(127, 3), shared, 0.1, dtype=dtype)
    for byte, code in ((0, 0), (9, 0), (143, 15), (255, 1)):
        got = one_call(D, missing(byte, code), shared, 0.1, dtype=dtype)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), byte
