"""GPU tests of block plans at the ends of their domain."""
import numpy as np
import pytest

import cache_ref as R
from test_cache_gpu import ints

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def xf():
    import recv_fifo_plane_amd
    return recv_fifo_plane_amd


@pytest.mark.parametrize("rows", [2 ** 31 - 1, 2 ** 31 - 1000, 2 ** 30 + 7])
def test_as_many_rows_as_an_int_holds(rows):
    """Rows behind the packed ones are marked, up to the last of 2^31 - 1."""
    B, T = 300, 16
    cached, added = [i % 40 for i in range(B)], [i % 3 for i in range(B)]
    table = [[100 * i + p if p < -(-cached[i] // T) else -1 for p in range(4)] for i in range(B)]
    free = list(range(50000, 50700))
    plan = xf().plan_blocks(ints(cached), ints(added), ints(table), ints(free), T, rows)
    n = sum(added)
    slots, positions, starts, lengths, counts, _ = R.plan(cached, added, table, free, T, n)
    assert plan.slots[:n].tolist() == slots and plan.positions[:n].tolist() == positions
    assert plan.starts.tolist() == starts and plan.lengths.tolist() == lengths
    assert plan.counts.tolist() == counts
    step = 1 << 28
    for x in (plan.slots, plan.positions):
        assert x.numel() == rows
        for at in range(n, rows, step):
            assert bool((x[at:at + step] == -1).all()), at


@pytest.mark.parametrize("T", [16, 32, 64])
@pytest.mark.parametrize("nfree", [0, 40, 5000])
@pytest.mark.parametrize("B,width", [(1, 4), (60, 5), (1500, 6)])
def test_lost_tokens_are_those_without_a_slot(B, width, nfree, T):
    """Also where a request's last block is missing from its table, as an earlier plan
    without room leaves it."""
    rng = np.random.default_rng(B + nfree + T)
    cached, added = (rng.integers(0, 7 * T, B).tolist() for _ in range(2))
    held = [-(-c // T) for c in cached]
    table = [[(-1 if rng.random() < 0.3 else 100 * i + p) if p < held[i] else -1 for p in range(width)]
             for i in range(B)]
    free = list(range(200000, 200000 + nfree))
    n = sum(added)
    plan = xf().plan_blocks(ints(cached), ints(added), ints(table), ints(free), T, n + 3)
    slots = R.plan(cached, added, table, free, T, n)[0]
    assert plan.slots[:n].tolist() == slots
    assert plan.counts.tolist()[1] == slots.count(-1)


def test_no_room_then_the_next_token():
    """A token lost in one plan: the next one of the same block is lost too, and counted."""
    table = ints([[-1, -1]])
    first = xf().plan_blocks(ints([0]), ints([1]), table, ints([]), 16, 1)
    second = xf().plan_blocks(ints([1]), ints([1]), table, ints([7, 8]), 16, 1)
    for plan in (first, second):
        assert plan.slots.tolist() == [-1] and plan.counts.tolist()[1] == 1
