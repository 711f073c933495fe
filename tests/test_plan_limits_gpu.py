"""GPU tests of block plans at the ends of their domain."""
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
