"""GPU tests of stores by the number of rows of a call, which decides how the runs
are dealt to workgroups: ragged prompts that go on with blocks that hold tokens
already, with padded rows among them, compared bit by bit."""
import numpy as np
import pytest

from test_cache_gpu import check_store

pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = ["bf16", "fp16", "fp32"]


def prompts(T, rows, seed, longest, in_order=False):
    """Slots of `rows` packed rows of prompts of up to `longest` tokens, each behind a
    cached part, with padding between some; and the blocks of their pool."""
    rng = np.random.default_rng(seed)
    runs, total = [], 0
    while total < rows:
        first = int(rng.integers(0, T)) if rng.random() < 0.8 else 0  # of the block it goes on with
        runs.append((first, int(rng.integers(1, longest + 1))))
        total += runs[-1][1]
    blocks = sum(-(-(first + n) // T) for first, n in runs) + 5
    ids = list(range(blocks)) if in_order else rng.permutation(blocks).tolist()
    slots = []
    for first, n in runs:
        need = -(-(first + n) // T)
        mine, ids = ids[:need], ids[need:]
        slots += [mine[p // T] * T + p % T for p in range(first, first + n)]
        if rng.random() < 0.4:
            slots += [-1] * int(rng.integers(1, 5))
        elif rng.random() < 0.2:
            slots += [blocks * T + int(rng.integers(0, 99))]
    return slots[:rows], blocks


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D,H", [(64, 3), (96, 1), (128, 3), (192, 1), (256, 3)])
@pytest.mark.parametrize("T", [16, 32, 64])
def test_prompts(T, D, H, dtype):
    for rows, longest in ((2049 + T + D % 61, 5 * T + 3), (2600 + D, 700), (257, 3 * T), (1999, 90),
                          (2048, 1500)):
        slots, blocks = prompts(T, rows, T + D + rows, longest)
        check_store(T, H, D, dtype, slots, seed=rows, blocks=blocks)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [16, 32, 64])
def test_consecutive_blocks(T, dtype):
    """Runs of neighbouring blocks whose slots go on across the border."""
    for rows in (300, 2500):
        slots, blocks = prompts(T, rows, T, 4 * T, in_order=True)
        check_store(T, 2, 128, dtype, slots, seed=T, blocks=blocks)


@pytest.mark.parametrize("T", [16, 32, 64])
@pytest.mark.parametrize("rows", [255, 256, 257, 2047, 2048, 2049, 2111, 4500])
def test_single_tokens(T, rows):
    rng = np.random.default_rng(rows)
    slots = (rng.permutation(rows + 9)[:rows] * T + rng.integers(0, T, rows)).tolist()
    check_store(T, 1, 64, "bf16", slots, seed=rows, blocks=rows + 9)


def test_shared_rows_and_strides():
    """Rows and heads of a wider tensor, by thousands."""
    slots, blocks = prompts(64, 2333, 5, 400)
    check_store(64, 3, 128, "fp16", slots, seed=1, blocks=blocks, strides=True)
    slots, blocks = prompts(16, 1111, 6, 200)
    check_store(16, 3, 96, "fp32", slots, seed=2, blocks=blocks, strides=True)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,D", [(16, 64), (64, 128), (64, 256), (32, 96)])
def test_not_finite_in_long_calls(T, D, dtype):
    slots, blocks = prompts(T, 2222, T, 300)

    def edit(k, v):
        rng = np.random.default_rng(D)
        for x in (k, v):
            at = rng.integers(0, 2222, 60)
            x[at, rng.integers(0, 2, 60), rng.integers(0, D, 60)] = rng.choice([np.nan, np.inf, -np.inf], 60)
        k[100:300] = np.nan  # whole runs of them
    check_store(T, 2, D, dtype, slots, seed=3, blocks=blocks, edit=edit)
