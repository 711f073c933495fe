"""GPU parity of block transfers (xfer_run_blocks): destination pool, counters
and FIFO bytes are those of the oracle's transfer of the gathered bytes."""
import numpy as np
import pytest

import oracle
from gpu_cases import compare_state, oracle_proto

pytestmark = pytest.mark.gpu


def torch_mod():
    import torch
    return torch


def ints(a):
    torch = torch_mod()
    return torch.tensor(np.asarray(a, dtype=np.int64).tolist(), dtype=torch.int32, device="cuda")


def run_blocks(proto, nch, nslots, slot, size, ns, nd, frm, to, fifo_loc="device", repeat=2, jitter=0,
               **attr):
    import recv_fifo_plane_amd as xf
    torch = torch_mod()
    rng = np.random.default_rng(size + len(frm))
    conn = xf.Conn(proto, nch, nslots, slot, fifo_loc, timeout_ms=20000, **attr)
    if jitter:
        conn.set_jitter(jitter)
    ocn = oracle.Conn(oracle_proto(proto, fifo_loc), nch, nslots, slot)
    src = rng.integers(0, 256, (ns, size), dtype=np.uint8)
    dst = rng.integers(0, 256, (nd, size), dtype=np.uint8)
    a, b = torch.from_numpy(src).cuda(), torch.from_numpy(dst).cuda()
    guard = torch.full((4096,), 99, dtype=torch.uint8, device="cuda")
    frm, to = np.asarray(frm, dtype=np.int64), np.asarray(to, dtype=np.int64)
    ok = (frm >= 0) & (frm < ns) & (to >= 0) & (to < nd)
    for _ in range(repeat):
        conn.run_blocks(a, b, size, ints(frm), ints(to))
        gathered = np.where(ok[:, None], src[np.where(ok, frm, 0)], 0).astype(np.uint8).reshape(-1)
        there = np.zeros_like(gathered)
        ocn.run(gathered, there)
        there = there.reshape(len(frm), size)
        dst[to[ok]] = there[ok]
        torch.cuda.synchronize()
        compare_state(conn, ocn, nch, "%s %d" % (proto, size))
        got = b.cpu().numpy()
        assert np.array_equal(got, dst), np.argwhere(got != dst)[:5]
        assert np.array_equal(a.cpu().numpy(), src)
    assert torch.all(guard == 99)
    conn.close()
    ocn.close()


PROTOS = [("simple", "device"), ("simple", "host"), ("simple", "relay"), ("zcd", "device"), ("zcd", "host")]


@pytest.mark.parametrize("proto,fifo_loc", PROTOS)
@pytest.mark.parametrize("size", [16, 48, 1008, 1024, 1040, 2176, 4096, 33280])
def test_blocks(proto, fifo_loc, size):
    rng = np.random.default_rng(size)
    n = 57
    run_blocks(proto, 4, 4, 16384, size, 80, 90, rng.permutation(80)[:n], rng.permutation(90)[:n],
               fifo_loc, wgs_per_channel=2)


@pytest.mark.parametrize("proto", ["simple", "zcd"])
@pytest.mark.parametrize("nch,lanes,block,slot", [(1, 1, 64, 4096), (3, 4, 256, 65536), (8, 16, 128, 8192),
                                                  (32, 4, 768, 524288), (32, 16, 128, 524288),
                                                  (2, 1, 1024, 1 << 20), (1, 3, 192, 48)])
def test_blocks_shapes(proto, nch, lanes, block, slot):
    rng = np.random.default_rng(nch + slot)
    for size, n in ((33280, 70), (80, 401)):
        run_blocks(proto, nch, 3, slot, size, n + 9, n + 2, rng.permutation(n + 9)[:n],
                   rng.permutation(n + 2)[:n], wgs_per_channel=lanes, block_threads=block)


@pytest.mark.parametrize("proto,fifo_loc", PROTOS)
@pytest.mark.parametrize("size", [64, 2176, 16640])
def test_entries_outside_the_pools_move_nothing(proto, fifo_loc, size):
    rng = np.random.default_rng(3)
    n, ns, nd = 60, 70, 65
    frm, to = rng.permutation(ns)[:n], rng.permutation(nd)[:n]
    frm[[0, 7, 30]] = [-1, ns, 2 ** 31 - 1]
    to[[3, 30, n - 1]] = [nd, -1, -2 ** 31]
    run_blocks(proto, 4, 2, 8192, size, ns, nd, frm, to, fifo_loc, wgs_per_channel=2)
    run_blocks(proto, 2, 2, 8192, size, ns, nd, np.full(9, -1), to[:9], fifo_loc)


@pytest.mark.parametrize("proto", ["simple", "zcd"])
def test_one_block_and_repeats(proto):
    run_blocks(proto, 4, 2, 4096, 4096, 3, 3, [2], [0])
    run_blocks(proto, 4, 2, 4096, 2176, 3, 9, [1] * 9, range(9))  # one source block, many places


@pytest.mark.parametrize("proto", ["simple", "zcd"])
@pytest.mark.parametrize("kw", [dict(ordering=1), dict(xcd_pairing=-1), dict(jitter=77), dict(cooperative=1)])
def test_blocks_variants(proto, kw):
    rng = np.random.default_rng(1)
    run_blocks(proto, 8, 4, 32768, 16640, 40, 40, rng.permutation(40), rng.permutation(40),
               wgs_per_channel=4, **kw)


def test_blocks_p2p_read():
    rng = np.random.default_rng(2)
    run_blocks("simple", 8, 4, 32768, 16640, 40, 40, rng.permutation(40), rng.permutation(40),
               wgs_per_channel=4, p2p_read=1)


def test_blocks_between_transfers():
    """Counters carry on between block transfers and others on one connection."""
    import recv_fifo_plane_amd as xf
    torch = torch_mod()
    conn, ocn = xf.Conn("simple", 2, 2, 4096), oracle.Conn("simple", 2, 2, 4096)
    src = np.random.default_rng(1).integers(0, 256, (30, 2176), dtype=np.uint8)
    a, b = torch.from_numpy(src).cuda(), torch.zeros(30, 2176, dtype=torch.uint8, device="cuda")
    order = np.random.default_rng(2).permutation(30)
    conn.run(a, b, 30 * 2176)
    conn.run_blocks(a, b, 2176, ints(order), ints(range(30)))
    torch.cuda.synchronize()
    tmp = np.zeros(30 * 2176, dtype=np.uint8)
    ocn.run(src.reshape(-1), tmp)
    ocn.run(src[order].reshape(-1), tmp)
    assert np.array_equal(b.cpu().numpy().reshape(-1), tmp)
    compare_state(conn, ocn, 2, "mixed")
    conn.close()


def test_far_blocks():
    """Blocks beyond 4 GiB of a pool."""
    import recv_fifo_plane_amd as xf
    torch = torch_mod()
    size, nb = 1 << 20, 4500
    conn = xf.Conn("zcd", 4, 1, 65536, wgs_per_channel=2)
    a = torch.zeros(nb, size, dtype=torch.uint8, device="cuda")
    b = torch.zeros(nb, size, dtype=torch.uint8, device="cuda")
    ids = [0, 2049, 4499, 4100]
    for i in ids:
        a[i] = i % 251 + 1
    conn.run_blocks(a, b, size, ints(ids), ints([4498, 4200, 1, 2050]))
    torch.cuda.synchronize()
    for f, t in zip(ids, [4498, 4200, 1, 2050]):
        assert torch.equal(a[f], b[t])
    assert int((b.sum(1, dtype=torch.int64) > 0).sum()) == 4
    conn.close()


def test_refusals():
    import recv_fifo_plane_amd as xf
    from recv_fifo_plane_amd import xfer as X
    torch = torch_mod()
    pool = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    other = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    p, q, ids = pool.data_ptr(), other.data_ptr(), ints([0, 1]).data_ptr()
    L = xf.lib()
    for proto in ("ll", "zc"):
        c = xf.Conn(proto, 1, 2, 4096)
        assert L.xfer_run_blocks(c.handle, p, 4, q, 4, 1024, ids, ids, 2, None) == X.XFER_ERR_INVALID_ARG
        c.close()
    c = xf.Conn("simple", 1, 2, 4096)
    ok = [c.handle, p, 4, q, 4, 1024, ids, ids, 2, None]
    for i, bad in ((1, None), (3, None), (6, None), (7, None), (5, 0), (5, 24), (5, (1 << 30) + 16),
                   (1, p + 8), (3, q + 4), (6, ids + 2), (7, ids + 1), (2, 1 << 31), (4, 1 << 31),
                   (8, 1 << 31), (3, p), (3, p + 1024), (1, q + 2048), (6, q), (7, q + 4092)):
        args = list(ok)
        args[i] = bad
        assert L.xfer_run_blocks(*args) == X.XFER_ERR_INVALID_ARG, (i, bad)
        assert "xfer_run_blocks" in xf.last_error()
    assert L.xfer_run_blocks(c.handle, None, 0, None, 0, 1024, None, None, 0, None) == 0
    torch.cuda.synchronize()
    assert c.query(0)["steps"] == 0
    c.close()
