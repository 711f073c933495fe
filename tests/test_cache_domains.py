"""CPU tests of refusals: calls that the cache's operators would answer wrongly
without a word."""
import ctypes as C

import pytest
import torch

import cache_ref as R
import recv_fifo_plane_amd as xf
from recv_fifo_plane_amd import cache as K
from recv_fifo_plane_amd import xfer as X
from test_cache_refusals import FakeTensor, Unreachable


@pytest.fixture
def cache(monkeypatch):
    c = xf.PagedCache(10, 16, 2, 128, buffer=FakeTensor((10, R.block_bytes(16, 2, 128)), torch.uint8))
    monkeypatch.setattr(X, "_lib", Unreachable())
    return c


@pytest.mark.parametrize("dtype", [torch.uint32, torch.int64, torch.float32, torch.int16])
@pytest.mark.parametrize("which", [0, 1])
def test_block_lists_are_int32(cache, which, dtype):
    """(uint32 among them: its large numbers are not the blocks that int32 ids name)"""
    conn = X.Conn("simple", 1, 8, 4096, _handle=0x1234)
    conn.device = 0
    try:
        pools = [FakeTensor((10, 4096), torch.uint8, ptr=p << 40) for p in (1, 2)]
        ids = [FakeTensor((4,)), FakeTensor((4,))]
        n = 16 // torch.empty(0, dtype=dtype).element_size()  # as many bytes as four int32
        ids[which] = FakeTensor((n,), dtype)
        with pytest.raises(TypeError, match="int32"):
            conn.run_blocks(*pools, 4096, *ids)
    finally:
        conn._h = None


BF = torch.bfloat16


def attend_args(**query):
    q = FakeTensor((4, 4, 128), BF)
    q.__dict__.update(query)
    return q, FakeTensor((3, 8)), FakeTensor((3,)), FakeTensor((4,))


class Launched(Exception):
    pass


def launches(monkeypatch):
    class Library:
        def __getattr__(self, name):
            raise Launched(name)
    monkeypatch.setattr(X, "_lib", Library())


def test_attend_has_no_gradient(cache, monkeypatch):
    """A query (or out) that asks for a gradient gets an error, not a result without
    one; under no_grad it is computed."""
    out = FakeTensor((4, 4, 128), BF)
    with pytest.raises(ValueError, match="gradient"):
        cache.attend(*attend_args(requires_grad=True), out=out)
    out.requires_grad = True
    with pytest.raises(ValueError, match="gradient"):
        cache.attend(*attend_args(), out=out)
    launches(monkeypatch)
    for context in (torch.no_grad, torch.inference_mode):
        with context(), pytest.raises(Launched):
            cache.attend(*attend_args(requires_grad=True), out=out)
    with pytest.raises(Launched):
        cache.attend(*attend_args(requires_grad=False), out=FakeTensor((4, 4, 128), BF))


OVERLAPPING = [  # strides of a row and of a head, rows, heads: elements that two rows would write
    (0, 128, 4, 4), (256, 128, 4, 4), (512, 64, 4, 4), (512, 0, 4, 4), (64, 512, 4, 4), (128, 256, 4, 4),
    (-256, 128, 4, 4), (512, -64, 4, 4), (127, 128, 4, 1), (1, 1, 2, 1), (384, 127, 1, 4),
    (1 << 62, 1 << 62, 4, 4), (-(1 << 63), 100, 4, 4)]
APART = [  # and those that write each element once
    (512, 128, 4, 4), (128, 512, 4, 4), (520, 130, 4, 4), (-512, 128, 4, 4), (512, -128, 4, 4),
    (0, 128, 1, 4), (128, 0, 4, 1), (0, 0, 1, 1), (1 << 40, 1 << 50, 4, 4), (-(1 << 63), 128, 4, 4)]


def raw_attend(row, head, rows, heads, **kw):
    p = 1 << 40
    a = X.xfer_attend(p, p, None, p, p, p, None, 0, 512, 128, row, head, 1, 1, rows, heads, 1, 0, 1.0, 0, 0)
    for k, v in kw.items():
        setattr(a, k, v)
    return X.lib().xfer_cache_attend(C.byref(X.xfer_cache_shape(16, 1, 128, 10)), p, C.byref(a), None)


@pytest.mark.parametrize("row,head,rows,heads", OVERLAPPING)
def test_attend_refuses_overlapping_outputs(row, head, rows, heads):
    assert raw_attend(row, head, rows, heads) == X.XFER_ERR_INVALID_ARG
    assert "overlap" in xf.last_error()


@pytest.mark.parametrize("row,head,rows,heads", APART)
def test_attend_takes_outputs_that_do_not_overlap(row, head, rows, heads):
    """(refused for the workspace, which is looked at behind the strides)"""
    assert raw_attend(row, head, rows, heads, workspace_bytes=0, table_width=1 << 20,
                      table_stride=1 << 20) == X.XFER_ERR_INVALID_ARG
    assert "workspace" in xf.last_error()


def test_attend_refuses_an_expanded_out(monkeypatch):
    c = xf.PagedCache(10, 16, 2, 128, buffer=FakeTensor((10, R.block_bytes(16, 2, 128)), torch.uint8))
    K._kinds()
    monkeypatch.setattr(K, "_RAW", lambda device: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(xf.XferError, match="overlap"):
        c.attend(*attend_args(), out=FakeTensor((4, 4, 128), BF, strides=(0, 128, 1)))


BIG = 1 << 32  # what a C int drops


@pytest.mark.parametrize("i", range(4))
def test_sizes_of_a_cache_beyond_an_int(i):
    sizes = [10, 16, 2, 128]
    sizes[i] += BIG
    with pytest.raises(ValueError, match="2\\^31"):
        xf.PagedCache(*sizes, buffer=FakeTensor((sizes[0], R.block_bytes(16, 2, 128)), torch.uint8))


@pytest.mark.parametrize("block,rows", [(BIG + 16, 20), (16 - BIG, 20), (16, BIG + 20), (16, (1 << 31) + 20)])
def test_sizes_of_a_plan_beyond_an_int(cache, block, rows):
    out = xf.BlockPlan(*(FakeTensor((n,)) for n in (rows, rows, 4, 3, 2)))
    with pytest.raises(ValueError, match="2\\^31"):
        K.plan_blocks(FakeTensor((3,)), FakeTensor((3,)), FakeTensor((3, 8)), FakeTensor((5,)), block, rows,
                      out=out)


@pytest.mark.parametrize("free,width", [(BIG + 5, 8), (5, BIG + 8)])
def test_lists_of_a_plan_beyond_an_int(cache, free, width):
    out = xf.BlockPlan(*(FakeTensor((n,)) for n in (20, 20, 4, 3, 2)))
    with pytest.raises(ValueError, match="2\\^31"):
        K.plan_blocks(FakeTensor((3,)), FakeTensor((3,)), FakeTensor((3, width)), FakeTensor((free,)), 16, 20,
                      out=out)


@pytest.mark.parametrize("kw", [dict(max_query=BIG), dict(max_length=BIG + 5), dict(max_query=5 - BIG), dict(max_length=1 << 31)])
def test_hints_beyond_an_int(cache, kw):
    with pytest.raises(ValueError, match="2\\^31"):
        cache.attend(*attend_args(), out=FakeTensor((4, 4, 128), BF), **kw)


def test_rows_of_a_store_beyond_an_int(cache):
    rows = FakeTensor((BIG + 4, 2, 128), BF, strides=(0, 128, 1))
    with pytest.raises(ValueError, match="2\\^31"):
        cache.store(rows, rows, FakeTensor((BIG + 4,)))
