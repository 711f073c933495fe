"""CPU tests of refusals: calls that the cache's operators would answer wrongly
without a word."""
import pytest
import torch

import cache_ref as R
import recv_fifo_plane_amd as xf
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
