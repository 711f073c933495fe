"""CPU tests of the paged cache's argument checks: a call outside the
documented domain is refused before anything is launched."""
import ctypes as C

import numpy as np
import pytest
import torch

import cache_ref as R
import recv_fifo_plane_amd as xf
from recv_fifo_plane_amd import cache as K
from recv_fifo_plane_amd import xfer as X

INVALID = X.XFER_ERR_INVALID_ARG
P = 1 << 40  # an aligned address that no refused call may touch


def _shape(t=16, h=2, d=128, blocks=10):
    return X.xfer_cache_shape(t, h, d, blocks)


def test_block_bytes():
    n = C.c_size_t()
    for t in (16, 32, 64):
        for h in (1, 3, 16, 17, 1024):
            for d in (64, 96, 128, 192, 256):
                assert X.lib().xfer_cache_block_bytes(C.byref(_shape(t, h, d)), C.byref(n)) == 0
                assert n.value == R.block_bytes(t, h, d) and n.value % 128 == 0


BAD_SHAPES = [(8, 2, 128, 10), (48, 2, 128, 10), (128, 2, 128, 10), (0, 2, 128, 10),
              (16, 0, 128, 10), (16, 1025, 128, 10), (16, -1, 128, 10), (16, 2, 80, 10),
              (16, 2, 0, 10), (16, 2, 512, 10), (16, 2, 128, 0), (16, 2, 128, -4),
              (16, 2, 128, 1 << 27), (64, 2, 128, 1 << 25)]


@pytest.mark.parametrize("shape", BAD_SHAPES)
def test_shapes_are_refused(shape):
    L, g, n = X.lib(), C.byref(_shape(*shape)), C.c_size_t()
    assert L.xfer_cache_block_bytes(g, C.byref(n)) == INVALID
    assert L.xfer_cache_store(g, P, P, 1, 1, P, 1, 1, 0, P, 4, None) == INVALID
    a = _attend()
    assert L.xfer_cache_attend(g, P, C.byref(a), None) == INVALID
    assert L.xfer_cache_attend_workspace(g, C.byref(a), C.byref(n)) == INVALID
    with pytest.raises(xf.XferError):
        xf.PagedCache(shape[3], *shape[:3])
    assert L.xfer_cache_block_bytes(None, C.byref(n)) == INVALID


def _attend(**kw):
    a = X.xfer_attend(P, P, None, P, P, P, P, 1 << 40, 256, 128, 256, 128, 4, 2, 3, 2, 4, 0, 1.0, 0, 0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw", [dict(batch=-1), dict(rows=-1), dict(table_width=-1),
                                dict(table_stride=3), dict(heads=0), dict(heads=3),
                                dict(heads=1 << 17), dict(dtype=2), dict(dtype=-1),
                                dict(rows=1 << 29, heads=4), dict(batch=1 << 23), dict(workspace_bytes=0, table_width=1 << 20, table_stride=1 << 20),
                                dict(workspace=None, table_width=1 << 20, table_stride=1 << 20),
                                dict(workspace=P + 8, table_width=1 << 20, table_stride=1 << 20),
                                dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")),
                                dict(scale=float("nan")), dict(max_query=-1), dict(max_length=-1),
                                dict(query=None), dict(out=None), dict(table=None),
                                dict(lengths=None), dict(starts=None), dict(query=P + 1),
                                dict(out=P + 1), dict(lse=P + 2), dict(table=P + 2),
                                dict(lengths=P + 2), dict(starts=P + 2)])
def test_attend_refuses(kw):
    a = _attend(**kw)
    assert X.lib().xfer_cache_attend(C.byref(_shape()), P, C.byref(a), None) == INVALID
    assert xf.last_error().startswith("xfer_cache_attend")


def test_attend_refuses_the_rest():
    L, g = X.lib(), C.byref(_shape())
    assert L.xfer_cache_attend(g, None, C.byref(_attend()), None) == INVALID
    assert L.xfer_cache_attend(g, P + 8, C.byref(_attend()), None) == INVALID
    assert L.xfer_cache_attend(g, P, None, None) == INVALID
    assert L.xfer_cache_attend_workspace(g, C.byref(_attend()), None) == INVALID
    # nothing to compute: nothing is touched
    assert L.xfer_cache_attend(g, None, C.byref(_attend(rows=0, query=None)), None) == 0
    assert L.xfer_cache_attend(g, None, C.byref(_attend(batch=0)), None) == 0


@pytest.mark.parametrize("i,bad", [(1, None), (1, P + 4), (2, None), (2, P + 1), (5, None),
                                   (5, P + 1), (8, 3), (8, -1), (9, None), (9, P + 2), (10, -1)])
def test_store_refuses(i, bad):
    args = [C.byref(_shape()), P, P, 256, 128, P, 256, 128, 0, P, 4, None]
    args[i] = bad
    assert X.lib().xfer_cache_store(*args) == INVALID
    assert xf.last_error().startswith("xfer_cache_store")


def test_store_refuses_too_many_workgroups():
    args = [C.byref(_shape(h=1024)), P, P, 256, 128, P, 256, 128, 0, P, 1 << 30, None]
    assert X.lib().xfer_cache_store(*args) == INVALID and "too many" in xf.last_error()


def test_store_of_nothing():
    assert X.lib().xfer_cache_store(C.byref(_shape()), None, None, 0, 0, None, 0, 0, 1, None, 0,
                                    None) == 0


PLAN = [P, P, 3, P, 8, 8, P, 5, 16, P, P, 20, P, P, P, None]


@pytest.mark.parametrize("i,bad", [(0, None), (1, None), (2, -1), (3, None), (4, 7), (5, -1),
                                   (5, 9), (6, None), (7, -1), (8, 0), (8, 24), (9, None),
                                   (10, None), (11, -1), (12, None), (13, None), (14, None),
                                   (0, P + 2), (1, P + 1), (3, P + 2), (6, P + 2), (9, P + 2),
                                   (10, P + 2), (12, P + 2), (13, P + 2), (14, P + 2)])
def test_plan_refuses(i, bad):
    args = list(PLAN)
    args[i] = bad
    assert X.lib().xfer_cache_plan(*args) == INVALID
    assert xf.last_error().startswith("xfer_cache_plan")


def test_run_blocks_refuses_no_connection():
    assert X.lib().xfer_run_blocks(None, P, 1, P, 1, 16, P, P, 1, None) == INVALID


# ------------------------------------------------------------------- binding
class FakeTensor:
    """A tensor's attributes, as the checks read them, without a GPU."""

    def __init__(self, shape, dtype=torch.int32, device=0, strides=None, ptr=P, cuda=True):
        self.shape = torch.Size(shape)
        self.dtype = dtype
        self.device = torch.device("cuda", device)
        self.is_cuda = cuda
        self._ptr = ptr
        self._strides = strides or tuple(int(np.prod(shape[i + 1:])) for i in range(len(shape)))

    def data_ptr(self):
        return self._ptr

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        return self._strides if i is None else self._strides[i]

    def get_device(self):
        return self.device.index

    def numel(self):
        return int(np.prod(self.shape))

    def element_size(self):
        return torch.empty(0, dtype=self.dtype).element_size()

    def is_contiguous(self):
        return self._strides == tuple(int(np.prod(self.shape[i + 1:]))
                                      for i in range(len(self.shape)))


class Unreachable:
    def __getattr__(self, name):
        raise AssertionError("library called: " + name)


@pytest.fixture
def cache(monkeypatch):
    c = xf.PagedCache(10, 16, 2, 128, buffer=FakeTensor((10, R.block_bytes(16, 2, 128)), torch.uint8))
    monkeypatch.setattr(X, "_lib", Unreachable())
    return c


def test_buffer_is_checked():
    size = R.block_bytes(16, 2, 128)
    for bad, err in ((FakeTensor((10, size + 1), torch.uint8), ValueError),
                     (FakeTensor((9, size), torch.uint8), ValueError),
                     (FakeTensor((10, size), torch.int8), TypeError),
                     (FakeTensor((10, size), torch.uint8, ptr=P + 8), ValueError),
                     (FakeTensor((10, size), torch.uint8, strides=(size + 128, 1)), ValueError),
                     (torch.zeros(10, size, dtype=torch.uint8), ValueError)):
        with pytest.raises(err):
            xf.PagedCache(10, 16, 2, 128, buffer=bad)


BF = torch.bfloat16


@pytest.mark.parametrize("which,bad,err", [
    (0, FakeTensor((4, 2, 128), torch.float64), TypeError),
    (0, FakeTensor((4, 2, 64), BF), ValueError),
    (0, FakeTensor((4, 3, 128), BF), ValueError),
    (0, FakeTensor((4, 256), BF), ValueError),
    (0, FakeTensor((4, 2, 128), BF, strides=(256, 1, 2)), ValueError),
    (0, FakeTensor((4, 2, 128), BF, device=1), ValueError),
    (0, torch.zeros(4, 2, 128, dtype=BF), ValueError),
    (0, [1, 2], TypeError),
    (1, FakeTensor((4, 2, 128), torch.float16), TypeError),
    (1, FakeTensor((5, 2, 128), BF), ValueError),
    (2, FakeTensor((5,)), ValueError),
    (2, FakeTensor((4,), torch.int64), TypeError),
    (2, FakeTensor((4,), strides=(2,)), ValueError),
])
def test_store_arguments(cache, which, bad, err):
    args = [FakeTensor((4, 2, 128), BF), FakeTensor((4, 2, 128), BF), FakeTensor((4,))]
    args[which] = bad
    with pytest.raises(err):
        cache.store(*args)


@pytest.mark.parametrize("which,bad,err", [
    (0, FakeTensor((4, 4, 128), torch.float32), TypeError),
    (0, FakeTensor((4, 4, 64), BF), ValueError),
    (0, FakeTensor((4, 4, 128), BF, strides=(512, 1, 4)), ValueError),
    (0, FakeTensor((4, 4, 128), BF, device=1), ValueError),
    (1, FakeTensor((2, 8)), ValueError),
    (1, FakeTensor((3, 8), torch.int64), TypeError),
    (1, FakeTensor((3, 8), strides=(1, 3)), ValueError),
    (1, FakeTensor((3, 8), strides=(4, 1)), ValueError),
    (2, FakeTensor((3,), torch.int64), TypeError),
    (3, FakeTensor((3,)), ValueError),
    (3, FakeTensor((4,), strides=(0,)), ValueError),
])
def test_attend_arguments(cache, which, bad, err):
    args = [FakeTensor((4, 4, 128), BF), FakeTensor((3, 8)), FakeTensor((3,)), FakeTensor((4,))]
    args[which] = bad
    with pytest.raises(err):
        cache.attend(*args, out=FakeTensor((4, 4, 128), BF))


@pytest.mark.parametrize("kw,err", [
    (dict(out=FakeTensor((4, 4, 128), torch.float16)), TypeError),
    (dict(out=FakeTensor((4, 8, 128), BF)), ValueError),
    (dict(out=FakeTensor((4, 4, 128), BF, strides=(1, 4, 16))), ValueError),
    (dict(lse=FakeTensor((4, 4), torch.float16)), TypeError),
    (dict(lse=FakeTensor((4, 5), torch.float32)), ValueError),
    (dict(lse=FakeTensor((4, 4), torch.float32, strides=(1, 4))), ValueError),
])
def test_attend_outputs(cache, kw, err):
    args = [FakeTensor((4, 4, 128), BF), FakeTensor((3, 8)), FakeTensor((3,)), FakeTensor((4,))]
    with pytest.raises(err):
        cache.attend(*args, **dict(dict(out=FakeTensor((4, 4, 128), BF)), **kw))


@pytest.mark.parametrize("which,bad,err", [
    (0, torch.zeros(3, dtype=torch.int32), ValueError),
    (0, FakeTensor((3,), torch.int64), TypeError),
    (1, FakeTensor((4,)), ValueError),
    (2, FakeTensor((2, 8)), ValueError),
    (2, FakeTensor((3, 8), strides=(8, 2)), ValueError),
    (3, FakeTensor((5,), strides=(2,)), ValueError),
    (3, FakeTensor((5,), device=1), ValueError),
    (5, -1, ValueError),
])
def test_plan_arguments(cache, which, bad, err):
    args = [FakeTensor((3,)), FakeTensor((3,)), FakeTensor((3, 8)), FakeTensor((5,)), 16, 20]
    args[which] = bad
    sizes = (20, 20, 4, 3, 2)
    with pytest.raises(err):
        K.plan_blocks(*args, out=xf.BlockPlan(*(FakeTensor((n,)) for n in sizes)))


@pytest.mark.parametrize("i", range(5))
def test_plan_outputs(cache, i):
    sizes = [20, 20, 4, 3, 2]
    sizes[i] += 1
    with pytest.raises(ValueError):
        K.plan_blocks(FakeTensor((3,)), FakeTensor((3,)), FakeTensor((3, 8)), FakeTensor((5,)), 16, 20,
                      out=xf.BlockPlan(*(FakeTensor((n,)) for n in sizes)))


def test_send_and_run_blocks_arguments(cache):
    conn = X.Conn("simple", 1, 8, 4096, _handle=0x1234)
    conn.device = 0
    try:
        other = xf.PagedCache.__new__(xf.PagedCache)
        other.__dict__.update(cache.__dict__, kv_heads=4)
        with pytest.raises(ValueError, match="cannot go"):
            cache.send(conn, other, FakeTensor((3,)), FakeTensor((3,)))
        for ids in ((FakeTensor((3,)), FakeTensor((4,))), (torch.zeros(3, dtype=torch.int32), FakeTensor((3,))),
                    (FakeTensor((3,), strides=(2,)), FakeTensor((3,))), (FakeTensor((3,), device=1), FakeTensor((3,)))):
            with pytest.raises(ValueError):
                cache.send(conn, cache, *ids)
        with pytest.raises(TypeError):
            cache.send(conn, cache, FakeTensor((3,)), FakeTensor((3,), torch.int64))
        conn.device = 1
        with pytest.raises(ValueError, match="cuda:1"):
            cache.send(conn, cache, FakeTensor((3,)), FakeTensor((3,)))
        conn.device = 0
        pool = FakeTensor((10, 4096), torch.uint8)
        with pytest.raises(ValueError, match="ids"):
            conn.run_blocks(pool, pool, 4096, FakeTensor((3,)), FakeTensor((4,)))
        with pytest.raises(TypeError, match="int32"):
            conn.run_blocks(pool, pool, 4096, FakeTensor((3,), torch.int64), FakeTensor((6,)))
        with pytest.raises(ValueError, match="count"):
            conn.run_blocks(P, pool, 4096, FakeTensor((3,)), FakeTensor((3,)))
        with pytest.raises(ValueError, match="positive"):
            conn.run_blocks(pool, pool, 0, FakeTensor((3,)), FakeTensor((3,)))
        with pytest.raises(ValueError, match="holds"):
            conn.run_blocks(pool, pool, 4096, FakeTensor((3,)), FakeTensor((3,)), src_blocks=11)
        with pytest.raises(ValueError, match="not in GPU"):
            conn.run_blocks(pool, torch.zeros(10, 4096, dtype=torch.uint8), 4096, FakeTensor((3,)),
                            FakeTensor((3,)))
        with pytest.raises(ValueError, match="negative"):
            conn.run_blocks(pool, P, 4096, FakeTensor((3,)), FakeTensor((3,)), dst_blocks=-1)
    finally:
        conn._h = None


# ------------------------------------------------------------ the plain forms
def test_plain_e4m3_rounding():
    """The tests' own rounding against torch's conversion, over every float16."""
    x = np.arange(1 << 16, dtype=np.uint16).view(np.float16).astype(np.float64)
    x = x[np.abs(x) <= 448]
    want = torch.tensor(x).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(R.to_codes(x), want)
    assert np.array_equal(R.VALUES[~np.isnan(R.VALUES)],
                          torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
                          .numpy()[~np.isnan(R.VALUES)])
