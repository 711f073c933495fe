"""CPU tests of the argument checks of the 4-bit cache and of reading a cache back: a
call outside the documented domain is refused before anything is launched."""
import ctypes as C

import pytest
import torch

import mxcache_ref as R
import recv_fifo_plane_amd as xf
from recv_fifo_plane_amd import xfer as X
from test_cache_refusals import BAD_SHAPES, BF, FakeTensor, INVALID, P, Unreachable, _attend, _shape


def test_block_bytes():
    n = C.c_size_t()
    for t in (16, 32, 64):
        for h in (1, 3, 16, 17, 1024):
            for d in (64, 96, 128, 192, 256):
                assert X.lib().xfer_mxcache_block_bytes(C.byref(_shape(t, h, d)), C.byref(n)) == 0
                assert n.value == R.block_bytes(t, h, d) and n.value % 128 == 0


def _load(**kw):
    a = X.xfer_load(P, P, P, P, P, 256, 128, 256, 128, 4, 2, 3, 4, 0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("shape", BAD_SHAPES)
def test_shapes_are_refused(shape):
    L, g, n = X.lib(), C.byref(_shape(*shape)), C.c_size_t()
    assert L.xfer_mxcache_block_bytes(g, C.byref(n)) == INVALID
    assert L.xfer_mxcache_store(g, P, P, 1, 1, P, 1, 1, 0, P, 4, None) == INVALID
    assert L.xfer_mxcache_load(g, P, C.byref(_load()), None) == INVALID
    assert L.xfer_cache_load(g, P, C.byref(_load()), None) == INVALID
    a = _attend()
    assert L.xfer_mxcache_attend(g, P, C.byref(a), None) == INVALID
    assert L.xfer_mxcache_attend_workspace(g, C.byref(a), C.byref(n)) == INVALID
    with pytest.raises(xf.XferError):
        xf.PagedCache(shape[3], *shape[:3], bits=4)
    assert L.xfer_mxcache_block_bytes(None, C.byref(n)) == INVALID
    assert L.xfer_mxcache_block_bytes(C.byref(_shape()), None) == INVALID


@pytest.mark.parametrize("kw", [dict(batch=-1), dict(rows=-1), dict(table_width=-1),
                                dict(table_stride=3), dict(heads=0), dict(heads=3),
                                dict(heads=1 << 17), dict(dtype=2), dict(dtype=-1),
                                dict(rows=1 << 29, heads=4), dict(batch=1 << 23),
                                dict(workspace_bytes=0, table_width=1 << 20, table_stride=1 << 20),
                                dict(workspace=None, table_width=1 << 20, table_stride=1 << 20),
                                dict(workspace=P + 8, table_width=1 << 20, table_stride=1 << 20),
                                dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")),
                                dict(scale=float("nan")), dict(max_query=-1), dict(max_length=-1),
                                dict(query=None), dict(out=None), dict(table=None),
                                dict(lengths=None), dict(starts=None), dict(query=P + 1),
                                dict(out=P + 1), dict(lse=P + 2), dict(table=P + 2),
                                dict(lengths=P + 2), dict(starts=P + 2), dict(out_head=127),
                                dict(out_row=128), dict(out_row=0)])
def test_attend_refuses(kw):
    assert X.lib().xfer_mxcache_attend(C.byref(_shape()), P, C.byref(_attend(**kw)), None) == INVALID
    assert xf.last_error().startswith("xfer_mxcache_attend")


def test_attend_refuses_the_rest():
    L, g = X.lib(), C.byref(_shape())
    assert L.xfer_mxcache_attend(g, None, C.byref(_attend()), None) == INVALID
    assert L.xfer_mxcache_attend(g, P + 8, C.byref(_attend()), None) == INVALID
    assert L.xfer_mxcache_attend(g, P, None, None) == INVALID
    assert L.xfer_mxcache_attend_workspace(g, C.byref(_attend()), None) == INVALID
    # nothing to compute: nothing is touched
    assert L.xfer_mxcache_attend(g, None, C.byref(_attend(rows=0, query=None)), None) == 0
    assert L.xfer_mxcache_attend(g, None, C.byref(_attend(batch=0)), None) == 0


@pytest.mark.parametrize("i,bad", [(1, None), (1, P + 4), (2, None), (2, P + 1), (5, None),
                                   (5, P + 1), (8, 3), (8, -1), (9, None), (9, P + 2), (10, -1)])
def test_store_refuses(i, bad):
    args = [C.byref(_shape()), P, P, 256, 128, P, 256, 128, 0, P, 4, None]
    args[i] = bad
    assert X.lib().xfer_mxcache_store(*args) == INVALID
    assert xf.last_error().startswith("xfer_mxcache_store")


def test_store_refuses_too_many_workgroups():
    args = [C.byref(_shape(h=1024, d=256)), P, P, 256, 128, P, 256, 128, 0, P, (1 << 31) - 1, None]
    assert X.lib().xfer_mxcache_store(*args) == INVALID and "too many" in xf.last_error()


def test_store_of_nothing():
    assert X.lib().xfer_mxcache_store(C.byref(_shape()), None, None, 0, 0, None, 0, 0, 1, None, 0,
                                      None) == 0


@pytest.mark.parametrize("name", ["xfer_cache_load", "xfer_mxcache_load"])
@pytest.mark.parametrize("kw", [dict(batch=-1), dict(rows=-1), dict(table_width=-1),
                                dict(table_stride=3), dict(batch=1 << 27), dict(dtype=3),
                                dict(dtype=-1), dict(key=None), dict(value=None), dict(table=None),
                                dict(lengths=None), dict(starts=None), dict(key=P + 1),
                                dict(value=P + 1), dict(value=P + 2, dtype=2), dict(table=P + 2),
                                dict(lengths=P + 1), dict(starts=P + 2), dict(key_head=64),
                                dict(key_row=128), dict(value_row=0), dict(value_head=-127)])
def test_load_refuses(name, kw):
    L, g = X.lib(), C.byref(_shape())
    assert getattr(L, name)(g, P, C.byref(_load(**kw)), None) == INVALID
    assert xf.last_error().startswith(name)


@pytest.mark.parametrize("name", ["xfer_cache_load", "xfer_mxcache_load"])
def test_load_refuses_the_rest(name):
    fn, g = getattr(X.lib(), name), C.byref(_shape())
    assert fn(g, None, C.byref(_load()), None) == INVALID
    assert fn(g, P + 8, C.byref(_load()), None) == INVALID
    assert fn(g, P, None, None) == INVALID
    assert fn(g, None, C.byref(_load(rows=0, key=None)), None) == 0
    assert fn(g, None, C.byref(_load(batch=0)), None) == 0


# ------------------------------------------------------------------- binding
def make(bits=4):
    size = {4: R.block_bytes(16, 2, 128), 8: 8192 + 128}[bits]
    return xf.PagedCache(10, 16, 2, 128, buffer=FakeTensor((10, size), torch.uint8), bits=bits)


@pytest.fixture
def cache(monkeypatch):
    c = make()
    monkeypatch.setattr(X, "_lib", Unreachable())
    return c


@pytest.mark.parametrize("bits", [0, 2, 16, -4, "4", None, 4.5])
def test_bits_are_checked(bits):
    with pytest.raises(ValueError, match="bits"):
        xf.PagedCache(10, 16, 2, 128, buffer=FakeTensor((10, 128), torch.uint8), bits=bits)


def test_buffer_is_checked():
    size = R.block_bytes(16, 2, 128)
    for bad, err in ((FakeTensor((10, size + 1), torch.uint8), ValueError),
                     (FakeTensor((10, 8192 + 128), torch.uint8), ValueError),
                     (FakeTensor((10, size), torch.uint8, ptr=P + 8), ValueError)):
        with pytest.raises(err):
            xf.PagedCache(10, 16, 2, 128, buffer=bad, bits=4)


@pytest.mark.parametrize("view", ["keys", "values", "scales"])
def test_views_of_shared_bytes_are_refused(cache, view):
    with pytest.raises(ValueError, match="load"):
        getattr(cache, view)()


def test_send_between_forms_is_refused(cache):
    with pytest.raises(ValueError, match="bits"):
        other = xf.PagedCache.__new__(xf.PagedCache)
        other.__dict__.update(cache.__dict__, bits=8)
        cache.send(None, other, FakeTensor((3,)), FakeTensor((3,)))


@pytest.mark.parametrize("which,bad,err", [
    (0, FakeTensor((4, 2, 128), torch.float64), TypeError),
    (0, FakeTensor((4, 2, 64), BF), ValueError),
    (1, FakeTensor((4, 2, 128), torch.float16), TypeError),
    (2, FakeTensor((4,), torch.int64), TypeError),
])
def test_store_arguments(cache, which, bad, err):
    args = [FakeTensor((4, 2, 128), BF), FakeTensor((4, 2, 128), BF), FakeTensor((4,))]
    args[which] = bad
    with pytest.raises(err):
        cache.store(*args)


OUT = (FakeTensor((6, 2, 128), BF), FakeTensor((6, 2, 128), BF))


@pytest.mark.parametrize("which,bad,err", [
    (0, FakeTensor((2, 8)), ValueError),
    (0, FakeTensor((3, 8), torch.int64), TypeError),
    (0, FakeTensor((3, 8), strides=(4, 1)), ValueError),
    (0, FakeTensor((3, 8), device=1), ValueError),
    (1, FakeTensor((3,), torch.int64), TypeError),
    (1, torch.zeros(3, dtype=torch.int32), ValueError),
    (2, FakeTensor((3,)), ValueError),
    (2, FakeTensor((4,), strides=(0,)), ValueError),
    (3, -1, ValueError),
    (3, 1 << 31, ValueError),
    (3, 7, ValueError),
])
def test_load_arguments(cache, which, bad, err):
    args = [FakeTensor((3, 8)), FakeTensor((3,)), FakeTensor((4,)), 6]
    args[which] = bad
    with pytest.raises(err):
        cache.load(*args, out=OUT)


@pytest.mark.parametrize("kw,err", [
    (dict(dtype=torch.float64), TypeError),
    (dict(dtype=torch.int32), TypeError),
    (dict(dtype="bf16"), TypeError),
    (dict(out=(OUT[0],)), ValueError),
    (dict(out=(OUT[0], FakeTensor((6, 2, 128), torch.float16))), TypeError),
    (dict(out=(OUT[0], FakeTensor((5, 2, 128), BF))), ValueError),
    (dict(out=(FakeTensor((6, 2, 128), torch.int8),) * 2), TypeError),
    (dict(out=(FakeTensor((6, 2, 128), BF, strides=(1, 6, 12)), OUT[1])), ValueError),
    (dict(out=OUT, dtype=torch.float16), TypeError),
    (dict(out=(OUT[0], FakeTensor((6, 2, 128), BF, device=1))), ValueError),
])
def test_load_outputs(cache, kw, err):
    with pytest.raises(err):
        cache.load(FakeTensor((3, 8)), FakeTensor((3,)), FakeTensor((4,)), 6, **kw)


def test_load_refuses_a_recorded_gradient(cache):
    out = (FakeTensor((6, 2, 128), BF), FakeTensor((6, 2, 128), BF))
    out[1].requires_grad = True
    with pytest.raises(ValueError, match="gradient"):
        cache.load(FakeTensor((3, 8)), FakeTensor((3,)), FakeTensor((4,)), 6, out=out)


def test_calls_go_to_the_functions_of_their_form(monkeypatch):
    """The same calls reach xfer_cache_* with 8 bits and xfer_mxcache_* with 4."""
    called = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: called.append(name) or 0

    caches = {bits: make(bits) for bits in (8, 4)}
    monkeypatch.setattr(X, "_lib", Lib())
    monkeypatch.setattr(X, "_stream_handle", lambda s: s)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    from recv_fifo_plane_amd import cache as K
    K._kinds()
    monkeypatch.setattr(K, "_RAW", None)
    for bits, kind in ((8, "cache"), (4, "mxcache")):
        c, called[:] = caches[bits], []
        rows = FakeTensor((4, 2, 128), BF)
        c.store(rows, rows, FakeTensor((4,)))
        c.load(FakeTensor((3, 8)), FakeTensor((3,)), FakeTensor((4,)), 6, out=OUT)
        c.attend(FakeTensor((4, 4, 128), BF), FakeTensor((3, 8)), FakeTensor((3,)), FakeTensor((4,)),
                 out=FakeTensor((4, 4, 128), BF))
        assert called == ["xfer_%s_%s" % (kind, x) for x in ("store", "load", "attend_workspace", "attend")]
