"""CPU tests of where the cache's operators take memory from: with `stream=` on
another stream than the current one, what a call allocates must come from that
stream's pool.  The current stream's pool may hand out memory that was just freed
there and that kernels still queued on it use, which the launch on the other
stream would not wait for.  Results stay reserved for the current stream too."""
import pytest
import torch

import cache_ref as R
import recv_fifo_plane_amd as xf
from recv_fifo_plane_amd import cache as K
from recv_fifo_plane_amd import xfer as X
from test_cache_refusals import BF, FakeTensor

WORK = 4096  # bytes of workspace that the library asks for


class FakeStream:
    def __init__(self, handle, device=0):
        self.cuda_stream, self.device = handle, torch.device("cuda", device)

    def __eq__(self, other):
        return (self.cuda_stream, self.device) == (other.cuda_stream, other.device)

    __hash__ = None


class Allocated(FakeTensor):
    """A tensor that a call has made: the stream whose pool it came from, and
    those it was recorded on."""

    def __init__(self, shape, dtype, device, pool):
        super().__init__(shape, dtype, device=device)
        self.pool, self.recorded = pool, []

    def record_stream(self, stream):
        self.recorded.append(stream.cuda_stream)

    def split_with_sizes(self, sizes):
        return [FakeTensor((n,)) for n in sizes]


class World:
    """torch.cuda's streams of two devices, and the library, for one call."""

    def __init__(self, monkeypatch):
        self.device, self.made, self.launched = 0, [], []
        self.current = {0: FakeStream(0x10), 1: FakeStream(0x20, 1)}
        world = self

        class Use:
            def __init__(self, stream):
                self.stream = stream

            def __enter__(self):
                self.was = world.device, dict(world.current)
                world.device = self.stream.device.index
                world.current[world.device] = self.stream

            def __exit__(self, *_):
                world.device, world.current = self.was

        class Device(Use):
            def __init__(self, index):
                super().__init__(world.current[index])

        def new_empty(t, shape, dtype=None):
            shape = (shape,) if isinstance(shape, int) else tuple(shape)
            got = Allocated(shape, dtype or t.dtype, t.device.index,
                            world.current[t.device.index].cuda_stream)
            world.made.append(got)
            return got

        monkeypatch.setattr(FakeTensor, "new_empty", new_empty, raising=False)
        K._kinds()
        monkeypatch.setattr(K, "_RAW", lambda index: world.current[index].cuda_stream)
        number = lambda d: world.device if d is None else torch.device("cuda", d).index  # noqa: E731
        for name, fn in (("current_device", lambda: world.device),
                         ("is_initialized", lambda: False),
                         ("current_stream", lambda d=None: world.current[number(d)]),
                         ("default_stream", lambda d=None: FakeStream(0, number(d))),
                         ("ExternalStream", lambda h, device=None: FakeStream(h, number(device))),
                         ("Stream", FakeStream), ("stream", Use), ("device", Device)):
            monkeypatch.setattr(torch.cuda, name, fn)

        class Library:
            def xfer_cache_attend_workspace(self, shape, args, n):
                n._obj.value = WORK
                return 0

            def xfer_cache_plan(self, *args):
                world.launched.append((world.device, args[-1]))
                return 0

            xfer_cache_store = xfer_cache_plan

            def xfer_cache_attend(self, shape, base, args, stream):
                world.work = args._obj.workspace, args._obj.workspace_bytes
                world.launched.append((world.device, stream))
                return 0
        monkeypatch.setattr(X, "_lib", Library())


@pytest.fixture
def world(monkeypatch):
    # (made with the library itself: the shape's block size is its answer)
    caches = [xf.PagedCache(10, 16, 2, 128, buffer=FakeTensor((10, R.block_bytes(16, 2, 128)),
                                                              torch.uint8, device=d)) for d in (0, 1)]
    w = World(monkeypatch)
    w.caches = caches
    return w


def attend(world, device=0, **kw):
    on = lambda shape, dtype=torch.int32: FakeTensor(shape, dtype, device=device)  # noqa: E731
    return world.caches[device].attend(on((4, 4, 128), BF), on((3, 8)), on((3,)), on((4,)), lse=True,
                                       **kw)


def plan(world, device=0, **kw):
    on = lambda shape: FakeTensor(shape, device=device)  # noqa: E731
    return K.plan_blocks(on((3,)), on((3,)), on((3, 8)), on((5,)), 16, 20, **kw)


OTHER = [(FakeStream(0x77), 0x77), (0x77, 0x77), (0, None)]


@pytest.mark.parametrize("stream,handle", OTHER)
def test_attend_allocates_on_the_launch_stream(world, stream, handle):
    out, lse = attend(world, stream=stream)
    assert world.launched == [(0, handle)]
    assert len(world.made) == 3 and all(t.pool == (handle or 0) for t in world.made)
    work = world.made[-1]
    assert work.shape == (WORK,) and world.work == (work.data_ptr(), WORK)
    assert out.recorded == lse.recorded == [0x10]  # results are used on the current stream
    assert world.device == 0 and world.current[0].cuda_stream == 0x10


@pytest.mark.parametrize("stream,handle", OTHER)
def test_plan_allocates_on_the_launch_stream(world, stream, handle):
    plan(world, stream=stream)
    assert world.launched == [(0, handle)]
    assert [t.pool for t in world.made] == [handle or 0]
    assert world.made[0].recorded == [0x10]


@pytest.mark.parametrize("stream", [None, FakeStream(0x10), 0x10])
def test_the_current_stream_is_used_as_it_is(world, stream):
    attend(world, stream=stream)
    plan(world, stream=stream)
    assert world.launched == [(0, 0x10)] * 2
    assert all(t.pool == 0x10 and t.recorded == [] for t in world.made)


def test_a_handle_is_of_the_tensors_device(world):
    """The current device is 0, the tensors' 1: a raw handle is one of device 1."""
    attend(world, device=1, stream=0x88)
    plan(world, device=1, stream=0x88)
    assert world.launched == [(1, 0x88)] * 2
    assert all(t.pool == 0x88 for t in world.made)
    assert world.made[0].recorded == [0x20] and world.made[2].recorded == []
    attend(world, device=1)
    assert world.launched[-1] == (1, 0x20)


def test_a_stream_of_another_device_is_refused(world):
    for call in (attend, plan):
        with pytest.raises(ValueError, match="stream"):
            call(world, stream=FakeStream(0x77, 1))
    sizes = (20, 20, 4, 3, 2)
    with pytest.raises(ValueError, match="stream"):
        plan(world, out=xf.BlockPlan(*(FakeTensor((n,)) for n in sizes)), stream=FakeStream(0x77, 1))
    with pytest.raises(ValueError, match="stream"):
        world.caches[0].store(FakeTensor((4, 2, 128), BF), FakeTensor((4, 2, 128), BF),
                              FakeTensor((4,)), stream=FakeStream(0x77, 1))
    assert not world.launched and not world.made


def test_outputs_of_the_caller_allocate_nothing_else(world):
    sizes = (20, 20, 4, 3, 2)
    plan(world, out=xf.BlockPlan(*(FakeTensor((n,)) for n in sizes)), stream=0x77)
    assert not world.made and world.launched == [(0, 0x77)]
    world.caches[0].attend(FakeTensor((4, 4, 128), BF), FakeTensor((3, 8)), FakeTensor((3,)),
                           FakeTensor((4,)), out=FakeTensor((4, 4, 128), BF), stream=0x77)
    assert [t.pool for t in world.made] == [0x77]  # the workspace
