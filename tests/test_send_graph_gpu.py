"""GPU test of a hand-over in a captured graph: sends replayed on the stream that
the connection runs on, with eager ones and synchronisations between."""
import numpy as np
import pytest

from test_cache_gpu import ints

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("proto", ["zcd", "simple"])
def test_sends_replayed(proto):
    import recv_fifo_plane_amd as xf
    T, H, D, blocks, n = 16, 2, 128, 60, 21
    here, there = (xf.PagedCache(blocks, T, H, D) for _ in range(2))
    rng = np.random.default_rng(1)
    src, dst = ints([0] * n), ints(range(n))
    stream = torch.cuda.Stream()
    conn = xf.Conn(proto, 4, 2, 16384, wgs_per_channel=2, timeout_ms=20000)
    with torch.cuda.stream(stream):
        here.send(conn, there, src, dst)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            here.send(conn, there, src, dst)
        for it in range(6):
            here.buffer.random_(0, 256)
            there.buffer.zero_()
            src.copy_(ints(rng.permutation(blocks)[:n]))
            dst.copy_(ints(rng.permutation(blocks)[:n]))
            graph.replay()
            torch.cuda.synchronize()
            want = torch.zeros_like(there.buffer)
            want[dst.long()] = here.buffer[src.long()]
            assert torch.equal(there.buffer, want), it
            if it % 2:  # an eager one
                there.buffer.zero_()
                here.send(conn, there, src, dst)
                torch.cuda.synchronize()
                assert torch.equal(there.buffer, want), it
        state = conn.query(0)
    assert state["error"] == 0
    torch.cuda.synchronize()
    conn.close()


@pytest.mark.parametrize("fifo,jitter", [("relay", 0), ("device", 5)])
def test_sends_that_cannot_be_replayed_are_not_captured(fifo, jitter):
    """A replay would wait for proxies that were told of one transfer, or repeat the
    number of a debug launch."""
    import recv_fifo_plane_amd as xf
    here, there = (xf.PagedCache(8, 16, 2, 64) for _ in range(2))
    here.buffer.random_(0, 256)
    ids = ints(range(8))
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    conn = xf.Conn("simple", 2, 2, 4096, fifo, wgs_per_channel=2, timeout_ms=2000)
    conn.set_jitter(jitter)
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        here.send(conn, there, ids, ids)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            with pytest.raises(xf.XferError, match="relay"):
                here.send(conn, there, ids, ids)
            there.buffer.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert not there.buffer.any()
        here.send(conn, there, ids, ids)
        torch.cuda.synchronize()
    assert torch.equal(here.buffer, there.buffer) and conn.query(0)["error"] == 0
    conn.close()
