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
