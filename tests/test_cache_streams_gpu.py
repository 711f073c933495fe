"""GPU tests of `stream=`: calls on the current stream and on others, queued
without a synchronisation between them, give what each gives alone."""
import pytest

from test_cache_gpu import gpu_cache, ints, new_pool

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def xf():
    import recv_fifo_plane_amd
    return recv_fifo_plane_amd


def test_attend_on_the_current_stream_then_on_another():
    """Shared work, so every call has a workspace, freed on its return while
    its kernels are still queued."""
    T, H, D, B = 16, 2, 128, 2
    cache = gpu_cache(new_pool(700, T, H, D, 1))
    table = ints(range(600)).reshape(B, 300)
    args = [(torch.randn(B, 8, D, device="cuda").to(torch.bfloat16), table, ints(lens), ints([0, 1, 2]))
            for lens in ([4700, 3100], [4100, 4799], [2600, 17])]
    want = [cache.attend(*a, lse=True) for a in args]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        got = []
        for _ in range(10):
            for i, s in ((0, None), (1, stream), (2, None), (0, stream), (1, None), (2, stream)):
                got.append((i, cache.attend(*args[i], lse=True, stream=s)))
        torch.cuda.synchronize()
        for i, res in got:
            assert torch.equal(res[0], want[i][0]) and torch.equal(res[1], want[i][1])


def test_results_of_another_stream_are_used_and_dropped():
    """A result made on another stream, read on the current one and dropped there,
    is not overwritten by the other stream's next call."""
    T, H, D, B = 16, 2, 128, 2
    cache = gpu_cache(new_pool(700, T, H, D, 1))
    table, starts = ints(range(600)).reshape(B, 300), ints([0, 1, 2])
    lens = [ints(x) for x in ([4700, 3100], [4100, 4799], [2600, 17])]
    q = torch.randn(B, 8, D, device="cuda").to(torch.bfloat16)
    want = [cache.attend(q, table, x, starts).clone() for x in lens]
    side, here = torch.cuda.Stream(), torch.cuda.current_stream()
    busy = torch.randn(2048, 2048, device="cuda")
    torch.cuda.synchronize()
    got = []
    for n in range(12):
        out = cache.attend(q, table, lens[n % 3], starts, stream=side)
        here.wait_stream(side)
        busy @ busy  # the current stream lags behind the other
        got.append(out.clone())
        del out
    torch.cuda.synchronize()
    for n, x in enumerate(got):
        assert torch.equal(x, want[n % 3]), n


def test_plans_on_the_current_stream_then_on_another():
    T, B = 16, 500
    free = ints(range(40000))
    sets = []
    for k in range(3):
        cached, added = ints([(7 * i + k) % 90 for i in range(B)]), ints([(5 * i + k) % 40 for i in range(B)])
        sets.append((cached, added, int(added.sum())))
    tables = [[ints([-1] * (B * 12)).reshape(B, 12) for _ in range(3)] for _ in range(2)]
    for t in tables[0] + tables[1]:
        t.copy_(ints(range(B * 12)).reshape(B, 12) + 50000)
    want = [[x.clone() for x in xf().plan_blocks(c, a, tables[0][i], free, T, n)]
            for i, (c, a, n) in enumerate(sets)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for i, s in ((0, None), (1, side), (2, None)):
            c, a, n = sets[i]
            got.append((i, xf().plan_blocks(c, a, tables[1][i], free, T, n, stream=s)))
    torch.cuda.synchronize()
    for i, res in got:
        assert all(torch.equal(x, y) for x, y in zip(res, want[i]))
