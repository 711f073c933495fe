"""GPU tests of the paged cache's operators as a program uses them: one endpoint
plans, stores and sends, the other attends; eagerly, in captured graphs, on
streams of their own and beyond 4 GiB."""
import math

import numpy as np
import pytest

import cache_ref as R
from test_cache_gpu import dev, gpu_cache, ints, new_pool

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def xf():
    import recv_fifo_plane_amd
    return recv_fifo_plane_amd


class Answers:
    """Requests that the prompt endpoint hands to the answering endpoint, kept in
    64 bits beside the operators."""

    def __init__(self, T=16, H=2, group=4, D=128, blocks=120, seed=0, proto="zcd"):
        self.T, self.H, self.group, self.D, self.blocks = T, H, group, D, blocks
        self.rng = np.random.default_rng(seed)
        self.here, self.there = (xf().PagedCache(blocks, T, H, D) for _ in range(2))
        self.ref = R.Cache(np.zeros((blocks, R.block_bytes(T, H, D)), np.uint8), T, H, D)
        self.ref_there = R.Cache(np.zeros((blocks, R.block_bytes(T, H, D)), np.uint8), T, H, D)
        self.conn = xf().Conn(proto, 4, 2, 16384, wgs_per_channel=2, timeout_ms=20000)

    def rows(self, n):
        g = torch.Generator().manual_seed(int(self.rng.integers(1 << 30)))
        make = lambda h: torch.randn(n, h, self.D, generator=g).to(torch.bfloat16)  # noqa: E731
        return make(self.H), make(self.H), make(self.H * self.group)

    def check(self, out, lse, q, table, lengths, starts):
        sc = 1 / math.sqrt(self.D)
        want = R.attend(self.ref_there, q.double().numpy(), table, lengths, starts, sc)
        tol, tol_lse = R.attend_bounds(want, max(lengths), self.D, 2.0 ** -8)
        n = starts[-1]
        assert np.all(np.abs(out.double().cpu().numpy() - want[0])[:n] <= tol[:n])
        assert np.all(np.abs(lse.double().cpu().numpy() - want[1])[:n] <= tol_lse[:n])


@pytest.mark.parametrize("proto", ["zcd", "simple"])
@pytest.mark.parametrize("T,H,group,D", [(16, 2, 4, 128), (64, 3, 1, 64), (32, 1, 7, 256)])
def test_prompt_handed_over_then_answered(T, H, group, D, proto):
    a = Answers(T, H, group, D, proto=proto)
    lens = [100, 1, 37, 64]
    B, width = len(lens), 12
    free = a.rng.permutation(a.blocks)
    table = ints(np.full(B * width, -1)).reshape(B, width)
    # the prompt endpoint
    n = sum(lens)
    plan = xf().plan_blocks(ints([0] * B), ints(lens), table, ints(free), T, n)
    key, value, _ = a.rows(n)
    a.here.store(key.cuda(), value.cuda(), plan.slots)
    slots, _, _, _, _, want_table = R.plan([0] * B, lens, [[-1] * width] * B, free.tolist(), T, n)
    R.store(a.ref, key.double().numpy(), value.double().numpy(), slots)
    # its blocks, as a padded list on the GPU, into blocks of the answering endpoint
    src = np.array(want_table).reshape(-1)
    there = a.rng.permutation(a.blocks)[:src.size]
    dst = np.where(src >= 0, there, -1)
    a.here.send(a.conn, a.there, table.reshape(-1), ints(dst))
    for s, d in zip(src[src >= 0], dst[src >= 0]):
        a.ref_there.k[d], a.ref_there.v[d], a.ref_there.s[d] = a.ref.k[s], a.ref.v[s], a.ref.s[s]
    # the answering endpoint: a token at a time, then three drafted ones
    t2 = ints(dst).reshape(B, width)
    used = set(dst.tolist())
    free2 = [b for b in range(a.blocks) if b not in used]
    host_table, cached = dst.reshape(B, width).tolist(), list(lens)
    for step in (1, 1, 3, 1):
        added = [step] * B
        n = step * B
        plan = xf().plan_blocks(ints(cached), ints(added), t2, ints(free2), T, n + 2)
        slots, _, starts, lengths, counts, host_table = R.plan(cached, added, host_table, free2, T, n + 2)
        assert plan.slots.tolist() == slots and plan.counts.tolist() == counts
        key, value, q = a.rows(n + 2)
        a.there.store(key.cuda(), value.cuda(), plan.slots)
        R.store(a.ref_there, key.double().numpy(), value.double().numpy(), slots)
        out, lse = a.there.attend(q.cuda(), t2, plan.lengths, plan.starts, lse=True)
        a.check(out, lse, q, host_table, lengths, starts)
        free2 = free2[counts[0]:]
        cached = lengths
    torch.cuda.synchronize()
    assert a.conn.query(0)["error"] == 0
    a.conn.close()


def test_decode_step_in_graphs():
    """Plan, store and attend captured twice (two graphs alive, each with its own
    buffers), replayed in turn with eager calls between; each replay is the eager
    result."""
    T, H, group, D, B, width = 16, 2, 4, 128, 3, 300
    ref = new_pool(1000, T, H, D, 1)
    pool = dev(ref.raw())
    free = ints(np.arange(900, 950))
    stage = [dict(cached=ints([0] * B), added=ints([1] * B), table=ints(np.arange(B * width)).reshape(B, width),
                  key=torch.zeros(B, H, D, dtype=torch.bfloat16, device="cuda"),
                  value=torch.zeros(B, H, D, dtype=torch.bfloat16, device="cuda"),
                  query=torch.zeros(B, H * group, D, dtype=torch.bfloat16, device="cuda"),
                  cache=xf().PagedCache(1000, T, H, D, buffer=pool.clone())) for _ in range(3)]

    def step(s):
        plan = xf().plan_blocks(s["cached"], s["added"], s["table"], free, T, B)
        s["cache"].store(s["key"], s["value"], plan.slots)
        return s["cache"].attend(s["query"], s["table"], plan.lengths, plan.starts, max_query=1,
                                 max_length=4800, lse=True)

    graphs = []
    for s in stage[:2]:
        step(s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = step(s)
        graphs.append((g, res))
    eager = stage[2]
    torch.cuda.synchronize()
    for s in stage:
        s["cache"].buffer.copy_(pool)
    rng = np.random.default_rng(0)
    for it in range(6):
        lens = rng.integers(0, 4790, B)
        lens[it % B] = it  # short ones too
        g0 = torch.Generator(device="cuda").manual_seed(it)
        new = [torch.randn(x.shape, generator=g0, device="cuda").to(torch.bfloat16)
               for x in (eager["key"], eager["value"], eager["query"])]
        for s in stage:
            s["cached"].copy_(ints(lens))
            s["table"].copy_(ints(np.arange(B * width)).reshape(B, width))
            for x, y in zip((s["key"], s["value"], s["query"]), new):
                x.copy_(y)
        want = step(eager)
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for (g, res), s in zip(graphs, stage):
            assert torch.equal(res[0], want[0]) and torch.equal(res[1], want[1]), it
            assert torch.equal(s["cache"].buffer, eager["cache"].buffer), it


def test_other_streams():
    """Two streams at once, each with its own cache: results are those of one stream."""
    T, H, D, B = 16, 2, 128, 2
    ref = new_pool(700, T, H, D, 1)
    want = []
    streams = [torch.cuda.Stream() for _ in range(2)]
    q = torch.randn(B, 8, D, device="cuda").to(torch.bfloat16)
    kv = torch.randn(2, 40, H, D, device="cuda").to(torch.bfloat16)
    table, lens, starts = ints(np.arange(600)).reshape(B, 300), ints([4700, 3100]), ints([0, 1, 2])
    slots = ints(list(range(16 * 650, 16 * 650 + 40)))
    cached, added, free = ints([20, 0]), ints([3, 37]), ints(range(690, 700))
    tables = [ints([680, 681, -1, -1, -1, -1, -1, -1]).reshape(2, 4) for _ in range(3)]
    caches = [gpu_cache(ref) for _ in range(3)]
    torch.cuda.synchronize()

    def work(i, stream):
        plan = xf().plan_blocks(cached, added, tables[i], free, T, 45, stream=stream)
        caches[i].store(kv[0], kv[1], slots, stream=stream)
        out, lse = caches[i].attend(q, table, lens, starts, lse=True, stream=stream)
        return list(plan) + [out, lse]
    for rep in range(3):
        got = [work(i, s) for i, s in enumerate(streams)]
        torch.cuda.synchronize()
        want = work(2, None)
        torch.cuda.synchronize()
        for i in range(2):
            for x, y in zip(got[i], want):
                assert torch.equal(x, y)
            assert torch.equal(caches[i].buffer, caches[2].buffer)
            assert torch.equal(tables[i], tables[2])
    raw = streams[0].cuda_stream
    got = work(0, raw)  # a stream by its handle
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_blocks_beyond_4_gib():
    """Stores, transfers and attention whose blocks lie past 4 GiB of the pool."""
    T, H, D = 64, 8, 256
    size = R.block_bytes(T, H, D)
    blocks = (9 << 29) // size + 40                      # 4.5 GiB and some
    far = [blocks - 1, 3, blocks - 20, blocks // 2 + 1]
    c, c2 = (xf().PagedCache(blocks, T, H, D) for _ in range(2))
    n = 3 * T + 17
    key, value = (torch.randn(n, H, D, device="cuda").to(torch.float16) for _ in range(2))
    slots = [far[i // T] * T + i % T for i in range(n)]
    c.store(key, value, ints(slots))
    to = [5, blocks - 2, 7, blocks - 9]
    conn = xf().Conn("zcd", 4, 1, 65536, wgs_per_channel=2)
    c.send(conn, c2, ints(far), ints(to))
    q = torch.randn(2, 16, D, device="cuda").to(torch.float16)
    got = [x.attend(q, ints(t).reshape(1, 4), ints([n]), ints([0, 2]), lse=True) for x, t in ((c, far), (c2, to))]
    torch.cuda.synchronize()
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    small = R.Cache(c.buffer[far].cpu().numpy(), T, H, D)
    ref = R.Cache(np.zeros((4, size), np.uint8), T, H, D)
    R.store(ref, key.double().cpu().numpy(), value.double().cpu().numpy(), list(range(n)))
    assert np.array_equal(small.k, ref.k) and np.array_equal(small.v, ref.v) and np.array_equal(small.s, ref.s)
    want = R.attend(ref, q.double().cpu().numpy(), [[0, 1, 2, 3]], [n], [0, 2], 1 / math.sqrt(D))
    tol, tol_lse = R.attend_bounds(want, n, D, 2.0 ** -11)
    assert np.all(np.abs(got[0][0].double().cpu().numpy() - want[0]) <= tol)
    assert np.all(np.abs(got[0][1].double().cpu().numpy() - want[1]) <= tol_lse)
    conn.close()


def test_parts_of_a_context_join():
    """Attention over two halves of a context joined by their log sums is attention
    over the whole."""
    T, H, D = 16, 2, 128
    ref = new_pool(40, T, H, D, 3)
    c = gpu_cache(ref)
    q = torch.randn(1, 8, D, device="cuda").to(torch.bfloat16)
    t = ints(np.arange(36)).reshape(1, 36)
    whole, lse = c.attend(q, t, ints([576]), ints([0, 1]), lse=True)
    parts = [c.attend(q, x.contiguous(), ints([288]), ints([0, 1]), lse=True) for x in (t[:, :18], t[:, 18:])]
    ls = torch.stack([p[1] for p in parts]).double()
    total = torch.logsumexp(ls, 0)
    joined = sum(p[0].double() * (x - total).exp()[..., None] for p, x in zip(parts, ls))
    # each of the three outputs is rounded to bfloat16 (2^-8) and has weights rounded so (2^-8)
    mag = R.attend(ref, q.double().cpu().numpy(), t.tolist(), [576], [0, 1], 1 / math.sqrt(D))[2]
    assert np.all(np.abs((joined - whole.double()).cpu().numpy()) <= 4.1 * 2.0 ** -8 * mag + 1e-30)
    assert torch.allclose(total, lse.double(), atol=1e-4, rtol=0)
