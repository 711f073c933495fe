"""GPU tests of the 4-bit cache as a program uses it: one endpoint plans, stores and sends,
the other attends and reads back; eagerly, in captured graphs, on streams of their own and
beyond 4 GiB."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import cache_ref  # noqa: E402
import mxcache_ref as R  # noqa: E402
from mxcache_cases import bounds, gpu_cache, ints, new_pool, xf  # noqa: E402

pytestmark = pytest.mark.gpu


def empty_ref(blocks, T, H, D):
    return R.Cache(np.zeros((blocks, R.block_bytes(T, H, D)), np.uint8), T, H, D)


@pytest.mark.parametrize("proto", ["zcd", "simple"])
@pytest.mark.parametrize("T,H,group,D", [(16, 2, 4, 128), (64, 3, 1, 64), (32, 1, 7, 256), (16, 2, 3, 96)])
def test_prompt_handed_over_then_answered(T, H, group, D, proto):
    blocks, lens, width = 120, [100, 1, 37, 64], 12
    B, n = len(lens), sum(lens)
    rng, gen = np.random.default_rng(T + D), torch.Generator().manual_seed(D)
    here, there = (xf().PagedCache(blocks, T, H, D, bits=4) for _ in range(2))
    here.buffer.zero_()
    there.buffer.zero_()
    ref, ref_there = (empty_ref(blocks, T, H, D) for _ in range(2))
    conn = xf().Conn(proto, 4, 2, 16384, wgs_per_channel=2, timeout_ms=20000)

    def rows(n):
        return [torch.randn(n, h, D, generator=gen).to(torch.bfloat16) for h in (H, H, H * group)]

    # the prompt endpoint
    free = rng.permutation(blocks)
    table = ints(np.full(B * width, -1)).reshape(B, width)
    plan = xf().plan_blocks(ints([0] * B), ints(lens), table, ints(free), T, n)
    key, value, q = rows(n)
    here.store(key.cuda(), value.cuda(), plan.slots)
    slots, _, starts, lengths, _, want_table = cache_ref.plan([0] * B, lens, [[-1] * width] * B, free.tolist(), T, n)
    R.store(ref, key.double().numpy(), value.double().numpy(), slots)
    out, lse = here.attend(q.cuda(), table, plan.lengths, plan.starts, max_query=100, max_length=100, lse=True)
    want = R.attend(ref, q.double().numpy(), want_table, lengths, starts, 1 / math.sqrt(D))
    tol, tol_lse = bounds(want, 100, D, "bf16", False)
    assert np.all(np.abs(out.double().cpu().numpy() - want[0]) <= tol)
    # its blocks into blocks of the answering endpoint
    src = np.array(want_table).reshape(-1)
    dst = np.where(src >= 0, rng.permutation(blocks)[:src.size], -1)
    here.send(conn, there, table.reshape(-1), ints(dst))
    for s, d in zip(src[src >= 0], dst[src >= 0]):
        ref_there.k[d], ref_there.v[d], ref_there.s[d] = ref.k[s], ref.v[s], ref.s[s]
    # the answering endpoint: single tokens and drafted ones, then everything read back
    t2 = ints(dst).reshape(B, width)
    used = set(dst.tolist())
    free2 = [b for b in range(blocks) if b not in used]
    host_table, cached = dst.reshape(B, width).tolist(), list(lens)
    for step in (1, 1, 3, 1):
        added, n = [step] * B, step * B
        plan = xf().plan_blocks(ints(cached), ints(added), t2, ints(free2), T, n + 2)
        slots, _, starts, lengths, counts, host_table = cache_ref.plan(cached, added, host_table, free2, T, n + 2)
        key, value, q = rows(n + 2)
        there.store(key.cuda(), value.cuda(), plan.slots)
        R.store(ref_there, key.double().numpy(), value.double().numpy(), slots)
        out, lse = there.attend(q.cuda(), t2, plan.lengths, plan.starts, lse=True)
        want = R.attend(ref_there, q.double().numpy(), host_table, lengths, starts, 1 / math.sqrt(D))
        tol, tol_lse = bounds(want, max(lengths), D, "bf16", False)
        assert np.all(np.abs(out.double().cpu().numpy() - want[0])[:n] <= tol[:n])
        assert np.all(np.abs(lse.double().cpu().numpy() - want[1])[:n] <= tol_lse[:n])
        free2, cached = free2[counts[0]:], lengths
    starts = np.cumsum([0] + cached).tolist()
    got = there.load(t2, ints(cached), ints(starts), starts[-1], dtype=torch.float32)
    want = R.load(ref_there, host_table, cached, starts, starts[-1])
    for g, w in zip(got, want[:2]):
        assert np.array_equal(g.double().cpu().numpy(), w)
    assert np.array_equal(there.buffer.cpu().numpy(), ref_there.raw())
    torch.cuda.synchronize()
    assert conn.query(0)["error"] == 0
    conn.close()


def test_steps_in_graphs():
    """Plan, store, attend (single rows, and many that are shared out) and load, captured
    twice: two graphs alive, replayed in turn with eager calls between, give what eager
    calls give."""
    T, H, group, D, B, width = 16, 2, 4, 128, 3, 1000
    ref = new_pool(1000, T, H, D, 1)
    pool = gpu_cache(ref).buffer
    free = ints(np.arange(900, 950))
    pages = ints(np.arange(B * 290)).reshape(B, 290)
    many = [90, 5, 77]

    def stage():
        return dict(cached=ints([0] * B), added=ints([1] * B), table=ints(np.full(B * width, -1)).reshape(B, width),
                    key=torch.zeros(B, H, D, dtype=torch.bfloat16, device="cuda"),
                    value=torch.zeros(B, H, D, dtype=torch.bfloat16, device="cuda"),
                    query=torch.zeros(B, H * group, D, dtype=torch.bfloat16, device="cuda"),
                    rows=torch.zeros(sum(many), H * group, D, dtype=torch.bfloat16, device="cuda"),
                    starts=ints(np.cumsum([0] + many)),
                    cache=xf().PagedCache(1000, T, H, D, buffer=pool.clone(), bits=4))

    def step(s):
        plan = xf().plan_blocks(s["cached"], s["added"], s["table"], free, T, B)
        s["cache"].store(s["key"], s["value"], plan.slots)
        res = list(s["cache"].attend(s["query"], s["table"], plan.lengths, plan.starts, max_query=1,
                                     max_length=4640, lse=True))
        res += s["cache"].attend(s["rows"], s["table"], plan.lengths, s["starts"], lse=True)
        res += s["cache"].load(s["table"], plan.lengths, s["starts"], sum(many), dtype=torch.float16)
        return res

    stages, graphs = [stage() for _ in range(3)], []
    for s in stages[:2]:
        step(s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = step(s)
        graphs.append((g, res))
    torch.cuda.synchronize()
    for s in stages:
        s["cache"].buffer.copy_(pool)
    rng = np.random.default_rng(0)
    for it in range(6):
        lens = rng.integers(100, 4600, B)
        lens[it % B] = 90 + it
        gen = torch.Generator(device="cuda").manual_seed(it)
        new = [torch.randn(stages[2][x].shape, generator=gen, device="cuda").to(torch.bfloat16)
               for x in ("key", "value", "query", "rows")]
        for s in stages:
            s["cached"].copy_(ints(lens))
            s["table"].fill_(-1)
            s["table"][:, :290] = pages
            for x, y in zip(("key", "value", "query", "rows"), new):
                s[x].copy_(y)
        want = step(stages[2])
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for (_, res), s in zip(graphs, stages):
            assert all(torch.equal(x, y) for x, y in zip(res, want)), it
            assert torch.equal(s["cache"].buffer, stages[2]["cache"].buffer), it


def test_on_the_current_stream_and_on_others():
    """Calls queued on the current stream and on another without a synchronisation between
    them; every attention here has a workspace, freed on its return."""
    T, H, D, B = 16, 2, 128, 2
    caches = [gpu_cache(new_pool(700, T, H, D, 1)) for _ in range(3)]
    table = torch.full((B, 15000), -1, dtype=torch.int32, device="cuda")
    table[:, :300] = ints(range(600)).reshape(B, 300)
    kv = torch.randn(2, 40, H, D, device="cuda").to(torch.bfloat16)
    slots = ints(list(range(16 * 650, 16 * 650 + 40)))
    sets = [(torch.randn(rows[-1], 8, D, device="cuda").to(torch.bfloat16), ints(lens), ints(rows))
            for lens, rows in (([4700, 3100], [0, 1, 2]), ([4100, 4799], [0, 70, 150]), ([2600, 170], [0, 1, 2]))]

    def work(cache, i, stream):
        q, lens, starts = sets[i]
        cache.store(kv[0], kv[1], slots, stream=stream)
        out, lse = cache.attend(q, table, lens, starts, lse=True, stream=stream)
        return [out, lse] + list(cache.load(table, lens, starts, q.shape[0], stream=stream))

    want = [work(caches[2], i, None) for i in range(3)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        got = []
        for _ in range(6):
            for i, s in ((0, None), (1, stream), (2, None), (0, stream), (1, None), (2, stream)):
                got.append((i, work(caches[0 if s is None else 1], i, s)))
        torch.cuda.synchronize()
        for i, res in got:
            assert all(torch.equal(x, y) for x, y in zip(res, want[i])), i
        assert torch.equal(caches[0].buffer, caches[2].buffer) and torch.equal(caches[1].buffer, caches[2].buffer)


def test_blocks_beyond_4_gib():
    """Stores, transfers, attention and reading back with blocks past 4 GiB of the pool."""
    T, H, D = 64, 8, 256
    size = R.block_bytes(T, H, D)
    blocks = (9 << 29) // size + 40                      # 4.5 GiB and some
    far = [blocks - 1, 3, blocks - 20, blocks // 2 + 1]
    to = [5, blocks - 2, 7, blocks - 9]
    c, c2 = (xf().PagedCache(blocks, T, H, D, bits=4) for _ in range(2))
    n = 3 * T + 17
    key, value = (torch.randn(n, H, D, device="cuda").to(torch.float16) for _ in range(2))
    slots = [far[i // T] * T + i % T for i in range(n)]
    c.store(key, value, ints(slots))
    conn = xf().Conn("zcd", 4, 1, 65536, wgs_per_channel=2)
    c.send(conn, c2, ints(far), ints(to))
    small = empty_ref(4, T, H, D)
    R.store(small, key.double().cpu().numpy(), value.double().cpu().numpy(), [i for i in range(n)])
    for rows, told in ((2, 0), (60, 0), (60, 1 << 20)):  # (the last: tiles of many rows)
        q = torch.randn(rows, 16, D, device="cuda").to(torch.float16)
        want = R.attend(small, q.double().cpu().numpy(), [[0, 1, 2, 3]], [n], [0, rows], 1 / math.sqrt(D))
        tol, tol_lse = bounds(want, n, D, "fp16", told > 0)
        for x, blocks_at in ((c, far), (c2, to)):
            table = torch.full((1, 1 << 14), -1, dtype=torch.int32, device="cuda")[:, :1 << 14 if told else 4]
            table[:, :4] = ints(blocks_at)
            out, lse = x.attend(q, table, ints([n]), ints([0, rows]), max_query=rows, max_length=told, lse=True)
            assert np.all(np.abs(out.double().cpu().numpy() - want[0]) <= tol), (rows, told)
            assert np.all(np.abs(lse.double().cpu().numpy() - want[1]) <= tol_lse), (rows, told)
    want = R.load(small, [[0, 1, 2, 3]], [n], [0, n], n)
    for x, blocks_at in ((c, far), (c2, to)):
        got = x.load(ints(blocks_at).reshape(1, 4), ints([n]), ints([0, n]), n, dtype=torch.float32)
        assert all(np.array_equal(g.double().cpu().numpy(), w) for g, w in zip(got, want[:2]))
    torch.cuda.synchronize()
    assert conn.query(0)["error"] == 0
    conn.close()


def test_8_bit_cache_read_back_together():
    """The 8-bit cache's rows after plan and store are those that attention uses: within an
    8-bit rounding of what was stored, on another stream and in a replayed graph."""
    T, H, D, B = 16, 3, 96, 4
    lens = [33, 1, 64, 100]
    n = sum(lens)
    cache = xf().PagedCache(60, T, H, D)
    table = ints(np.full(B * 9, -1)).reshape(B, 9)
    plan = xf().plan_blocks(ints([0] * B), ints(lens), table, ints(range(50)), T, n)
    key, value = (torch.randn(n, H, D, device="cuda").to(torch.bfloat16) for _ in range(2))
    cache.store(key, value, plan.slots)
    want = cache.load(table, plan.lengths, plan.starts, n, dtype=torch.float32)
    for x, y in zip((key, value), want):
        # a block's scale is its largest / 448 or a power of two near it, codes have 4 bits
        assert torch.all((x.float() - y).abs() <= x.float().abs() * 2.0 ** -4 + x.float().abs().max() * 2.0 ** -9)
    outs = [torch.zeros(n, H, D, device="cuda") for _ in range(2)]
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        cache.load(table, plan.lengths, plan.starts, n, out=outs)
    side = torch.cuda.Stream()
    for _ in range(3):
        for o in outs:
            o.zero_()
        g.replay()
        other = cache.load(table, plan.lengths, plan.starts, n, dtype=torch.float32, stream=side)
        torch.cuda.synchronize()
        for x, y, z in zip(outs, other, want):
            assert torch.equal(x, z) and torch.equal(y, z)
