"""Cases of the paged 8-bit cache: block plans, stores, block transfers and attention.

A cache is a pool of blocks, each one record of bytes (the unit that a
connection moves): for every key/value head the key codes [T][D], then the
value codes [D][T], and after the heads a float32 pair of scales (key, value)
per head, padded to 128 bytes.  A code is an e4m3 number; it stands for code x
scale, where the scale is the smallest power of two 2^e, e >= -118, that
brings the largest finite magnitude of the block's tokens in that head to 448
or below.  A block that already holds tokens keeps the larger of its scale and
the one its new tokens need, and its earlier codes are rounded again to it.
Numbers that are not finite are held as NaN.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # One decode step of a small batch: a token each, latency only.
        dict(name="plan_decode_64", op="plan", batch=64, cached_lo=1, cached_hi=4096, added_lo=1,
             added_hi=1, block=16, rows_pad=0),
        # A wave of new prompts, some with a cached prefix, in a padded batch.
        dict(name="plan_prompts_1000", op="plan", batch=1000, cached_lo=0, cached_hi=500,
             added_lo=1, added_hi=1200, block=64, rows_pad=777),
        # The keys and values of one decode step: one token in each request's last block.
        dict(name="store_decode_256", op="store", batch=256, cached_lo=1, cached_hi=2000,
             added_lo=1, added_hi=1, kv_heads=8, dim=128, block=16, dtype="bf16"),
        # Packed prompts of a prefill batch, ragged, some continuing a cached prefix.
        dict(name="store_prompts_29", op="store", batch=29, cached_lo=0, cached_hi=300,
             added_lo=40, added_hi=4000, kv_heads=8, dim=128, block=64, dtype="fp16"),
        # One short request handed to the answering endpoint.
        dict(name="send_request_12", op="send", count=12, kv_heads=8, dim=128, block=16),
        # Everything a busy prompt endpoint has finished, in one transfer.
        dict(name="send_bulk_16000", op="send", count=16000, kv_heads=8, dim=128, block=16),
        # A single short conversation: latency only.
        dict(name="attend_single_300", op="attend", batch=1, len_lo=300, len_hi=300, q_lo=1,
             q_hi=1, heads=32, kv_heads=8, dim=128, block=16, dtype="bf16"),
        # An ordinary decode batch with grouped heads.
        dict(name="attend_decode_64", op="attend", batch=64, len_lo=500, len_hi=8000, q_lo=1,
             q_hi=1, heads=32, kv_heads=8, dim=128, block=16, dtype="bf16"),
        # Two very long documents: few rows, the work split over the length.
        dict(name="attend_long_2", op="attend", batch=2, len_lo=65001, len_hi=131071, q_lo=1,
             q_hi=1, heads=64, kv_heads=8, dim=128, block=64, dtype="fp16"),
        # Wide heads in an odd group, with a few drafted tokens each.
        dict(name="attend_draft_48", op="attend", batch=48, len_lo=17, len_hi=3001, q_lo=1,
             q_hi=5, heads=12, kv_heads=2, dim=256, block=32, dtype="bf16"),
        # A head of its own for every query head, narrow.
        dict(name="attend_heads_33", op="attend", batch=33, len_lo=1, len_hi=2500, q_lo=1, q_hi=1,
             heads=16, kv_heads=16, dim=64, block=16, dtype="fp16"),
        # Chunks of prompts over their cached prefix, beside decoding requests.
        dict(name="attend_chunks_8", op="attend", batch=8, len_lo=700, len_hi=5000, q_lo=1,
             q_hi=600, heads=32, kv_heads=8, dim=128, block=64, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "store", "send", "attend", "attend", "attend"])
    block = rng.choice([16, 32, 64])
    dim = rng.choice([64, 96, 128, 128, 192, 256])
    kv = rng.choice([1, 2, 3, 4, 5, 8, 8, 16])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "plan":
        return dict(op=op, batch=_log(rng, 1, 3000), cached_lo=0, cached_hi=_log(rng, 1, 8000),
                    added_lo=rng.choice([0, 1]), added_hi=_log(rng, 1, 700), block=block,
                    rows_pad=rng.choice([0, rng.randint(1, 999)]))
    if op == "store":
        one = rng.random() < 0.4
        batch = _log(rng, 1, 500) if one else _log(rng, 1, 40)
        hi = 1 if one else _log(rng, 2, 2500)
        return dict(op=op, batch=batch, cached_lo=0, cached_hi=_log(rng, 1, 500),
                    added_lo=1, added_hi=hi, kv_heads=min(kv, 8), dim=dim, block=block,
                    dtype=rng.choice(["bf16", "fp16", "fp32"]) if one else dtype)
    if op == "send":
        size = 2 * kv * dim * block
        return dict(op=op, count=max(1, _log(rng, 1, min(30000, (500 << 20) // size))),
                    kv_heads=kv, dim=dim, block=block)
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 8, 16])
    kv = min(kv, 8)
    kind = rng.choice(["decode", "decode", "draft", "chunk"])
    if kind == "chunk":
        batch, hi, q = rng.randint(1, 6), _log(rng, 600, 4500), rng.randint(16, 500)
        group = min(group, 4)
    else:
        batch = _log(rng, 1, 80)
        hi = min(_log(rng, 2, 90000), max(2, int(4e8 / (batch * kv * dim * 2))))
        q = 1 if kind == "decode" else rng.randint(2, 8)
    return dict(op=op, batch=batch, len_lo=max(1, hi // rng.choice([1, 3, 20])), len_hi=hi,
                q_lo=1, q_hi=q, heads=kv * group, kv_heads=kv, dim=dim, block=block, dtype=dtype)


# --------------------------------------------------- lengths of a case's requests
def _spread(n, lo, hi, turn):
    """n whole numbers from lo to hi, even in their logarithm, in a mixed order."""
    if n == 1:
        return [hi]
    got = [int(round((lo + 1) * ((hi + 1) / (lo + 1)) ** (i / (n - 1)))) - 1 for i in range(n)]
    step = next(s for s in range(turn, turn + n + 2) if math.gcd(s, n) == 1)
    return [got[(i * step + turn) % n] for i in range(n)]


def _growth(case):
    b = case["batch"]
    return (_spread(b, case["cached_lo"], case["cached_hi"], 7),
            _spread(b, case["added_lo"], case["added_hi"], 11))


def _reach(case):
    """Tokens in the cache and query rows of each request."""
    b = case["batch"]
    lens = _spread(b, case["len_lo"], case["len_hi"], 7)
    rows = _spread(b, case["q_lo"], case["q_hi"], 11)
    return lens, rows


def _up(n, to):
    return -(-n // to) * to


def _block_bytes(case):
    h, d, t = case["kv_heads"], case["dim"], case["block"]
    return 2 * h * d * t + _up(8 * h, 128)


# ------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 1000003 + 17)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _views(pool, h, d, t):
    """Codes of keys [blocks, H, T, D] and values [blocks, H, D, T], scales [blocks, H, 2]."""
    n, size = pool.shape
    codes = pool.view(torch.float8_e4m3fn)
    k = codes.as_strided((n, h, t, d), (size, 2 * t * d, d, 1), 0)
    v = codes.as_strided((n, h, d, t), (size, 2 * t * d, t, 1), t * d)
    s = pool.view(torch.float32).as_strided((n, h, 2), (size // 4, 2, 1), 2 * h * t * d // 4)
    return k, v, s


def _pool(case, blocks, g):
    """A pool of `blocks` blocks full of codes, as earlier requests left them."""
    h, d, t = case["kv_heads"], case["dim"], case["block"]
    pool = torch.zeros(blocks, _block_bytes(case), dtype=torch.uint8, device=DEV)
    k, v, s = _views(pool, h, d, t)
    step = max(1, (64 << 20) // (h * d * t))
    for x in (k, v):
        for i in range(0, blocks, step):
            part = x[i:i + step]
            part.copy_((torch.randn(part.shape, generator=g, device=DEV) * 90).clamp_(-448, 448)
                       .to(torch.float8_e4m3fn))
    s.copy_(torch.exp2(torch.randint(-8, -5, s.shape, generator=g, device=DEV).float()))
    return pool


def _table(held, width, order):
    """Block ids of each request (the first `held` of its row), -1 behind them; the ids are taken in `order`."""
    b = len(held)
    n = torch.tensor(held, device=DEV)
    base = torch.cumsum(n, 0) - n
    at = torch.arange(width, device=DEV)
    there = at[None, :] < n[:, None]
    idx = torch.where(there, base[:, None] + at[None, :], torch.zeros((), dtype=torch.int64, device=DEV))
    table = torch.where(there, order[idx.clamp_(max=order.numel() - 1)], torch.full((), -1, dtype=order.dtype, device=DEV))
    return table.to(torch.int32).reshape(b, width).contiguous()


def _rows(counts):
    """Request and place within it of each packed row."""
    n = torch.tensor(counts, device=DEV)
    who = torch.repeat_interleave(torch.arange(len(counts), device=DEV), n)
    place = torch.arange(who.numel(), device=DEV) - (torch.cumsum(n, 0) - n)[who]
    return who, place


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = dict(case=dict(case))
    t = case["block"]
    if op == "plan":
        cached, added = _growth(case)
        held = [-(-c // t) for c in cached]
        want = [-(-(c + a) // t) for c, a in zip(cached, added)]
        order = torch.randperm(sum(want) + 32, generator=g, device=DEV)
        st["cached"], st["added"] = _ints(cached), _ints(added)
        st["table"] = _table(held, max(want) + 3, order)
        st["free"] = order[sum(held):].to(torch.int32).contiguous()
        st["rows"] = sum(added) + case["rows_pad"]
        return st
    h, d = case["kv_heads"], case["dim"]
    if op == "send":
        n = case["count"]
        total = n + n // 8 + 3
        st["src"] = _pool(case, total, g)
        st["dst"] = torch.zeros(total, _block_bytes(case), dtype=torch.uint8, device=DEV)
        st["from"] = torch.randperm(total, generator=g, device=DEV)[:n].to(torch.int32).contiguous()
        st["to"] = torch.randperm(total, generator=g, device=DEV)[:n].to(torch.int32).contiguous()
        if own:  # the endpoints' open connection and caches
            from recv_fifo_plane_amd import PagedCache
            st["conn"] = _connection()
            st["caches"] = [PagedCache(total, t, h, d, buffer=st[x]) for x in ("src", "dst")]
        return st
    dtype = DTYPES[case["dtype"]]
    if op == "store":
        cached, added = _growth(case)
        want = [-(-(c + a) // t) for c, a in zip(cached, added)]
        total = sum(want) + 5
        st["pool"] = _pool(case, total, g)
        table = _table(want, max(want), torch.randperm(total, generator=g, device=DEV))
        who, place = _rows(added)
        pos = torch.tensor(cached, device=DEV)[who] + place
        st["slots"] = (table[who, pos // t].long() * t + pos % t).to(torch.int32)
        n = who.numel()
        st["runs"] = sum(w - c // t for w, c, a in zip(want, cached, added) if a)
        # as projections give them: one fused row per token, a few loud channels in the keys
        kv = torch.randn(n, 2 * h, d, generator=g, device=DEV)
        loud = 1 + 6 * (torch.rand(h, d, generator=g, device=DEV) > 0.97)
        kv[:, :h] *= loud
        st["kv"] = kv.to(dtype)
        st["key"], st["value"] = st["kv"][:, :h], st["kv"][:, h:]
        if own:
            from recv_fifo_plane_amd import PagedCache
            st["cache"] = PagedCache(total, t, h, d, buffer=st["pool"])
        return st
    lens, rows = _reach(case)
    used = [-(-x // t) for x in lens]
    total = sum(used) + 5
    st["pool"] = _pool(case, total, g)
    st["table"] = _table(used, max(used), torch.randperm(total, generator=g, device=DEV))
    # what stands behind a request's last token is not a number
    k, v, _ = _views(st["pool"], h, d, t)
    tail = [i for i, x in enumerate(lens) if x % t]
    if tail:
        last = st["table"][torch.tensor(tail, device=DEV), torch.tensor([used[i] - 1 for i in tail], device=DEV)].long()
        keep = torch.tensor([lens[i] % t for i in tail], device=DEV)
        gone = torch.arange(t, device=DEV)[None, :] >= keep[:, None]
        ku, vu = k.view(torch.uint8), v.view(torch.uint8)
        ku[last] = torch.where(gone[:, None, :, None], torch.full((), 127, dtype=torch.uint8, device=DEV), ku[last])
        vu[last] = torch.where(gone[:, None, None, :], torch.full((), 127, dtype=torch.uint8, device=DEV), vu[last])
    n = sum(rows)
    st["query"] = torch.randn(n, case["heads"], d, generator=g, device=DEV).to(dtype)
    st["lengths"] = _ints(lens)
    starts = [0]
    for r in rows:
        starts.append(starts[-1] + r)
    st["starts"] = _ints(starts)
    st["longest"], st["most"] = max(lens), max(rows)
    if own:
        from recv_fifo_plane_amd import PagedCache
        st["cache"] = PagedCache(total, t, h, d, buffer=st["pool"])
    return st


_conn = None


def _connection():
    """The program's connection between the two endpoints, opened once."""
    global _conn
    if _conn is None:
        from recv_fifo_plane_amd import workloads
        _conn = workloads.make_conn(workloads.W4D_PAIR)
    return _conn


# --------------------------------------------------------------------- run
def run(st):
    op = st["case"]["op"]
    if op == "plan":
        if own:
            from recv_fifo_plane_amd import plan_blocks
            plan = plan_blocks(st["cached"], st["added"], st["table"], st["free"],
                               st["case"]["block"], st["rows"])
            return dict(slots=plan.slots, positions=plan.positions, starts=plan.starts,
                        lengths=plan.lengths, counts=plan.counts, table=st["table"])
        return _plain_plan(st)
    if op == "store":
        if own:
            st["cache"].store(st["key"], st["value"], st["slots"])
        else:
            _plain_store(st)
        return _held(st["case"], st["pool"])
    if op == "send":
        if own:
            st["caches"][0].send(st["conn"], st["caches"][1], st["from"], st["to"])
        else:
            st["dst"][st["to"].long()] = st["src"][st["from"].long()]
        return _held(st["case"], st["dst"])
    if own:
        out, lse = st["cache"].attend(st["query"], st["table"], st["lengths"], st["starts"],
                                      max_query=st["most"], max_length=st["longest"], lse=True)
        return dict(out=out, lse=lse)
    return _plain_attend(st)


def _held(case, pool):
    """The codes' values and the scales they are held with."""
    k, v, s = _views(pool, case["kv_heads"], case["dim"], case["block"])
    return dict(key=k, value=v, scales=s)


def _plain_plan(st):
    t = st["case"]["block"]
    cached, added, table, free = st["cached"].long(), st["added"].long(), st["table"], st["free"].long()
    width = table.shape[1]
    held, want = (cached + t - 1) // t, (cached + added + t - 1) // t
    first = torch.cumsum(want - held, 0) - (want - held)
    at = torch.arange(width, device=DEV)[None, :]
    take = first[:, None] + at - held[:, None]
    fresh = (at >= held[:, None]) & (at < want[:, None]) & (take < free.numel())
    ids = torch.where(fresh, free[take.clamp(0, max(free.numel() - 1, 0))], table.long())
    table.copy_(ids)
    starts = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), torch.cumsum(added, 0)])
    row = torch.arange(st["rows"], device=DEV)
    who = torch.searchsorted(starts[1:], row, right=True)
    real = who < cached.numel()
    who = who.clamp(max=cached.numel() - 1)
    pos = cached[who] + row - starts[who]
    page = pos // t
    got = ids[who, page.clamp(max=width - 1)]
    reach = torch.minimum(torch.full((), width, device=DEV), held + (free.numel() - first).clamp(min=0))
    there = real & (page < reach[who]) & (got >= 0)
    slots = torch.where(there, got * t + pos % t, -1)
    lost = (cached + added - torch.maximum(cached, reach * t)).clamp(min=0).sum()
    counts = torch.stack([(want - held).sum(), lost])
    whole = lambda x: x.to(torch.int32)  # noqa: E731
    return dict(slots=whole(slots), positions=whole(torch.where(real, pos, -1)), starts=whole(starts),
                lengths=whole(cached + added), counts=whole(counts), table=table)


def _power(amax):
    """The smallest power of two, at least 2^-118, that brings amax to 448 or below."""
    m, e = torch.frexp(amax)  # amax = m * 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    return torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, e, -118).clamp(min=-118))


def _codes(x):
    return torch.where(torch.isfinite(x), x, float("nan")).to(torch.float8_e4m3fn)


def _plain_store(st):
    case = st["case"]
    t, h, d = case["block"], case["kv_heads"], case["dim"]
    k, v, s = _views(st["pool"], h, d, t)
    slots = st["slots"].long()
    blk, off = slots // t, slots % t
    opens = (off == 0) | (slots != torch.roll(slots, 1) + 1)   # rows that begin a block's run
    opens[0] = True
    which = torch.cumsum(opens, 0) - 1
    touched = torch.zeros(st["runs"], dtype=torch.int64, device=DEV).scatter_(0, which, blk)
    first = torch.full((touched.numel(),), t, dtype=torch.int64, device=DEV).scatter_reduce_(0, which, off, "amin")
    place = torch.arange(t, device=DEV)
    olds = place[None, :] < first[:, None]
    news = []
    for side, (codes, x) in enumerate(((k, st["key"]), (v.transpose(2, 3), st["value"]))):
        x = x.float()
        amax = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(2)
        need = torch.zeros(touched.numel(), h, device=DEV).scatter_reduce_(
            0, which[:, None].expand(-1, h), amax, "amax")
        old = s[touched][:, :, side]
        new = _power(need)
        new = torch.where(first[:, None] > 0, torch.maximum(old, new), new)
        kept = codes.view(torch.uint8)[touched].view(torch.float8_e4m3fn)
        again = _codes(kept.float() * (old / new)[:, :, None, None])
        mixed = torch.where(olds[:, None, :, None], again.view(torch.uint8), kept.view(torch.uint8))
        mixed = mixed.permute(0, 2, 1, 3).contiguous()
        mixed[which, off] = _codes(x / new[which][:, :, None]).view(torch.uint8)
        codes.view(torch.uint8)[touched] = mixed.permute(0, 2, 1, 3)
        news.append(new)
    s[touched] = torch.stack(news, 2)


def _plain_attend(st):
    case = st["case"]
    t, h, d, heads = case["block"], case["kv_heads"], case["dim"], case["heads"]
    k, v, s = _views(st["pool"], h, d, t)
    lens, starts = st["lengths"].long(), st["starts"].long()
    b, group = lens.numel(), heads // h
    pages = -(-st["longest"] // t)
    ids = st["table"][:, :pages].long()
    good = ids >= 0
    ids = ids.clamp(min=0)
    sc = s[ids]                                                       # [b, pages, h, 2]
    keys = k.view(torch.uint8)[ids].view(torch.float8_e4m3fn).float() * sc[..., 0, None, None]
    keys = keys.permute(0, 2, 1, 3, 4).reshape(b, h, pages * t, d)
    vals = v.view(torch.uint8)[ids].view(torch.float8_e4m3fn).float() * sc[..., 1, None, None]
    vals = vals.permute(0, 2, 1, 4, 3).reshape(b, h, pages * t, d)
    pos = torch.arange(pages * t, device=DEV)
    there = (pos[None, :] < lens[:, None]) & good.repeat_interleave(t, 1)   # [b, L]
    vals = torch.where(there[:, None, :, None], vals, 0.0)
    place = torch.arange(st["most"], device=DEV)
    count = starts[1:] - starts[:-1]
    real = place[None, :] < count[:, None]                            # [b, rows]
    row = torch.where(real, starts[:-1, None] + place[None, :], 0)
    q = st["query"].float()[row]                                      # [b, rows, heads, d]
    q = q.reshape(b, -1, h, group, d).permute(0, 2, 1, 3, 4).reshape(b, h, -1, d)
    scores = torch.matmul(q, keys.transpose(2, 3)).mul_(1 / math.sqrt(d))
    last = (lens - count)[:, None] + place[None, :]                   # the last token that a row sees
    seen = there[:, None, :] & (pos[None, None, :] <= last[:, :, None])
    scores = scores.reshape(b, h, st["most"], group, -1)
    scores.masked_fill_(~seen[:, None, :, None, :], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(b, h, -1, pages * t), vals).reshape(b, h, -1, group, d)
    o = torch.where(total > 0, o / total.clamp(min=1e-38), 0.0)
    lse = (top + total.log()).squeeze(-1)
    at = torch.arange(st["query"].shape[0], device=DEV)
    who = torch.searchsorted(starts[1:], at, right=True)
    at = at - starts[who]
    out = o.permute(0, 2, 1, 3, 4).reshape(b, -1, heads, d)[who, at]
    return dict(out=out.to(st["query"].dtype), lse=lse.permute(0, 2, 1, 3).reshape(b, -1, heads)[who, at])


# -------------------------------------------------------------------- work
def work(case):
    op, t = case["op"], case["block"]
    if op == "plan":
        cached, added = _growth(case)
        new = sum(-(-(c + a) // t) - -(-c // t) for c, a in zip(cached, added))
        rows = sum(added) + case["rows_pad"]
        return dict(bytes=8 * case["batch"] + 8 * new + 8 * rows + 8 * case["batch"], flops=0)
    h, d = case["kv_heads"], case["dim"]
    if op == "send":
        return dict(bytes=2 * case["count"] * _block_bytes(case) + 8 * case["count"], flops=0)
    size = 4 if case["dtype"] == "fp32" else 2
    if op == "store":
        cached, added = _growth(case)
        blocks = sum(-(-(c + a) // t) - c // t for c, a in zip(cached, added) if a)
        n = sum(added)
        return dict(bytes=n * 2 * h * d * (size + 1) + 4 * n + 8 * h * blocks, flops=0)
    lens, rows = _reach(case)
    blocks = sum(-(-x // t) for x in lens)
    n, heads = sum(rows), case["heads"]
    pairs = sum(sum(max(0, x - r + j + 1) for j in range(r)) for x, r in zip(lens, rows))
    return dict(bytes=2 * h * d * sum(lens) + (8 * h + 4) * blocks + n * heads * (2 * d * size + 4),
                flops=4 * d * heads * pairs)


# ------------------------------------------------------------------- exact
def exact(case, seed):
    global own
    kept, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = kept
    return {"plan": _exact_plan, "store": _exact_store, "send": _exact_send, "attend": _exact_attend}[case["op"]](st)


def _exact_plan(st):
    """Request by request, taking each new block from the front of the free list."""
    t = st["case"]["block"]
    cached, added = st["cached"].tolist(), st["added"].tolist()
    table, free = st["table"].tolist(), st["free"].tolist()
    slots, positions, starts, taken, lost = [], [], [0], 0, 0
    for i, (c, a) in enumerate(zip(cached, added)):
        for p in range(-(-c // t), -(-(c + a) // t)):
            if p < len(table[i]) and taken < len(free):
                table[i][p] = free[taken]
            taken += 1
        for p in range(c, c + a):
            block = table[i][p // t] if p // t < len(table[i]) else -1
            slots.append(block * t + p % t if block >= 0 else -1)
            lost += block < 0
            positions.append(p)
        starts.append(starts[-1] + a)
    pad = [-1] * (st["rows"] - len(slots))
    lens = [c + a for c, a in zip(cached, added)]
    named = dict(slots=slots + pad, positions=positions + pad, starts=starts, lengths=lens,
                 counts=[taken, lost], table=table)
    return {k: torch.tensor(v, dtype=torch.int32) for k, v in named.items()}


def _round_e4m3(x):
    """Nearest e4m3 number, ties to the even one; x in 64 bits, 448 at most."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -30)))
    e = torch.where(torch.exp2(e) > x.abs(), e - 1, e)
    e = torch.where(torch.exp2(e + 1) <= x.abs(), e + 1, e).clamp(min=-6)
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def _exact_store(st):
    case = st["case"]
    t, h, d = case["block"], case["kv_heads"], case["dim"]
    k, v, s = _views(st["pool"], h, d, t)
    out = [k.double(), v.double().transpose(2, 3).contiguous(), s.double()]
    k64, v64, s64 = out
    slots = st["slots"].tolist()
    runs = []  # (block, first place, first row, rows)
    for n, slot in enumerate(slots):
        if runs and slot % t and slot == slots[n - 1] + 1:
            runs[-1][3] += 1
        else:
            runs.append([slot // t, slot % t, n, 1])
    if len(runs) > 20000:
        return None
    blk, off, row, cnt = (torch.tensor(x, device=DEV) for x in zip(*runs))
    for side, (codes, x) in enumerate(((k64, st["key"].double()), (v64, st["value"].double()))):
        # every run's rows, in a frame of the block's places
        place = torch.arange(t, device=DEV)[None, :]
        mine = (place >= off[:, None]) & (place < (off + cnt)[:, None])
        rows = torch.where(mine, row[:, None] + place - off[:, None], 0)
        step = max(1, (32 << 20) // (t * h * d))
        for i in range(0, len(runs), step):
            c = slice(i, i + step)
            new = x[rows[c]].permute(0, 2, 1, 3)                      # [runs, h, t, d]
            m = mine[c][:, None, :, None]
            peak = torch.where(m, new.abs(), 0.0).amax((2, 3))
            e = torch.ceil(torch.log2(peak.clamp(min=1e-300) / 448)).clamp(min=-118)
            e = torch.where(peak > 448 * torch.exp2(e), e + 1, e)
            e = torch.where((peak <= 448 * torch.exp2(e - 1)) & (e > -118), e - 1, e)
            scale = torch.exp2(e)
            was = s64[blk[c], :, side]
            scale = torch.where(off[c][:, None] > 0, torch.maximum(scale, was), scale)
            held = codes[blk[c]]
            again = _round_e4m3(held * (was / scale)[:, :, None, None])
            before = (place[:, None, :, None] < off[c][:, None, None, None])
            codes[blk[c]] = torch.where(m, _round_e4m3(new / scale[:, :, None, None]),
                                        torch.where(before, again, held))
            s64[blk[c], :, side] = scale
    return dict(key=k64, value=v64.transpose(2, 3), scales=s64)


def _exact_send(st):
    case = st["case"]
    src, dst = st["src"], st["dst"]
    for i, j in zip(st["from"].tolist(), st["to"].tolist()):
        dst[j] = src[i]
    got = _held(case, dst)
    return {k: v.double() for k, v in got.items()}


def _exact_attend(st):
    case = st["case"]
    t, h, d, heads = case["block"], case["kv_heads"], case["dim"], case["heads"]
    k, v, s = _views(st["pool"], h, d, t)
    lens, starts = st["lengths"].tolist(), st["starts"].tolist()
    n = starts[-1]
    out = torch.zeros(n, heads, d, dtype=torch.float64, device=DEV)
    lse = torch.full((n, heads), float("-inf"), dtype=torch.float64, device=DEV)
    for i, length in enumerate(lens):
        r0, r1 = starts[i], starts[i + 1]
        if r1 == r0 or length == 0:
            continue
        ids = st["table"][i, : -(-length // t)].long()
        limit = length - (r1 - r0) + torch.arange(r1 - r0, device=DEV)
        seen = torch.arange(length, device=DEV)[None, :] <= limit[:, None]
        for j in range(h):
            keys = (k[:, j].view(torch.uint8)[ids].view(torch.float8_e4m3fn).double()
                    * s[ids, j, 0].double()[:, None, None]).reshape(-1, d)[:length]
            vals = (v[:, j].view(torch.uint8)[ids].view(torch.float8_e4m3fn).double()
                    * s[ids, j, 1].double()[:, None, None]).transpose(1, 2).reshape(-1, d)[:length]
            mine = slice(j * (heads // h), (j + 1) * (heads // h))
            q = st["query"][r0:r1, mine].double()
            x = (q.reshape(-1, d) @ keys.T).reshape(r1 - r0, -1, length) / math.sqrt(d)
            x = torch.where(seen[:, None, :], x, float("-inf"))
            some = limit >= 0
            z = torch.logsumexp(x, -1)
            lse[r0:r1, mine] = z
            p = torch.exp(x - torch.where(some[:, None], z, 0.0)[:, :, None])
            out[r0:r1, mine] = (p.reshape(-1, length) @ vals).reshape(r1 - r0, -1, d)
    return dict(out=out, lse=lse)
