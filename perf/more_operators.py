"""Cases of the paged cache in 4 bits (stores read back, attention), and of reading
either cache back into rows.

The cache of 4 bits is a pool of blocks of T tokens, each one record of bytes: for
every key/value head the key codes, then the value codes (D / 2 bytes a token
each), and behind the heads a byte of scale for each head, side (key, value), 32
dims and token ([H][2][D / 32][T]), padded to 128 bytes.  A code is an e2m1
number; it stands for code x 2^(byte - 127).  The power is the smallest 2^e, e
from -118 to 125, with the largest magnitude of the token's 32 dims at most 7 x
2^e (a code ends at 6, which is the nearest to anything up to 7 and beyond); byte
255 stands for 32 dims of which some are not finite: all are held as NaN.

Key codes lie as [T][D / 2], dim 2j in the lower half of byte j.  Value codes lie
in parts of 128, 64 or 32 dims, as D is made of (96 = 64 + 32, 192 = 128 + 64);
in a part a sixteenth of its dims, b = 4, 2 or 1 bytes, of 16 / b tokens lie
together: [T / u][16][u][b], u = 16 / b.

The cache of 8 bits is that of operators.py: e4m3 key codes [T][D], value codes
[D][T] and a float32 pair of scales a head.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases
def listed():
    return [
        # The keys and values of one decode step, in a batch padded for its graph: a
        # token each into its request's last block, and read back.
        dict(name="store_decode_256", op="store", batch=256, cached_lo=1, cached_hi=2000,
             added_lo=1, added_hi=1, pad=32, kv_heads=8, dim=128, block=16, dtype="bf16"),
        # Packed prompts of a prefill batch, ragged, some going on after a cached prefix.
        dict(name="store_prompts_29", op="store", batch=29, cached_lo=0, cached_hi=300,
             added_lo=40, added_hi=4000, pad=0, kv_heads=8, dim=128, block=64, dtype="fp16"),
        # A short context read back for another use: latency only.
        dict(name="load_context_300", op="load", bits=4, batch=1, len_lo=300, len_hi=300,
             kv_heads=8, dim=128, block=16, dtype="bf16"),
        # The cached prefixes of many requests, as rows for a prompt's own attention.
        dict(name="load_prefixes_4bit", op="load", bits=4, batch=24, len_lo=200, len_hi=9001,
             kv_heads=8, dim=128, block=16, dtype="bf16"),
        # The same of a cache in 8 bits, heads of an odd size.
        dict(name="load_prefixes_8bit", op="load", bits=8, batch=17, len_lo=77, len_hi=12001,
             kv_heads=5, dim=192, block=32, dtype="fp16"),
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
        # Whole prompts, each row over what stands before it.
        dict(name="attend_prompts_5", op="attend", batch=5, len_lo=300, len_hi=2900, q_lo=300,
             q_hi=2900, whole=True, heads=24, kv_heads=6, dim=96, block=32, dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "load", "attend", "attend"])
    block = rng.choice([16, 32, 64])
    dim = rng.choice([64, 96, 128, 128, 192, 256])
    kv = rng.choice([1, 2, 3, 4, 5, 8, 8])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "store":
        one = rng.random() < 0.4
        batch = _log(rng, 1, 500) if one else _log(rng, 1, 40)
        hi = 1 if one else min(_log(rng, 2, 2500), max(2, int(6e7 / (batch * kv * dim))))
        return dict(op=op, batch=batch, cached_lo=0, cached_hi=_log(rng, 1, 500), added_lo=1,
                    added_hi=hi, pad=rng.choice([0, rng.randint(1, 99)]), kv_heads=kv, dim=dim,
                    block=block, dtype=rng.choice(["bf16", "fp16", "fp32"]))
    if op == "load":
        batch = _log(rng, 1, 60)
        hi = min(_log(rng, 2, 40000), max(2, int(3e7 / (batch * kv * dim))))
        return dict(op=op, bits=rng.choice([4, 4, 8]), batch=batch,
                    len_lo=max(1, hi // rng.choice([1, 3, 20])), len_hi=hi, kv_heads=kv, dim=dim,
                    block=block, dtype=rng.choice(["bf16", "fp16", "fp32"]))
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 8, 16])
    kind = rng.choice(["decode", "decode", "draft", "chunk", "whole"])
    if kind == "chunk":
        batch, hi, q = rng.randint(1, 5), _log(rng, 600, 4000), rng.randint(16, 400)
        group = min(group, 4)
    elif kind == "whole":
        batch, group = rng.randint(1, 4), min(group, 4)
        hi = min(_log(rng, 40, 2000), int(math.sqrt(2.7e10 / (batch * kv * group * dim))))
        q = hi
    else:
        batch = _log(rng, 1, 80)
        hi = min(_log(rng, 2, 90000), max(2, int(4e8 / (batch * kv * dim * 2))))
        q = 1 if kind == "decode" else rng.randint(2, 8)
    lo = max(1, hi // rng.choice([1, 3, 20]))
    return dict(op=op, batch=batch, len_lo=lo, len_hi=hi, q_lo=lo if kind == "whole" else 1, q_hi=q,
                whole=kind == "whole", heads=kv * group, kv_heads=kv, dim=dim, block=block,
                dtype=dtype)


# --------------------------------------------------- lengths of a case's requests
def _spread(n, lo, hi, turn):
    """n whole numbers from lo to hi, even in their logarithm, in a mixed order."""
    if n == 1:
        return [hi]
    got = [int(round((lo + 1) * ((hi + 1) / (lo + 1)) ** (i / (n - 1)))) - 1 for i in range(n)]
    step = next(s for s in range(turn, turn + n + 2) if math.gcd(s, n) == 1)
    return [got[(i * step + turn) % n] for i in range(n)]


def _growth(case):
    """Tokens in the cache and tokens that a store adds, of each request."""
    b = case["batch"]
    return (_spread(b, case["cached_lo"], case["cached_hi"], 7),
            _spread(b, case["added_lo"], case["added_hi"], 11))


def _reach(case):
    """Tokens in the cache and rows of each request."""
    b = case["batch"]
    lens = _spread(b, case["len_lo"], case["len_hi"], 7)
    if case["op"] == "load" or case.get("whole"):
        return lens, lens
    return lens, _spread(b, case["q_lo"], case["q_hi"], 11)


def _up(n, to):
    return -(-n // to) * to


def _parts(d):
    """(first dim, dims) of the parts that value codes lie in."""
    return {64: [(0, 64)], 96: [(0, 64), (64, 32)], 128: [(0, 128)], 192: [(0, 128), (128, 64)],
            256: [(0, 128), (128, 128)]}[d]


def _block_bytes(case):
    h, d, t = case["kv_heads"], case["dim"], case["block"]
    if case.get("bits") == 8:
        return 2 * h * d * t + _up(8 * h, 128)
    return h * d * t + _up(h * d * t // 16, 128)


# ------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 1000003 + 29)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _views4(pool, h, d, t):
    """Of a pool of 4 bits, as bytes: keys [blocks, H, T, D / 2], values a list of
    [blocks, H, T / u, 16, u, b], scales [blocks, H, 2, D / 32, T]."""
    n, size = pool.shape
    k = pool.as_strided((n, h, t, d // 2), (size, t * d, d // 2, 1), 0)
    v = []
    for at, dims in _parts(d):
        b = dims // 32
        u = 16 // b
        v.append(pool.as_strided((n, h, t // u, 16, u, b), (size, t * d, 256, 16, b, 1),
                                 t * d // 2 + t * at // 2))
    s = pool.as_strided((n, h, 2, d // 32, t), (size, 2 * d // 32 * t, d // 32 * t, t, 1), h * t * d)
    return k, v, s


def _views8(pool, h, d, t):
    """Of a pool of 8 bits: key codes [blocks, H, T, D], value codes [blocks, H, D,
    T], scales [blocks, H, 2]."""
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
    step = max(1, (16 << 20) // (h * d * t))
    if case.get("bits") == 8:
        k, v, s = _views8(pool, h, d, t)
        for x in (k, v):
            for i in range(0, blocks, step):
                part = x[i:i + step]
                part.copy_((torch.randn(part.shape, generator=g, device=DEV) * 90)
                           .clamp_(-448, 448).to(torch.float8_e4m3fn))
        s.copy_(torch.exp2(torch.randint(-8, -5, s.shape, generator=g, device=DEV).float()))
        return pool
    # bytes of two codes, magnitudes as those of normal numbers of about 2.5 to their scale
    k, v, s = _views4(pool, h, d, t)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    share = torch.erf(edges / 2.5 / math.sqrt(2.0))
    at = (torch.arange(4096, device=DEV) + 0.5) / 4096
    code = (at[:, None] > share[None, :]).sum(1).to(torch.uint8)      # of 4096 equal shares
    for x in [k] + v:
        for i in range(0, blocks, step):
            part = x[i:i + step]
            r = torch.randint(0, 1 << 26, part.shape, generator=g, device=DEV, dtype=torch.int32)
            signs = ((r >> 24) & 1) * 8 + ((r >> 25) & 1) * 128
            part.copy_(code[(r & 4095).long()] | code[((r >> 12) & 4095).long()] << 4
                       | signs.to(torch.uint8))
    s.copy_(torch.randint(125, 128, s.shape, generator=g, device=DEV, dtype=torch.uint8))
    return pool


def _table(held, width, order):
    """Block ids of each request (the first `held` of its row), -1 behind them; the ids
    are taken in `order`."""
    b = len(held)
    n = torch.tensor(held, device=DEV)
    base = torch.cumsum(n, 0) - n
    at = torch.arange(width, device=DEV)
    there = at[None, :] < n[:, None]
    idx = torch.where(there, base[:, None] + at[None, :], 0)
    table = torch.where(there, order[idx.clamp_(max=order.numel() - 1)], -1)
    return table.to(torch.int32).reshape(b, width).contiguous()


def _rows(counts):
    """Request and place within it of each packed row."""
    n = torch.tensor(counts, device=DEV)
    who = torch.repeat_interleave(torch.arange(len(counts), device=DEV), n)
    place = torch.arange(who.numel(), device=DEV) - (torch.cumsum(n, 0) - n)[who]
    return who, place


def _starts(rows):
    starts = [0]
    for r in rows:
        starts.append(starts[-1] + r)
    return _ints(starts)


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case=dict(case))
    t, h, d = case["block"], case["kv_heads"], case["dim"]
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "store":
        cached, added = _growth(case)
        lens = [c + a for c, a in zip(cached, added)]
        rows = added
    else:
        lens, rows = _reach(case)
    used = [-(-x // t) for x in lens]
    total = sum(used) + 5
    st["pool"] = _pool(case, total, g)
    st["table"] = _table(used, max(used), torch.randperm(total, generator=g, device=DEV))
    st["lengths"], st["starts"], st["rows"] = _ints(lens), _starts(rows), sum(rows)
    st["longest"], st["most"] = max(lens), max(rows)
    if case["op"] == "store":
        who, place = _rows(added)
        pos = torch.tensor(cached, device=DEV)[who] + place
        slots = (st["table"][who, pos // t].long() * t + pos % t).to(torch.int32)
        pad = torch.full((case["pad"],), -1, dtype=torch.int32, device=DEV)
        st["slots"] = torch.cat([slots, pad])
        # as projections give them: one fused row per token, a few loud channels in the keys
        kv = torch.randn(who.numel() + case["pad"], 2 * h, d, generator=g, device=DEV)
        loud = 1 + 6 * (torch.rand(h, d, generator=g, device=DEV) > 0.97)
        kv[:, :h] *= loud
        st["kv"] = kv.to(dtype)
        st["key"], st["value"] = st["kv"][:, :h], st["kv"][:, h:]
    elif case["op"] == "attend":
        # what stands behind a request's last token is not a number
        k, v, s = _views4(st["pool"], h, d, t)
        tail = [i for i, x in enumerate(lens) if x % t]
        if tail:
            last = st["table"][torch.tensor(tail, device=DEV),
                               torch.tensor([used[i] - 1 for i in tail], device=DEV)].long()
            keep = torch.tensor([lens[i] % t for i in tail], device=DEV)
            gone = torch.arange(t, device=DEV)[None, :] >= keep[:, None]
            s[last] = torch.where(gone[:, None, None, None, :], 255, s[last])
        st["query"] = torch.randn(st["rows"], case["heads"], d, generator=g, device=DEV).to(dtype)
    if own:
        from recv_fifo_plane_amd import PagedCache
        st["cache"] = PagedCache(total, t, h, d, buffer=st["pool"], bits=case.get("bits", 4))
    return st


# --------------------------------------------------------------------- run
def run(st):
    case = st["case"]
    if case["op"] == "store":
        if own:
            st["cache"].store(st["key"], st["value"], st["slots"])
            key, value = st["cache"].load(st["table"], st["lengths"], st["starts"], st["rows"],
                                          dtype=st["key"].dtype)
            return dict(key=key, value=value)
        _plain_store(st)
        return _plain_load(st)
    if case["op"] == "load":
        if own:
            key, value = st["cache"].load(st["table"], st["lengths"], st["starts"], st["rows"],
                                          dtype=DTYPES[case["dtype"]])
            return dict(key=key, value=value)
        return _plain_load(st)
    if own:
        out, lse = st["cache"].attend(st["query"], st["table"], st["lengths"], st["starts"],
                                      max_query=st["most"], max_length=st["longest"], lse=True)
        return dict(out=out, lse=lse)
    return _plain_attend(st)


def _pair(codes):
    """Codes of even and odd dims as bytes."""
    return codes[..., 0::2] | codes[..., 1::2] << 4


def _plain_store(st):
    case = st["case"]
    t, h, d = case["block"], case["kv_heads"], case["dim"]
    k, v, s = _views4(st["pool"], h, d, t)
    n = st["rows"]                                      # (the rows behind have no slot)
    slots = st["slots"][:n].long()
    blk, off = slots // t, slots % t
    scales = []
    for side, x in enumerate((st["key"], st["value"])):
        x = x[:n].float().reshape(n, h, d // 32, 32)
        fine = torch.isfinite(x).all(-1)
        x = torch.where(fine[..., None], x, 0.0)
        m, e = torch.frexp(x.abs().amax(-1))            # 0.5 <= m < 1; 7 = 0.875 * 2^3
        e = torch.where(m > 0.875, e - 2, e - 3)
        e = torch.where(m > 0, e, -118).clamp(-118, 125)
        # (in two steps: 2^118 times the largest number would pass a float's range on the way)
        y = torch.ldexp(torch.ldexp(x, -(e // 2)[..., None]), -(e - e // 2)[..., None])
        a = y.abs()
        code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
                + (a >= 3.5) + (a > 5.0)).to(torch.uint8)
        code = torch.where(torch.signbit(y), code | 8, code).reshape(n, h, d)
        packed = _pair(code)
        if side == 0:
            k[blk, :, off] = packed
        else:
            for (at, dims), part in zip(_parts(d), v):
                b = dims // 32
                u = 16 // b
                part[blk, :, off // u, :, off % u] = (
                    packed[..., at // 2:(at + dims) // 2].reshape(n, h, 16, b))
        scales.append(torch.where(fine, e + 127, 255).to(torch.uint8))
    s[blk, :, :, :, off] = torch.stack(scales, 2)


def _tokens4(case, pool, blk, off):
    """float32 keys and values [tokens, H, D] of a pool of 4 bits."""
    t, h, d = case["block"], case["kv_heads"], case["dim"]
    k, v, s = _views4(pool, h, d, t)
    n = blk.numel()
    half = torch.tensor(MAGNITUDES + tuple(-x for x in MAGNITUDES), device=DEV)
    both = torch.stack([half.repeat(16), half.repeat_interleave(16)], 1)     # of a byte's codes
    scale = s[blk, :, :, :, off]                                             # [n, H, 2, D / 32]
    power = torch.where(scale == 255, float("nan"), torch.exp2(scale.float() - 127))
    keys = k[blk, :, off]
    vals = torch.cat([part[blk, :, off // part.shape[4], :, off % part.shape[4]].reshape(n, h, -1)
                      for part in v], -1)
    return [(both[x.long()].reshape(n, h, d // 32, 32) * power[:, :, i, :, None]).reshape(n, h, d)
            for i, x in enumerate((keys, vals))]


def _tokens8(case, pool, blk, off):
    t, h, d = case["block"], case["kv_heads"], case["dim"]
    k, v, s = _views8(pool, h, d, t)
    codes = (k.view(torch.uint8)[blk, :, off], v.view(torch.uint8)[blk, :, :, off])
    return [x.view(torch.float8_e4m3fn).float() * s[blk][:, :, i, None] for i, x in enumerate(codes)]


def _plain_load(st):
    case, t = st["case"], st["case"]["block"]
    lens, starts = st["lengths"].long(), st["starts"].long()
    row = torch.arange(st["rows"], device=DEV)
    who = torch.searchsorted(starts[1:], row, right=True)
    pos = lens[who] - (starts[who + 1] - row)
    tokens = _tokens8 if case.get("bits") == 8 else _tokens4
    key, value = tokens(case, st["pool"], st["table"][who, pos // t].long(), pos % t)
    dtype = DTYPES[case["dtype"]]
    return dict(key=key.to(dtype), value=value.to(dtype))


def _plain_attend(st):
    case = st["case"]
    t, h, d, heads = case["block"], case["kv_heads"], case["dim"], case["heads"]
    lens, starts = st["lengths"].long(), st["starts"].long()
    b, group = lens.numel(), heads // h
    pages = -(-st["longest"] // t)
    ids = st["table"][:, :pages].long()
    good = ids >= 0
    ids = ids.clamp(min=0)
    pos = torch.arange(pages * t, device=DEV)
    keys, vals = _tokens4(case, st["pool"], ids[:, pos // t].reshape(-1), (pos % t).repeat(b))
    there = (pos[None, :] < lens[:, None]) & good.repeat_interleave(t, 1)   # [b, L]
    keys, vals = (torch.where(there[:, None, :, None],
                              x.reshape(b, -1, h, d).permute(0, 2, 1, 3), 0.0) for x in (keys, vals))
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
    h, d, t = case["kv_heads"], case["dim"], case["block"]
    size = 4 if case["dtype"] == "fp32" else 2
    token = h * (d + d // 16)                           # bytes of a token in 4 bits, both sides
    if case["op"] == "store":
        n = sum(_growth(case)[1])
        blocks = sum(-(-(c + a) // t) for c, a in zip(*_growth(case)))
        return dict(bytes=n * (2 * (2 * h * d * size + token) + 4) + 4 * blocks, flops=0)
    lens, rows = _reach(case)
    blocks = sum(-(-x // t) for x in lens)
    n = sum(rows)
    if case["op"] == "load":
        held = n * 2 * h * d + 8 * h * blocks if case["bits"] == 8 else n * token
        return dict(bytes=held + n * 2 * h * d * size + 4 * blocks, flops=0)
    heads = case["heads"]
    pairs = sum(sum(max(0, x - r + j + 1) for j in range(r)) for x, r in zip(lens, rows))
    return dict(bytes=token * sum(lens) + 4 * blocks + n * heads * (2 * d * size + 4),
                flops=4 * d * heads * pairs)


# ------------------------------------------------------------------- exact
def exact(case, seed):
    global own
    kept, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = kept
    if case["op"] == "store":
        return _exact_store(st)
    return _exact_load(st) if case["op"] == "load" else _exact_attend(st)


def _exact_store(st):
    """What is held for each row: the nearest of a code's sixteen numbers, as many
    times 2^e as the 32 dims' largest magnitude asks for."""
    case = st["case"]
    d, n = case["dim"], st["rows"]
    levels = torch.tensor(MAGNITUDES, dtype=torch.float64, device=DEV)
    odd = torch.tensor([0, 1] * 4, dtype=torch.float64, device=DEV)
    out = {}
    for name in ("key", "value"):
        x = st[name][:n].double().reshape(n, -1, 32)
        held = torch.empty_like(x)
        step = max(1, (8 << 20) // x[0].numel())
        for i in range(0, n, step):
            y = x[i:i + step]
            e = torch.ceil(torch.log2(y.abs().amax(-1).clamp(min=1e-300) / 7)).clamp(-118, 125)
            e = torch.where(y.abs().amax(-1) > 7 * torch.exp2(e), e + 1, e)
            e = torch.where(y.abs().amax(-1) <= 7 * torch.exp2(e - 1), e - 1, e).clamp(-118, 125)
            scale = torch.exp2(e)[..., None]
            far = ((y / scale).abs()[..., None] - levels).abs()
            near = (far + 1e-9 * odd).argmin(-1)        # of two as near, the even code
            held[i:i + step] = levels[near] * torch.sign(y) * scale
        out[name] = held.reshape(n, -1, d)
    return out


def _records(st, i, j, side):
    """float64 [tokens, D] of request i's blocks and head j, the keys (side 0) or values."""
    case = st["case"]
    t, h, d = case["block"], case["kv_heads"], case["dim"]
    ids = st["table"][i, :-(-int(st["lengths"][i]) // t)].long()
    if case.get("bits") == 8:
        k, v, s = _views8(st["pool"], h, d, t)
        x = (k if side == 0 else v)[:, j].view(torch.uint8)[ids].view(torch.float8_e4m3fn).double()
        x = x if side == 0 else x.transpose(1, 2)
        return (x * s[ids, j, side].double()[:, None, None]).reshape(-1, d)
    raw = st["pool"][ids]
    body = raw[:, j * t * d:(j + 1) * t * d].reshape(len(ids), 2, t * d // 2)[:, side]
    if side == 0:
        codes = body.reshape(-1, t, d // 2)
    else:
        codes, at = [], 0
        for _, dims in _parts(d):
            b = dims // 32
            piece = body[:, at:at + t * dims // 2].reshape(-1, b * t // 16, 16, 16 // b, b)
            codes.append(piece.permute(0, 1, 3, 2, 4).reshape(-1, t, dims // 2))
            at += t * dims // 2
        codes = torch.cat(codes, -1)
    codes = torch.stack([codes & 15, codes >> 4], -1).reshape(-1, t, d // 32, 32)
    e, m = ((codes >> 1) & 3).double(), (codes & 1).double()
    x = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2(e - 1)) * (1 - 2 * (codes >> 3).double())
    g = d // 32
    at = h * t * d + (2 * j + side) * g * t
    s = raw[:, at:at + g * t].reshape(-1, g, t).transpose(1, 2)
    s = torch.where(s == 255, float("nan"), torch.exp2(s.double() - 127))
    return (x * s[..., None]).reshape(-1, d)


def _exact_load(st):
    case = st["case"]
    h, d = case["kv_heads"], case["dim"]
    lens, starts = st["lengths"].tolist(), st["starts"].tolist()
    out = [torch.empty(st["rows"], h, d, dtype=torch.float64, device=DEV) for _ in range(2)]
    for i, length in enumerate(lens):
        r = starts[i + 1] - starts[i]
        for j in range(h):
            for side in range(2):
                out[side][starts[i]:starts[i + 1], j] = _records(st, i, j, side)[length - r:length]
    return dict(key=out[0], value=out[1])


def _exact_attend(st):
    case = st["case"]
    h, d, heads = case["kv_heads"], case["dim"], case["heads"]
    lens, starts = st["lengths"].tolist(), st["starts"].tolist()
    n, group = starts[-1], heads // h
    out = torch.zeros(n, heads, d, dtype=torch.float64, device=DEV)
    lse = torch.full((n, heads), float("-inf"), dtype=torch.float64, device=DEV)
    for i, length in enumerate(lens):
        first, end = starts[i], starts[i + 1]
        for j in range(h):
            keys, vals = (_records(st, i, j, side)[:length] for side in range(2))
            mine = slice(j * group, (j + 1) * group)
            step = max(1, (64 << 20) // (group * max(length, 1)))
            for r0 in range(first, end, step):
                r1 = min(end, r0 + step)
                limit = length - (end - first) + torch.arange(r0 - first, r1 - first, device=DEV)
                seen = torch.arange(length, device=DEV)[None, :] <= limit[:, None]
                q = st["query"][r0:r1, mine].double()
                x = (q.reshape(-1, d) @ keys.T).reshape(r1 - r0, -1, length) / math.sqrt(d)
                x = torch.where(seen[:, None, :], x, float("-inf"))
                z = torch.logsumexp(x, -1)
                lse[r0:r1, mine] = z
                p = torch.exp(x - torch.where(torch.isfinite(z), z, 0.0)[..., None])
                out[r0:r1, mine] = (p.reshape(-1, length) @ vals).reshape(r1 - r0, group, d)
    return dict(out=out, lse=lse)
