"""A paged cache of keys and values in 8 or 4 bits, whose blocks a connection moves.

The endpoint that runs a prompt plans room for its tokens (plan_blocks), stores
their keys and values (PagedCache.store) and sends the blocks
(PagedCache.send); the endpoint that answers attends to them
(PagedCache.attend), or reads them back as rows (PagedCache.load).  Argument checks
and marshalling only: the work is that of the library's HIP kernels (xfer_cache_*,
xfer_mxcache_* and xfer_run_blocks in include/xfer.h).
"""
from __future__ import annotations

import ctypes as C
import math
from collections import namedtuple

from . import xfer as X

BlockPlan = namedtuple("BlockPlan", "slots positions starts lengths counts")
BlockPlan.__doc__ = """Where the next tokens of a batch go (int32 tensors).

slots[rows]: cache slot of each packed row, -1 where there is none; positions[rows]:
the token's place in its request; starts[batch + 1]: first row of each request;
lengths[batch]: tokens of each request with the new ones; counts[2]: new blocks
needed, and tokens left without a slot."""

BLOCK_TOKENS = (16, 32, 64)
HEAD_DIMS = (64, 96, 128, 192, 256)


_KINDS = {}  # torch dtypes of rows to xfer_dtype, filled at the first call
_INT32 = _FLOAT32 = _UINT8 = None
_GRAD = None  # whether gradients are being recorded
_RAW = None  # the current stream's handle of a device, where torch gives it without an object


def _kinds():
    global _INT32, _FLOAT32, _UINT8, _RAW, _GRAD
    if not _KINDS:
        import torch
        _INT32, _FLOAT32, _UINT8 = torch.int32, torch.float32, torch.uint8
        _GRAD = torch.is_grad_enabled
        _RAW = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _KINDS.update({torch.bfloat16: 0, torch.float16: 1, torch.float32: 2})
    return _KINDS


_MOST = 0x7FFFFFFF  # the library's sizes are C ints, which would drop what lies above


def _int(v, what):
    v = int(v)
    if not -_MOST - 1 <= v <= _MOST:
        raise ValueError("%s: %d is not within 2^31" % (what, v))
    return v


def _tensor(t, what, dtypes, ndim, device):
    """A GPU tensor of one of `dtypes` with `ndim` dimensions on `device` (None: any)."""
    if not hasattr(t, "data_ptr"):
        raise TypeError("%s: expected a torch tensor, got %s" % (what, type(t).__name__))
    if not t.is_cuda:
        raise ValueError("%s: tensor is not in GPU memory (device %s)" % (what, t.device))
    if device is not None and t.device.index != device:
        raise ValueError("%s: tensor is on cuda:%s, not on cuda:%d" % (what, t.device.index, device))
    if t.dtype not in dtypes:
        raise TypeError("%s: unsupported dtype %s" % (what, t.dtype))
    if t.dim() != ndim:
        raise ValueError("%s: expected %d dimensions, got shape %s" % (what, ndim, tuple(t.shape)))
    return t


def _list(t, what, n, device):
    """Address of a contiguous int32 tensor of n entries (None: any number)."""
    try:  # the usual case, in few calls
        if (t.dtype is _INT32 and t.is_cuda and (device is None or t.get_device() == device)
                and t.dim() == 1 and t.is_contiguous() and (n is None or t.shape[0] == n)
                and t.shape[0] <= _MOST):
            return t.data_ptr()
    except AttributeError:
        pass
    _tensor(t, what, (_INT32,), 1, device)
    have = t.shape[0]
    if n is not None and have != n:
        raise ValueError("%s: expected %d entries, got %d" % (what, n, have))
    _int(have, what)
    raise ValueError("%s: tensor is not contiguous" % what)


def _table(t, what, batch, device):
    """Address, row stride and width of a block table [batch, width]: any row
    stride of at least the width."""
    _tensor(t, what, (_INT32,), 2, device)
    have, width = t.shape
    if have != batch:
        raise ValueError("%s: expected %d rows, got %d" % (what, batch, have))
    if width > _MOST:
        _int(width, what)
    stride = t.stride(0) if batch > 1 else width
    if (width > 1 and t.stride(1) != 1) or stride < width:
        raise ValueError("%s: rows must be contiguous and not overlap" % what)
    return t.data_ptr(), stride, width


def _rows(t, what, dtypes, device, rows, heads, dim):
    """Address and strides of rows [rows, heads, dim] with a contiguous last dimension."""
    _tensor(t, what, dtypes, 3, device)
    if t.shape != (rows, heads, dim):
        raise ValueError("%s must have shape (%d, %d, %d), got %s"
                         % (what, rows, heads, dim, tuple(t.shape)))
    row, head, last = t.stride()
    if last != 1:
        raise ValueError("%s: the last dimension must be contiguous" % what)
    return t.data_ptr(), row, head


def _on(stream, device):
    """Refuses a stream object of another device (a handle does not tell)."""
    own = getattr(stream, "device", None)
    if own is not None and own.index != device:
        raise ValueError("stream is of %s, the tensors are on cuda:%d" % (own, device))


def _no_grad(what):
    """Refuses a tensor that requires a gradient, which would be lost."""
    if _GRAD():
        raise ValueError("%s: there is no gradient of attention over the cache; call it under "
                         "torch.no_grad() or with a detached tensor" % what)


def _call(device, stream, fn, *args):
    """fn(*args, stream) with the tensors' device current."""
    import torch
    if stream is not None:
        _on(stream, device)
    if device == torch.cuda.current_device():
        rc = fn(*args, _RAW(device) or None if stream is None and _RAW else X._stream_handle(stream))
    else:
        with torch.cuda.device(device):
            rc = fn(*args, X._stream_handle(stream))
    if rc:
        X.check(rc)


def _side(stream, device):
    """The stream that a call launches on, None where it is the current one of
    `device`.  A handle is one of a stream of `device`."""
    if stream is None:
        return None
    import torch
    _on(stream, device)
    if not isinstance(stream, torch.cuda.Stream):
        handle = X._stream_handle(stream)
        stream = (torch.cuda.ExternalStream(handle, device=device) if handle
                  else torch.cuda.default_stream(device))
    return None if stream == torch.cuda.current_stream(device) else stream


def _empty(like, shape, dtype, side, result=True):
    """A new tensor that a launch on the stream `side` writes (None: the current one,
    where callers in a hurry call new_empty themselves).

    It comes from that stream's pool: the current stream's could hold memory
    that was freed there while kernels still queued use it, and a launch on
    another stream does not wait for those.  A result, which the caller goes on
    to use on the current stream, stays reserved for that one too."""
    if side is None:
        return like.new_empty(shape, dtype=dtype)
    import torch
    here = torch.cuda.current_stream(like.device.index)
    with torch.cuda.stream(side):
        t = like.new_empty(shape, dtype=dtype)
    if result:
        t.record_stream(here)
    return t


def plan_blocks(cached, added, table, free, block_tokens: int, rows: int, out=None,
                stream=None) -> BlockPlan:
    """Room for the next tokens of a batch, worked out on the GPU.

    Request i has cached[i] tokens and adds added[i]; its row of `table`
    [batch, width] is extended in place by the blocks that it needs, taken from
    `free` in order.  All int32 tensors.  rows: length of the packed rows'
    outputs (the batch's added tokens, or more where it is padded).  out: a
    BlockPlan to write into (a captured graph's), else new tensors."""
    _kinds()
    at_cached = _list(cached, "plan_blocks: cached", None, None)
    dev, batch = cached.device.index, cached.shape[0]
    at_added = _list(added, "plan_blocks: added", batch, dev)
    at_table, stride, width = _table(table, "plan_blocks: table", batch, dev)
    at_free = _list(free, "plan_blocks: free", None, dev)
    block_tokens, rows = int(block_tokens), int(rows)
    if rows < 0:
        raise ValueError("plan_blocks: rows must not be negative")
    if rows > _MOST or not 0 <= block_tokens <= _MOST:
        _int(rows, "plan_blocks: rows")
        _int(block_tokens, "plan_blocks: block_tokens")
    sizes = (rows, rows, batch + 1, batch, 2)
    if out is None:
        buf = (cached.new_empty(sum(sizes)) if stream is None
               else _empty(cached, sum(sizes), _INT32, _side(stream, dev)))
        out = BlockPlan(*buf.split_with_sizes(sizes))
        slots = buf.data_ptr()
        positions = slots + 4 * rows
        starts = positions + 4 * rows
        lengths = starts + 4 * (batch + 1)
        counts = lengths + 4 * batch
    else:
        slots, positions, starts, lengths, counts = (
            _list(t, "plan_blocks: out", n, dev) for t, n in zip(out, sizes))
    _call(dev, stream, X.lib().xfer_cache_plan, at_cached, at_added, batch, at_table, stride, width,
          at_free, free.shape[0], block_tokens, slots, positions, rows, starts, lengths,
          counts)
    return out


_Names = namedtuple("_Names", "block_bytes store load attend_workspace attend")


class PagedCache:
    """A pool of cache blocks in GPU memory: uint8 [blocks, block_bytes]."""

    bits = 8
    # The library's functions for codes of 8 and of 4 bits.
    _NAMES = {bits: _Names(*("xfer_%s_%s" % (kind, name) for name in _Names._fields))
              for bits, kind in ((8, "cache"), (4, "mxcache"))}

    def __init__(self, blocks: int, block_tokens: int, kv_heads: int, head_dim: int, device=None,
                 buffer=None, bits: int = 8):
        """buffer: a contiguous uint8 tensor [blocks, block_bytes] to use, else zeros.

        bits: 8 holds e4m3 numbers with a scale per block and head, 4 holds e2m1
        numbers with a scale per token, head and 32 dims (half the bytes)."""
        import torch
        if bits not in self._NAMES:
            raise ValueError("PagedCache: bits must be 8 or 4, got %r" % (bits,))
        self.bits = int(bits)
        self.blocks, self.block_tokens, self.kv_heads, self.head_dim = (
            _int(v, "PagedCache: " + what) for v, what in
            ((blocks, "blocks"), (block_tokens, "block_tokens"), (kv_heads, "kv_heads"),
             (head_dim, "head_dim")))
        self._shape = X.xfer_cache_shape(self.block_tokens, self.kv_heads, self.head_dim,
                                         self.blocks)
        n = C.c_size_t()
        X.check(getattr(X.lib(), self._NAMES[self.bits].block_bytes)(C.byref(self._shape), C.byref(n)))
        self.block_bytes = n.value
        if buffer is None:
            buffer = torch.zeros(self.blocks, self.block_bytes, dtype=torch.uint8,
                                 device="cuda" if device is None else device)
        _tensor(buffer, "PagedCache: buffer", (torch.uint8,), 2, None)
        if tuple(buffer.shape) != (self.blocks, self.block_bytes):
            raise ValueError("PagedCache: buffer must have shape (%d, %d), got %s"
                             % (self.blocks, self.block_bytes, tuple(buffer.shape)))
        if not buffer.is_contiguous() or buffer.data_ptr() % 16:
            raise ValueError("PagedCache: buffer must be contiguous and 16-byte aligned")
        self.buffer = buffer
        self.device = buffer.device.index
        self._ref, self._base = C.byref(self._shape), buffer.data_ptr()

    def _of_8_bits(self, what):
        if self.bits != 8:
            raise ValueError("%s: codes of 4 bits share bytes, and their scales are a token's own; "
                             "load() gives what they stand for" % what)

    def _view(self, dtype, shape, strides, at):
        b = self.buffer.view(dtype)
        return b.as_strided(shape, strides, b.storage_offset() + at)

    def keys(self):
        """Key codes, float8_e4m3fn [blocks, kv_heads, block_tokens, head_dim] (a view; 8 bits)."""
        self._of_8_bits("keys")
        import torch
        h, t, d = self.kv_heads, self.block_tokens, self.head_dim
        return self._view(torch.float8_e4m3fn, (self.blocks, h, t, d),
                          (self.block_bytes, 2 * t * d, d, 1), 0)

    def values(self):
        """Value codes, float8_e4m3fn [blocks, kv_heads, block_tokens, head_dim] (a view; 8 bits)."""
        self._of_8_bits("values")
        import torch
        h, t, d = self.kv_heads, self.block_tokens, self.head_dim
        return self._view(torch.float8_e4m3fn, (self.blocks, h, t, d),
                          (self.block_bytes, 2 * t * d, 1, t), t * d)

    def scales(self):
        """Scales of keys and values, float32 [blocks, kv_heads, 2] (a view; 8 bits)."""
        self._of_8_bits("scales")
        import torch
        h, t, d = self.kv_heads, self.block_tokens, self.head_dim
        return self._view(torch.float32, (self.blocks, h, 2), (self.block_bytes // 4, 2, 1),
                          2 * h * t * d // 4)

    def store(self, key, value, slots, stream=None) -> None:
        """Stores rows of keys and values [rows, kv_heads, head_dim] (bfloat16,
        float16 or float32; any strides of rows and heads) into their slots."""
        kinds = _kinds()
        _tensor(key, "store: key", kinds, 3, self.device)
        rows, dtype = key.shape[0], key.dtype
        k, k_row, k_head = _rows(key, "store: key", kinds, self.device, rows, self.kv_heads,
                                 self.head_dim)
        v, v_row, v_head = _rows(value, "store: value", (dtype,), self.device, rows, self.kv_heads,
                                 self.head_dim)
        at = _list(slots, "store: slots", rows, self.device)
        _call(self.device, stream, getattr(X.lib(), self._NAMES[self.bits].store), self._ref,
              self._base, k, k_row, k_head, v, v_row, v_head, kinds[dtype], at, rows)

    def load(self, table, lengths, starts, rows: int, dtype=None, out=None, stream=None):
        """Keys and values of the cache's tokens as packed rows [rows, kv_heads,
        head_dim] (bfloat16, float16 or float32; bfloat16 if dtype is None).

        Request b has the rows starts[b] .. starts[b + 1) and lengths[b] tokens, of
        which those rows are the last, as in attend: a plan's starts give the
        tokens that it added, sums of the lengths whole contexts.  table: int32
        [batch, width].  out: (key, value) to write into (any strides of rows and
        heads, but no memory in common), else new tensors.  Tokens that the table
        lacks give 0; rows of no request are left as they were (without `out`: undefined)."""
        kinds = _kinds()
        rows = int(rows)
        if rows < 0:
            raise ValueError("load: rows must not be negative")
        if rows > _MOST:
            _int(rows, "load: rows")
        at_lengths = _list(lengths, "load: lengths", None, self.device)
        batch = lengths.shape[0]
        at_starts = _list(starts, "load: starts", batch + 1, self.device)
        at_table, stride, width = _table(table, "load: table", batch, self.device)
        shape = (rows, self.kv_heads, self.head_dim)
        if dtype is not None and dtype not in kinds:
            raise TypeError("load: unsupported dtype %s" % (dtype,))
        if out is None:
            if dtype is None:
                import torch
                dtype = torch.bfloat16
            side = None if stream is None else _side(stream, self.device)
            out = tuple(self.buffer.new_empty(shape, dtype=dtype) if side is None
                        else _empty(self.buffer, shape, dtype, side) for _ in range(2))
        else:
            if len(out) != 2:
                raise ValueError("load: out must be a key and a value tensor")
            for t in out:
                if getattr(t, "requires_grad", False) and _GRAD():
                    raise ValueError("load: out requires a gradient; there is none of what is read")
        key, value = out
        k, k_row, k_head = _rows(key, "load: out key", kinds if dtype is None else (dtype,),
                                 self.device, *shape)
        v, v_row, v_head = _rows(value, "load: out value", (key.dtype,), self.device, *shape)
        a = X.xfer_load(k, v, at_table, at_lengths, at_starts, k_row, k_head, v_row, v_head, stride,
                        batch, rows, width, kinds[key.dtype])
        _call(self.device, stream, getattr(X.lib(), self._NAMES[self.bits].load), self._ref,
              self._base, C.byref(a))
        return key, value

    def attend(self, query, table, lengths, starts, scale=None, out=None, lse=False, max_query=0,
               max_length=0, stream=None):
        """Attention of packed query rows [rows, heads, head_dim] (bfloat16 or
        float16) over the cache; returns out, or (out, lse) with lse=True.

        Request b has the rows starts[b] .. starts[b + 1) and lengths[b] tokens,
        its rows' own included; row j of r sees tokens 0 .. lengths[b] - r + j.
        table: int32 [batch, width].  scale: 1 / sqrt(head_dim) if None.
        max_query, max_length: the batch's largest number of rows and of
        tokens, where known; they shape the launch only.  Rows of no request
        are left as they were (without `out`: undefined).  out must not share
        memory with query.  There is no gradient: where one is being recorded,
        a query or out that requires it is refused."""
        kinds = _kinds()
        _tensor(query, "attend: query", kinds, 3, self.device)
        if getattr(query, "requires_grad", False):
            _no_grad("attend: query")
        rows, heads, d = query.shape
        dtype = query.dtype
        if kinds[dtype] == 2:
            raise TypeError("attend: query: unsupported dtype %s" % dtype)
        q, q_row, q_head = _rows(query, "attend: query", kinds, self.device, rows, heads,
                                 self.head_dim)
        at_lengths = _list(lengths, "attend: lengths", None, self.device)
        batch = lengths.shape[0]
        at_starts = _list(starts, "attend: starts", batch + 1, self.device)
        at_table, stride, width = _table(table, "attend: table", batch, self.device)
        max_query, max_length = int(max_query), int(max_length)
        if not (0 <= max_query <= _MOST and 0 <= max_length <= _MOST):
            _int(max_query, "attend: max_query")
            _int(max_length, "attend: max_length")
        side = None if stream is None else _side(stream, self.device)
        if out is None:
            out = (query.new_empty((rows, heads, d)) if side is None
                   else _empty(query, (rows, heads, d), dtype, side))
        elif getattr(out, "requires_grad", False):
            _no_grad("attend: out")
        o, o_row, o_head = _rows(out, "attend: out", (dtype,), self.device, rows, heads, d)
        sums = None
        if lse is True:
            sums = (query.new_empty((rows, heads), dtype=_FLOAT32) if side is None
                    else _empty(query, (rows, heads), _FLOAT32, side))
        elif lse is not False and lse is not None:
            sums = _tensor(lse, "attend: lse", (_FLOAT32,), 2, self.device)
            if tuple(sums.shape) != (rows, heads) or not sums.is_contiguous():
                raise ValueError("attend: lse must be contiguous of shape (%d, %d)" % (rows, heads))
        a = X.xfer_attend(q, o, None if sums is None else sums.data_ptr(), at_table, at_lengths,
                          at_starts, None, 0, q_row, q_head, o_row, o_head, stride, batch, rows,
                          heads, width, kinds[dtype],
                          1.0 / math.sqrt(d) if scale is None else float(scale), max_query,
                          max_length)
        n, ref, lib, names = C.c_size_t(), C.byref(a), X.lib(), self._NAMES[self.bits]
        rc = getattr(lib, names.attend_workspace)(self._ref, ref, C.byref(n))
        if rc:
            X.check(rc)
        if n.value:
            work = (query.new_empty(n.value, dtype=_UINT8) if side is None
                    else _empty(query, n.value, _UINT8, side, result=False))
            a.workspace, a.workspace_bytes = work.data_ptr(), n.value
        _call(self.device, stream, getattr(lib, names.attend), self._ref, self._base, ref)
        return out if sums is None else (out, sums)

    def send(self, conn, dst, src_ids, dst_ids, stream=None) -> None:
        """Moves block src_ids[i] of this cache to block dst_ids[i] of the cache
        `dst` over a connection (as Conn.run_blocks does): int32 lists in GPU memory."""
        mine = (self.block_tokens, self.kv_heads, self.head_dim)
        other = (dst.block_tokens, dst.kv_heads, dst.head_dim)
        if self.bits != dst.bits:
            raise ValueError("send: blocks of %d bits cannot go into a cache of %d"
                             % (self.bits, dst.bits))
        if mine != other:
            raise ValueError("send: blocks of shape %s cannot go into blocks of shape %s"
                             % (mine, other))
        _kinds()
        if not self.device == dst.device == conn.device:
            raise ValueError("send: caches on cuda:%s and cuda:%s, the connection on cuda:%s"
                             % (self.device, dst.device, conn.device))
        a = _list(src_ids, "send: src_ids", None, self.device)
        n = src_ids.shape[0]
        b = _list(dst_ids, "send: dst_ids", n, self.device)
        _call(self.device, stream, X.lib().xfer_run_blocks, conn.handle, self._base, self.blocks,
              dst._base, dst.blocks, self.block_bytes, a, b, n)
