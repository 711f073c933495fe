"""What a cache is read back into: outputs that overlap one another are refused before anything is
launched (on the CPU), those that only lie between one another are written (on a GPU)."""
import ctypes as C

import numpy as np
import pytest
import torch

import recv_fifo_plane_amd as xf
from recv_fifo_plane_amd import xfer as X
from test_cache_refusals import INVALID, P, _shape
from test_mxcache_refusals import _load

NAMES = ["xfer_cache_load", "xfer_mxcache_load"]
KEY = P + (1 << 30)
H, D = 2, 128
LAYOUTS = [(256, 128), (512, 128), (512, 256), (520, 130), (128, 4096), (-512, 128), (512, -128), (300, 900)]
APART = [0, 1, -1, 64, -127, 127, 128, -128, 256, -256, 300, 390, 512, -600, 900, 1100, 4096, -4224]


def touched(at, row, head, rows):
    return {at + r * row + h * head + d for r in range(rows) for h in range(H) for d in range(D)}


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("row,head", LAYOUTS)
def test_overlaps_are_refused(name, row, head):
    """The value's rows [3, H, D] lie as the key's do, some elements on."""
    for dtype, size in ((0, 2), (2, 4)):
        for at in APART:
            if not touched(0, row, head, 3) & touched(at, row, head, 3):
                continue
            a = _load(key=KEY, value=KEY + size * at, rows=3, dtype=dtype, key_row=row, value_row=row,
                      key_head=head, value_head=head)
            assert getattr(X.lib(), name)(C.byref(_shape(h=H, d=D)), P, C.byref(a), None) == INVALID, at
            assert "overlap" in xf.last_error() and xf.last_error().startswith(name)


@pytest.mark.parametrize("name", NAMES)
def test_overlaps_of_single_rows_and_heads(name):
    """Strides of a dimension of one say nothing."""
    for kw in (dict(rows=1, key_row=5, value_row=7), dict(rows=1, key_row=0, value_row=-9, value=KEY + 2 * 255)):
        a = _load(**dict(dict(key=KEY, value=KEY), **kw))
        assert getattr(X.lib(), name)(C.byref(_shape()), P, C.byref(a), None) == INVALID
        assert "overlap" in xf.last_error()
    a = _load(key=KEY, value=KEY + 2 * 200, rows=2, key_head=3, value_head=4, key_row=128, value_row=128)
    assert getattr(X.lib(), name)(C.byref(_shape(h=1)), P, C.byref(a), None) == INVALID
    assert "overlap" in xf.last_error()


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 8])
def test_outputs_between_one_another(bits):
    """Every layout above whose rows lie between one another, and the usual fused ones."""
    cache = xf.PagedCache(4, 16, H, D, bits=bits)
    rng = np.random.default_rng(bits)
    rows = torch.tensor(rng.normal(0, 1, (2, 3, H, D)), dtype=torch.float32, device="cuda")
    slots = torch.tensor([17, 18, 19], dtype=torch.int32, device="cuda")
    cache.store(rows[0], rows[1], slots)
    table = torch.tensor([[1]], dtype=torch.int32, device="cuda")
    lengths = torch.tensor([4], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    want = cache.load(table, lengths, starts, 3, dtype=torch.float32)
    done = 0
    for row, head in LAYOUTS:
        if row < 0 or head < 0:
            continue
        for at in APART:
            if touched(0, row, head, 3) & touched(at, row, head, 3):
                continue
            base = torch.full((1 << 15,), 7.0, device="cuda")
            out = [base.as_strided((3, H, D), (row, head, 1), 8192 + x) for x in (0, at)]
            cache.load(table, lengths, starts, 3, out=out)
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]), (row, head, at)
            assert int((base != 7.0).sum()) <= 2 * 3 * H * D
            done += 1
    assert done == 23
    for fused, key, value in ((torch.zeros(3, 2 * H, D, device="cuda"), np.s_[:, :H], np.s_[:, H:]),
                              (torch.zeros(3, H, 2 * D, device="cuda"), np.s_[..., :D], np.s_[..., D:]),
                              (torch.zeros(2, 3, H, D, device="cuda"), np.s_[0], np.s_[1])):
        cache.load(table, lengths, starts, 3, out=(fused[key], fused[value]))
        assert torch.equal(fused[key], want[0]) and torch.equal(fused[value], want[1])
