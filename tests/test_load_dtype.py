"""CPU tests of the types that a cache is read back in: a wrong one is named as such, with and without
outputs of it."""
import pytest
import torch

from test_cache_refusals import FakeTensor
from test_mxcache_refusals import cache  # noqa: F401 (a fixture)


@pytest.mark.parametrize("dtype", [torch.int8, torch.float64, torch.int32, torch.uint8, torch.float8_e4m3fn, "bf16", 2])
@pytest.mark.parametrize("given", [False, True])
def test_unsupported_types_are_refused(cache, dtype, given):  # noqa: F811
    kind = dtype if isinstance(dtype, torch.dtype) else torch.bfloat16
    out = tuple(FakeTensor((6, 2, 128), kind, ptr=(1 << 40) + i * (1 << 20)) for i in range(2)) if given else None
    with pytest.raises(TypeError, match="unsupported dtype"):
        cache.load(FakeTensor((3, 8)), FakeTensor((3,)), FakeTensor((4,)), 6, dtype=dtype, out=out)
