"""CPU test of the compiled 4-bit cache kernels' resources: none may use scratch
(stack) memory, which would put a memory round trip into their inner loops."""
import pytest

from test_kernel_resources import test_no_kernel_uses_scratch as check


@pytest.mark.parametrize("name", ["mxcache.hip"])
def test_no_mxcache_kernel_uses_scratch(name):
    check(name)
