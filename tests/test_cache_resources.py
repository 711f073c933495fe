"""CPU test of the compiled cache kernels' resources: none may use scratch
(stack) memory, which would put a memory round trip into their inner loops."""
import pytest

from test_kernel_resources import test_no_kernel_uses_scratch as check


@pytest.mark.parametrize("name", ["cache.hip"])
def test_no_cache_kernel_uses_scratch(name):
    check(name)
