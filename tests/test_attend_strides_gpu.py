"""GPU test of attention over rows that are aligned to their elements only."""
import pytest

from test_cache_gpu import gpu_cache, ints, new_pool

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_attend_odd_strides():
    """Queries and outputs whose addresses are aligned to their elements only."""
    T, H, group, D = 16, 2, 3, 96
    c = gpu_cache(new_pool(40, T, H, D, 3))
    n, heads = 5, H * group
    table, lens, starts = ints(range(36)).reshape(3, 12), ints([150, 33, 190]), ints([0, 1, 3, 5])
    for dtype in (torch.bfloat16, torch.float16):
        q = torch.randn(n, heads, D, device="cuda").to(dtype)
        want, want_lse = c.attend(q, table, lens, starts, lse=True)
        flat = torch.zeros(n * (heads * (D + 3) + 5) + 9, dtype=dtype, device="cuda")
        odd = flat[1:].as_strided((n, heads, D), (heads * (D + 3) + 5, D + 3, 1))
        odd.copy_(q)
        out_flat = torch.full((n * (heads * (D + 1) + 4) + 9,), 7.0, dtype=dtype, device="cuda")
        out = out_flat[3:].as_strided((n, heads, D), (heads * (D + 1) + 4, D + 1, 1))
        _, lse = c.attend(odd, table, lens, starts, out=out, lse=True)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        out.fill_(7.0)
        assert bool((out_flat == 7.0).all())  # nothing beside the rows was written
