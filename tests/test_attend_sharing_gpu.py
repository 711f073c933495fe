"""GPU test of when attention's tokens are shared out: not where there are many
more tiles of rows than the GPU holds workgroups."""
import pytest

from test_attend_weights_gpu import is_shared
from test_cache_gpu import ints

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_which_calls_are_shared():
    def shared(batch, rows, tokens, most, H=8, group=4, D=128, T=16):
        return is_shared(batch, rows, T, H, group, D, "bf16", tokens // T, most, tokens)
    assert shared(8, 2000, 5008, 600)        # chunks of prompts
    assert shared(64, 64, 8000, 1) and shared(1024, 1024, 8000, 1)
    assert not shared(8, 8 * 4208, 4208, 4208) and not shared(1, 20000, 20000, 20000)


def test_whole_prompts_either_side_of_4096_tokens():
    """Prompts of 4200 tokens take 1.16 times the work of 3900 (shared out, in twice the
    time)."""
    import recv_fifo_plane_amd as xf
    B, H, group, D, T = 8, 8, 4, 128, 16
    took = {}
    for n in (3904, 4208):
        c = xf.PagedCache(B * n // T, T, H, D)
        c.scales().fill_(0.01)
        q = torch.randn(B * n, H * group, D, device="cuda").to(torch.bfloat16)
        args = q, ints(range(B * n // T)).reshape(B, -1), ints([n] * B), ints([i * n for i in range(B + 1)])
        out, times = torch.empty_like(q), []
        for _ in range(5):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            c.attend(*args, out=out, max_query=n, max_length=n)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        took[n] = min(times)
    assert took[4208] < 1.5 * took[3904], took
