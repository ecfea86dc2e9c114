"""Calls on kept caches at the ends of what their checks let through."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
tq = pytest.importorskip("bit_mixed_precision_amd.binding")

from test_decode_gpu import i32  # noqa: E402


@pytest.mark.parametrize("B", [1, 3, 700])
@pytest.mark.parametrize("S,budget", [(50, 20), (0, 20), (50, 0), (50, 50)])
def test_choice_without_heads(B, S, budget):
    """No heads: nothing is chosen, and the counts are what they are with heads."""
    lens = i32([(-3, 0, 7, 20, 49, 50, 10 ** 9)[b % 7] for b in range(B)])
    x = torch.rand(B, 2, S, device="cuda")
    want = tq.tq_cache_select(x, lens, budget, 3 if budget else 0, 2 if budget else 0)[1]
    stream = torch.cuda.current_stream().cuda_stream
    for kw in ({}, dict(stream=stream)):
        spoiled = torch.full((B,), 12345, dtype=torch.int32, device="cuda")  # handed out again
        del spoiled
        keep, counts, sums = tq.tq_cache_select(x[:, :0], lens, budget, 3 if budget else 0, 2 if budget else 0, **kw)
        assert keep.shape == sums.shape == (B, 0, budget)
        assert counts.tolist() == want.tolist()
