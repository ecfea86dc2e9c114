"""Calls on kept caches at the ends of what their checks let through."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
tq = pytest.importorskip("bit_mixed_precision_amd.binding")

from test_cache_gpu import check_keep, dealt, pool_of, some  # noqa: E402
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


@pytest.mark.parametrize("rows,size,free", [(12, 8, 0), (12, 8, 3), (300, 4, 40)])
def test_keep_where_pages_are_short(rows, size, free):
    """Every second row shares its first two pages with the row before it: rows that need pages when
    the free ones are used up are refused, and those that need none (nothing moves) go ahead, by
    either way of the bookkeeping."""
    rng = np.random.default_rng(rows)
    lens = rng.integers(2 * size, 6 * size, rows)
    pt, ln, _ = dealt(rows, lens, size, 0, width=7)
    pt[1::2, :2] = pt[::2, :2]
    held = pt >= 0
    pages, place = torch.unique(pt[held], return_inverse=True)
    pt[held] = place.int()
    counts = np.minimum(lens, rng.integers(size, 5 * size, rows))
    keep = some(rng, 1, rows, 1, lens, np.zeros(rows, int), counts, 5 * size)
    keep[0, ::3] = torch.arange(5 * size, device="cuda", dtype=torch.int32)  # these move nothing
    pool = pool_of(1, 2, len(pages) + free, size, 1, 16)
    _, left, short = check_keep(pool, pt, ln, keep, i32(counts), None, size)
    assert int(short) > 0 and left.tolist()[::3] == counts.tolist()[::3]
