"""Rows of tree attention: what one node sees reaches no other node's
bits, and what is no number reaches every row that sees it, however the row is cut."""

import pytest

from oracle import tree_paths_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
tq = pytest.importorskip("bit_mixed_precision_amd.binding")

from test_decode_gpu import NAN  # noqa: E402
from test_tree_gpu import parents_of, tree, words  # noqa: E402


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,Hq,Hkv,D,lens", [
    (8, 8, 2, 64, [400, 390]),        # up to 32 rows, four tiles a wave
    (6, 4, 1, 128, [3000, 700, 90]),  # the same, cut between workgroups
    (30, 8, 2, 128, [640, 600]),      # many rows, ten tiles a wave
    (24, 8, 1, 64, [5000, 1200]),     # the same, cut between workgroups
    (10, 4, 2, 256, [650, 2000])])    # long heads
def test_a_large_key_of_a_sibling_changes_no_bits(dtype, T, Hq, Hkv, D, lens):
    """A drafted key twenty times as long as the others lifts the maxima of the rows that see
    it, in a tile after their first; the rows beside them have the same bits as without it."""
    B = len(lens)
    q, k, v, pt, ln, nodes = tree(T + D, dtype, lens, [T] * B, T, Hq, Hkv, D, 16, poison=False)
    sees = tree_paths_ref(parents_of(D, B, T, 3.0))
    j = T // 3
    sees[:, j, j] = True
    kw = dict(mask=words(sees), nodes=nodes, return_lse=True)
    want = tq.tq_tree_attention(q, k, v, pt, ln, **kw)
    for b, n in enumerate(lens):
        at = pt[b, (n + j) // 16].long(), (n + j) % 16
        k[at] *= 20
        v[at] *= -30
    got = tq.tq_tree_attention(q, k, v, pt, ln, **kw)
    clean = torch.from_numpy(~sees[:, :, j]).cuda()
    assert clean.any() and not clean.all()
    assert not torch.equal(got[1][~clean], want[1][~clean])
    for x, y in zip(got, want):
        assert torch.equal(x[clean], y[clean])


LONG = [(4, 8, 2, 64, [9000]), (2, 4, 1, 128, [5000, 0, 12000]), (20, 8, 2, 128, [9000, 100]), (3, 4, 2, 256, [8000])]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,Hq,Hkv,D,lens", LONG)
def test_undefined_queries_of_long_rows(dtype, T, Hq, Hkv, D, lens):
    """A query of NaN: its output and log-sum-exp are NaN, and nothing else is."""
    q, k, v, pt, ln, nodes = tree(T, dtype, lens, [T] * len(lens), T, Hq, Hkv, D, 16, poison=False)
    want = tq.tq_tree_attention(q, k, v, pt, ln, return_lse=True)
    q[0, 1, Hq - 1] = NAN
    got = tq.tq_tree_attention(q, k, v, pt, ln, return_lse=True)
    assert torch.isnan(got[0][0, 1, Hq - 1]).all() and torch.isnan(got[1][0, 1, Hq - 1])
    rest = torch.ones(q.shape[:3], dtype=torch.bool, device="cuda")
    rest[0, 1, Hq - 1] = False
    for x, y in zip(got, want):
        assert torch.equal(x[rest], y[rest])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,Hq,Hkv,D,lens", LONG)
def test_undefined_keys_in_the_midst_of_long_rows(dtype, T, Hq, Hkv, D, lens):
    """Keys of NaN in a thousand neighbouring tokens, whole parts of a row that is cut: every
    row that sees them is NaN."""
    q, k, v, pt, ln, nodes = tree(T, dtype, lens, [T] * len(lens), T, Hq, Hkv, D, 16, poison=False)
    want = tq.tq_tree_attention(q, k, v, pt, ln, return_lse=True)
    k[pt[0, 128:192].long()] = NAN  # tokens 2048 .. 3071
    got = tq.tq_tree_attention(q, k, v, pt, ln, return_lse=True)
    for x, y in zip(got, want):
        assert torch.isnan(x[0]).all() and torch.isfinite(y).all()
        assert torch.equal(x[1:], y[1:])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,Hq,Hkv,D,lens", LONG)
def test_infinite_values_of_parts_that_weigh_nothing(dtype, T, Hq, Hkv, D, lens):
    """An infinite value of a token whose weight rounds to zero makes NaN (or stays infinite), and
    does so too where its whole part of a long row weighs nothing beside the others."""
    q, k, v, pt, ln, nodes = tree(T, dtype, lens, [T] * len(lens), T, Hq, Hkv, D, 16, poison=False)
    want = tq.tq_tree_attention(q, k, v, pt, ln, scale=30.0, return_lse=True)
    page = pt[0, 130].long()  # a part of a row whose keys are short: scores near zero
    k[pt[0, 128:192].long()] *= 2.0 ** -10
    v[page, 5, :, 3], v[page, 5, :, 7] = float("inf"), -float("inf")
    out, lse = tq.tq_tree_attention(q, k, v, pt, ln, scale=30.0, return_lse=True)
    other = [d for d in range(D) if d not in (3, 7)]
    assert not torch.isfinite(out[0][..., [3, 7]]).any()
    assert torch.isfinite(out[0][..., other]).all() and torch.isfinite(lse[0]).all()
    assert torch.equal(out[1:], want[0][1:])
