"""Rows of tree attention next to each other: what one node sees reaches no other node's bits."""

import pytest

from oracle import tree_paths_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
tq = pytest.importorskip("bit_mixed_precision_amd.binding")

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
