"""Argument checks of calls on kept caches at the ends of their ranges.  As in
test_tree_limits.py every call is refused, so that none reaches a device."""

import numpy as np
import pytest

from oracle import pages_keep_ref

torch = pytest.importorskip("torch")
tq = pytest.importorskip("bit_mixed_precision_amd.binding")

from test_tree_limits import A, G, N, S, keep, refuses, select  # noqa: E402


def test_choice_without_heads():
    """Counts are wanted all the same; nothing else is looked at."""
    none = dict(H=0, scores=None, keep=None, sums=None)
    refuses(select, N, dict(none, lens=None))
    refuses(select, G, dict(none, counts=A + 2), dict(none, lens=A + 2), dict(none, ss=-1, sh=-1, counts=A + 1))
    refuses(select, S, dict(none, B=(1 << 20) + 1), dict(none, recent=65), dict(none, S=(1 << 30) + 1))
    refuses(select, tq.TQ_OK, dict(none, counts=None), dict(none, B=0))


def test_lists_of_a_row_are_counted_in_32_bits():
    """2^31 lists and more (groups times heads) are refused, one less passes on to the last check."""
    refuses(keep, S, *(dict(groups=g, planes=g, heads=h, size=1, pb=16 * h)
                       for g, h in ((1 << 15, 1 << 16), (1 << 16, 1 << 15), (1 << 16, 1 << 16))))
    refuses(keep, G, *(dict(groups=g, planes=g, heads=h, size=1, pb=16 * h)
                       for g, h in (((1 << 15) - 1, 1 << 16), (1 << 16, (1 << 15) - 1))))


def test_large_batches_are_cut_where_their_tables_hold_long_rows():
    """Tree attention gives a workgroup a whole row only where the longest that the table
    holds does not outlast the others: the workspace is what a cut needs."""
    ws = tq.tq_tree_attention_workspace
    for T in (4, 16):  # either form
        for B in (255, 256, 300, 1000):
            assert ws(B, T, 64, 8, 128, 16, 8192) > 0, (T, B)
        assert ws(256, T, 64, 8, 128, 16, 100) == ws(1000, T, 64, 8, 128, 16, 400) == 0


def test_keep_oracle_where_pages_are_short():
    """Rows that need pages are refused once those are used up; one that needs none is not."""
    table = np.array([[0, 1], [0, 2], [0, 3], [4, 5]])
    lists = np.array([[[[1, 2]], [[1, 3]], [[0, 1]], [[1, 3]]]])
    got, lens, short, moves = pages_keep_ref(table, [4, 4, 4, 4], lists, [2, 2, 2, 2], None, 7, 2)
    assert got.tolist() == [[6, -1], [0, 2], [0, -1], [4, -1]]
    assert lens.tolist() == [2, 4, 2, 2] and short == 1
    assert {m[4] for m in moves} == {6, 4}
