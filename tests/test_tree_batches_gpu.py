"""Large batches of drafted trees: one long row among many short ones is shared by all
workgroups."""

import numpy as np
import pytest

from oracle import tree_paths_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
tq = pytest.importorskip("bit_mixed_precision_amd.binding")

from test_tree_gpu import parents_of, run, tree  # noqa: E402


@pytest.mark.parametrize("T,Hq,Hkv,D,B,long", [(3, 8, 8, 8, 400, 9000), (20, 16, 8, 16, 390, 4500)])
@pytest.mark.parametrize("at", [0, -1])
def test_one_long_row_in_a_large_batch(T, Hq, Hkv, D, B, long, at):
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 50, B)
    lens[at] = long
    nodes = rng.integers(0, T + 1, B)
    nodes[at] = T
    args = tree(1, "bf16", lens, nodes, T, Hq, Hkv, D, 16, poison=False)
    assert tq.tq_tree_attention_workspace(B, T, Hq, Hkv, D, 16, args[3].shape[1]) > 0  # rows are cut
    run(*args, tree_paths_ref(parents_of(2, B, T)), "bf16")
