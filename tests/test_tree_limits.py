"""Argument checks of the operators on drafted trees and on caches that are kept short, and
their oracles against hand-worked facts.

Every call of the library is refused (by a mistake of its own or, where nothing else is
wrong, by an unknown type or a misaligned address that only the last check sees), so
that none reaches a device; addresses are never dereferenced."""

import os
import subprocess
import sys

import numpy as np
import pytest

from oracle import (cache_select_ref, cache_weights_ref, mask_words_ref, pages_keep_ref,
                    tree_attention_ref, tree_paths_ref)

torch = pytest.importorskip("torch")
tq = pytest.importorskip("bit_mixed_precision_amd.binding")

A = 0x10000
N, S, G, V = tq.TQ_ERR_NULL, tq.TQ_ERR_SHAPE, tq.TQ_ERR_ALIGN, tq.TQ_ERR_VALUE
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def mask(parents=A, B=2, T=5, out=A + 4, depth=A):  # (out misaligned)
    return tq.raw_call("tq_tree_mask", parents, B, T, out, depth, None)


def tree(dtype=9, Q=A, qs=0, qt=512, qh=64, K=A, Vp=A, P=9, ps=16, pst=2048, rst=128, hst=64,
         table=A, width=40, lens=A, nodes=A, mask=A, mseq=5, B=2, T=5, Hq=8, Hkv=2, D=64, scale=1.0,
         window=0, out=A, lse=A, ws=A, room=1 << 40):
    return tq.raw_call("tq_tree_attention", dtype, Q, qs or qt * T, qt, qh, K, Vp, P, ps, pst, rst,
                       hst, table, width, lens, nodes, mask, mseq, B, T, Hq, Hkv, D, scale, window,
                       out, lse, ws, room, None)


def weights(dtype=9, Q=A, qs=0, qt=512, qh=64, K=A, P=9, ps=16, pst=2048, rst=128, hst=64, table=A,
            width=40, lens=A, nodes=A, mask=A, mseq=5, lse=A, B=2, T=5, Hq=8, Hkv=2, D=64, scale=1.0,
            window=0, decay=0.5, scores=A, ss=2000, sh=1000, S=900):
    return tq.raw_call("tq_cache_weights", dtype, Q, qs or qt * T, qt, qh, K, P, ps, pst, rst, hst,
                       table, width, lens, nodes, mask, mseq, lse, B, T, Hq, Hkv, D, scale, window,
                       decay, scores, ss, sh, S, None)


def select(scores=A, ss=2000, sh=1000, S=900, lens=A, B=2, H=2, budget=64, recent=8, sinks=4, keep=A,
           counts=A, sums=A + 2):  # (sums misaligned)
    return tq.raw_call("tq_cache_select", scores, ss, sh, S, lens, B, H, budget, recent, sinks, keep,
                       counts, sums, None)


def keep(pool=A, planes=4, P=9, pb=4096, table=A, lens=A, rows=3, width=4, size=16, lists=A, groups=2,
         heads=2, n=60, counts=A, base=A, table_out=A, lens_out=A, short=A + 2, ws=A, room=1 << 40):
    return tq.raw_call("tq_pages_keep", pool, planes, P, pb, table, lens, rows, width, size, lists,
                       groups, heads, n, counts, base, table_out, lens_out, short, ws, room, None)


def refuses(call, status, *bad):
    for kw in bad:
        assert call(**kw) == status, kw


def test_mask_refusals():
    assert mask() == G
    refuses(mask, N, dict(parents=None), dict(out=None))
    refuses(mask, S, dict(B=-1), dict(T=-1), dict(T=257), dict(B=(1 << 20) + 1))
    refuses(mask, G, dict(parents=A + 2, out=A), dict(out=A, depth=A + 2))
    refuses(mask, tq.TQ_OK, dict(B=0, parents=None), dict(T=0, out=None))
    assert mask(T=256, B=1 << 20, depth=None) == G


COMMON_NULL = [dict(Q=None), dict(K=None), dict(table=None), dict(lens=None)]
COMMON_SHAPE = [
    dict(B=-1), dict(T=-1), dict(T=257), dict(Hq=7), dict(Hkv=0), dict(Hq=4098), dict(D=60), dict(D=264),
    dict(D=0), dict(width=0), dict(ps=0), dict(width=1 << 27), dict(B=(1 << 20) + 1), dict(P=0),
    dict(P=1 << 31), dict(qt=516), dict(qh=68), dict(qs=2564), dict(pst=2052), dict(rst=132),
    dict(hst=68), dict(qt=-8), dict(rst=-8), dict(mseq=-1), dict(rst=(1 << 24) + 8), dict(pst=1 << 47),
    dict(qs=1 << 47), dict(qt=(1 << 46) + 8), dict(P=1 << 30, pst=1 << 30), dict(mseq=1 << 47),
    dict(window=4), dict(window=1)]
COMMON_ALIGN = [dict(Q=A + 8), dict(K=A + 8), dict(table=A + 2), dict(lens=A + 2), dict(nodes=A + 2),
                dict(mask=A + 4), dict(lse=A + 2)]
COMMON_VALUE = [dict(dtype=0, scale=float("nan")), dict(dtype=0, scale=3e38), dict(dtype=1, scale=-1e39),
                dict(dtype=0, window=-1), dict(dtype=2), dict(dtype=-1)]


def test_attention_refusals():
    assert tree() == V  # nothing but the type is wrong
    refuses(tree, N, *COMMON_NULL, dict(Vp=None), dict(out=None), dict(ws=None))
    refuses(tree, S, *COMMON_SHAPE, dict(room=0))
    refuses(tree, G, *COMMON_ALIGN, dict(Vp=A + 8), dict(out=A + 8), dict(ws=A + 8))
    refuses(tree, V, *COMMON_VALUE)
    refuses(tree, tq.TQ_OK, dict(B=0), dict(T=0, Q=None))
    # what need not be there, and strides of single entries
    refuses(tree, V, dict(nodes=None), dict(mask=None, mseq=-3), dict(lse=None), dict(window=5),
            dict(B=1, qs=3, mseq=-1), dict(T=1, qt=3, qs=512), dict(Hq=1, Hkv=1, qh=3, hst=5),
            dict(P=1, pst=-4), dict(ps=1, rst=-1, width=640))


def test_weights_refusals():
    assert weights() == V
    refuses(weights, N, *COMMON_NULL, dict(lse=None), dict(scores=None))
    refuses(weights, S, *COMMON_SHAPE, dict(S=-1), dict(S=(1 << 30) + 1, ss=1 << 40, sh=1 << 35),
            dict(ss=-1), dict(sh=-1), dict(ss=0), dict(sh=0), dict(sh=899), dict(ss=1500),
            dict(ss=1 << 47), dict(T=256, Hq=66, Hkv=2))  # 8448 rows
    refuses(weights, G, *COMMON_ALIGN, dict(scores=A + 2))
    refuses(weights, V, *COMMON_VALUE, dict(dtype=0, decay=-0.1), dict(dtype=0, decay=1.01),
            dict(dtype=0, decay=float("nan")))
    refuses(weights, tq.TQ_OK, dict(B=0), dict(T=0), dict(S=0, scores=None))
    refuses(weights, V, dict(nodes=None), dict(mask=None, mseq=-3), dict(B=1, ss=-1),
            dict(Hq=4, Hkv=1, sh=-1), dict(ss=1000, sh=2000), dict(T=256, Hq=64, Hkv=2))


def test_select_refusals():
    assert select() == G
    refuses(select, N, dict(scores=None), dict(lens=None), dict(keep=None), dict(counts=None))
    refuses(select, S, dict(B=-1), dict(H=-1), dict(S=-1), dict(budget=-1), dict(recent=-1),
            dict(sinks=-1), dict(recent=65), dict(recent=60, sinks=5), dict(recent=0, sinks=65),
            dict(S=(1 << 30) + 1), dict(budget=(1 << 30) + 1), dict(B=(1 << 20) + 1), dict(H=4097),
            dict(B=1 << 20, H=4, sh=0, ss=0), dict(ss=-1), dict(sh=1 << 47))
    refuses(select, G, dict(scores=A + 2, sums=A), dict(lens=A + 2, sums=A), dict(keep=A + 2, sums=A),
            dict(counts=A + 2, sums=A))
    refuses(select, tq.TQ_OK, dict(B=0, scores=None), dict(H=0, counts=None))
    refuses(select, G, dict(S=0, scores=None), dict(budget=0, recent=0, sinks=0, keep=None),
            dict(ss=0, sh=0), dict(B=1, ss=-1), dict(recent=60, sinks=4))


def test_keep_refusals():
    assert keep() == G
    refuses(keep, N, dict(pool=None), dict(table=None), dict(lens=None), dict(lists=None),
            dict(counts=None), dict(table_out=None), dict(lens_out=None), dict(short=None),
            dict(ws=None))
    refuses(keep, S, dict(rows=-1), dict(n=-1), dict(n=(1 << 30) + 1), dict(P=0), dict(width=0),
            dict(size=0), dict(planes=-1), dict(pb=4100), dict(pb=0), dict(groups=0), dict(groups=3),
            dict(heads=0), dict(heads=3), dict(size=15), dict(heads=32),  # 8 bytes of a token
            dict(room=64), dict(rows=(1 << 16) + 1), dict(P=(1 << 24) + 1), dict(width=1 << 27),
            dict(groups=(1 << 16) + 1, planes=0), dict(heads=1 << 17))
    refuses(keep, G, dict(pool=A + 8, short=A), dict(ws=A + 8, short=A), dict(lists=A + 1, short=A),
            dict(base=A + 2, short=A), dict(counts=A + 2, short=A), dict(table_out=A + 2, short=A))
    refuses(keep, G, dict(base=None), dict(n=0, lists=None), dict(planes=0, pool=None),
            dict(rows=0, table=None, lens=None, counts=None, table_out=None, lens_out=None, lists=None))


def test_workspaces():
    ws = tq.tq_tree_attention_workspace
    assert ws(0, 5, 8, 2, 64, 16, 40) == 0 and ws(3, 0, 8, 2, 64, 16, 40) == 0
    assert ws(1, 24, 8, 8, 64, 16, 4) == 0 and ws(1, 24, 8, 8, 64, 16, 10000) > 0
    for bad in ((1, 257, 8, 2, 64, 16, 40), (1, 5, 7, 2, 64, 16, 40), (1, 5, 8, 2, 63, 16, 40),
                (1, 5, 8, 2, 64, 0, 40), (-1, 5, 8, 2, 64, 16, 40), (1, 5, 8, 2, 64, 1 << 20, 1 << 11),
                (1 << 20, 1, 16, 16, 8, 1, 1), (1 << 17, 1, 8, 8, 64, 64, 1 << 12)):
        with pytest.raises(tq.TQError):
            ws(*bad)
    assert ws(1 << 20, 1, 15, 15, 8, 1, 1) == 0  # 2^24 blocks of rows are too many, fewer are not
    assert tq.tq_pages_keep_workspace(3, 40, 100) > 0
    with pytest.raises(tq.TQError):
        tq.tq_pages_keep_workspace(3, 0, 100)


def test_append_at_is_append_with_slots():
    def call(slots):
        return tq.raw_call("tq_rope_append_at", 9, A, 128, A, 8, 16, A, slots, None, A, 3, 4, A, A, 9, 16, 512,
                           32, 16, A, 3, 4, 2, 16, 0, None)
    assert call(None) == call(A) == V and call(A + 2) == G


# The binding: tensors on the CPU are refused by what is wrong with them, else by their device.

def error(fn, *a, **kw):
    with pytest.raises(tq.TQError) as e:
        fn(*a, **kw)
    return e.value.status


def i32(*x):
    return torch.tensor(x, dtype=torch.int32)


def args():
    q = torch.zeros(2, 5, 8, 64, dtype=torch.float16)
    k = torch.zeros(9, 16, 2, 64, dtype=torch.float16)
    return q, k, torch.zeros(2, 40, dtype=torch.int32), i32(30, 40)


def test_binding_refusals_of_trees():
    D = tq.TQ_ERR_DEVICE
    q, k, pt, lens = args()
    at = tq.tq_tree_attention
    assert error(at, q, k, k, pt, lens) == D
    assert error(at, q[0], k, k, pt, lens) == S and error(at, q.transpose(2, 3), k, k, pt, lens) == S
    assert error(at, q.float(), k, k, pt, lens) == V and error(at, q, k.bfloat16(), k, pt, lens) == V
    assert error(at, q, k, k, pt[:1], lens) == S and error(at, q, k, k, pt, lens[:1]) == S
    assert error(at, q, k, k, pt, lens, nodes=i32(1)) == S
    assert error(at, q, k, k, pt, lens.long()) == V
    for shape, status in (((2, 5, 1), D), ((1, 5, 1), D), ((5, 1), D), ((2, 5), S), ((5, 2), S),
                          ((3, 5, 1), S), ((2, 4, 1), S)):
        assert error(at, q, k, k, pt, lens, mask=torch.zeros(shape, dtype=torch.long)) == status, shape
    assert error(at, q, k, k, pt, lens, mask=torch.zeros(2, 5, 1, dtype=torch.int32)) == V
    assert error(at, q, k, k, pt, lens, mask=torch.zeros(2, 5, 2, dtype=torch.long)[..., :1]) == S
    assert error(at, q, k, k, pt, lens, mask=[1, 2]) == V
    assert error(at, q, k, k, pt, lens, out=q[:1]) == S
    assert error(at, q, k, k, pt, lens, workspace=torch.zeros(9)) == V
    assert error(tq.tq_tree_mask, pt) == D and error(tq.tq_tree_mask, pt[0]) == S
    assert error(tq.tq_tree_mask, pt.long()) == V and error(tq.tq_tree_mask, [1, 2]) != D


def test_binding_refusals_of_kept_caches():
    D = tq.TQ_ERR_DEVICE
    q, k, pt, lens = args()
    lse, x = torch.zeros(2, 5, 8), torch.zeros(2, 2, 100)
    w = tq.tq_cache_weights
    assert error(w, q, k, pt, lens, lse, x) == D
    assert error(w, q, k, pt, lens, lse[..., :7], x) == S and error(w, q, k, pt, lens, lse.half(), x) == V
    assert error(w, q, k, pt, lens, lse, x[:1]) == S and error(w, q, k, pt, lens, lse, x.half()) == V
    assert error(w, q, k, pt, lens, lse, x.transpose(1, 2)) == S
    assert error(w, q, k, pt, lens, lse, torch.zeros(2, 2, 100, 2)[..., 0]) == S
    assert error(w, q, k, pt[:1], lens, lse, x) == S and error(w, q, k, pt, lens, lse, 3) == V
    s = tq.tq_cache_select
    assert error(s, x, lens, 9) == D and error(s, x, lens, 9, 2, 1) == D
    assert error(s, x[0], lens, 9) == S and error(s, x, lens[:1], 9) == S and error(s, x, [3, 4], 9) == V
    p = tq.tq_pages_keep
    pool, lists = torch.zeros(4, 9, 16, 2, 64, dtype=torch.float16), torch.zeros(2, 60, dtype=torch.int32)
    assert error(p, pool, pt, lens, lists, lens, 16) == D
    for shape, status in (((2, 2, 60), D), ((2, 2, 2, 60), D), ((3, 60), S), ((60,), S), ((2, 3, 2, 60), S),
                          ((1, 1, 2, 2, 60), S)):
        assert error(p, pool, pt, lens, torch.zeros(shape, dtype=torch.int32), lens, 16) == status, shape
    assert error(p, pool, pt, lens, lists.long(), lens, 16) == V
    assert error(p, pool, pt, lens, lists, lens[:1], 16) == S
    assert error(p, pool, pt, lens, lists, lens, 16, base=lens[:1]) == S
    assert error(p, pool[:, :, ::2], pt, lens, lists, lens, 16) == S


def test_without_the_compiled_calls():
    """The binding without its compiled calls has every operator all the same."""
    code = ("import sys, torch; sys.modules['bit_mixed_precision_amd._tq_torch'] = None\n"
            "import bit_mixed_precision_amd.binding as b\n"
            "x = torch.zeros(1, 2, 3)\n"
            "try: b.tq_cache_select(x, torch.zeros(1, dtype=torch.int32), 2)\n"
            "except b.TQError as e: print(e.status == b.TQ_ERR_DEVICE)")
    out = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert out.stdout.strip() == "True", out.stdout + out.stderr


# The oracles against facts worked out by hand.

def test_paths_and_words():
    sees = tree_paths_ref(np.array([[-1, 0, 0, 2, 9]]))
    want = np.array([[1, 0, 0, 0, 0], [1, 1, 0, 0, 0], [1, 0, 1, 0, 0], [1, 0, 1, 1, 0], [0, 0, 0, 0, 1]])
    assert np.array_equal(sees[0], want.astype(bool))
    assert mask_words_ref(sees)[0, :, 0].tolist() == [1, 3, 5, 13, 16]


def test_attention_and_weights_oracles():
    """Two cached tokens and two nodes that do not see each other; scores worked out by hand."""
    k = np.zeros((1, 4, 1, 2))
    k[0, :, 0, 0] = [0, np.log(2), np.log(3), np.log(5)]
    v = np.arange(8.0).reshape(1, 4, 1, 2)
    q = np.ones((1, 2, 1, 2))
    sees = np.eye(2, dtype=bool)[None]
    out, lse, *_ = tree_attention_ref(q, k, v, np.array([[0]]), np.array([2]), np.array([2]), sees, 1.0, 0)
    assert np.allclose(np.exp(lse[0, :, 0]), [6, 8])
    assert np.allclose(out[0, 0, 0], (1 * v[0, 0, 0] + 2 * v[0, 1, 0] + 3 * v[0, 2, 0]) / 6)
    assert np.allclose(out[0, 1, 0], (1 * v[0, 0, 0] + 2 * v[0, 1, 0] + 5 * v[0, 3, 0]) / 8)
    got = cache_weights_ref(q, k, np.array([[0]]), np.array([2]), np.array([2]), sees, lse,
                            np.full((1, 1, 5), 8.0), 0.5, 1.0, 0)[0]
    assert np.allclose(got[0, 0], [4 + 1 / 6 + 1 / 8, 4 + 2 / 6 + 2 / 8, 3 / 6, 5 / 8, 8])


def test_select_and_keep_oracles():
    x = np.array([[[9, 1, 5, 5, 7, 0, 2]]], np.float32)
    keep, counts, sums = cache_select_ref(x, [7], 5, 1, 1)
    assert keep[0, 0].tolist() == [0, 2, 3, 4, 6] and counts.tolist() == [5]
    keep, counts, sums = cache_select_ref(x, [3], 5, 1, 1)
    assert keep[0, 0].tolist() == [0, 1, 2, -1, -1] and sums[0, 0].tolist() == [9, 1, 5, 0, 0]
    lists = np.array([[[[1, 3, 4]], [[0, 1, 2]]]])  # of two rows that share page 2
    table, lens, short, moves = pages_keep_ref([[2, 0, 1], [2, 3, -1]], [6, 4], lists, [3, 2], None, 6, 2)
    assert table.tolist() == [[4, 0, -1], [2, -1, -1]] and lens.tolist() == [3, 2] and short == 0
    assert moves == [(0, 0, 2, 1, 4, 0), (0, 0, 0, 1, 4, 1), (0, 0, 1, 0, 0, 0)]
