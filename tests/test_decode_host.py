"""Decode-side operators on the CPU: the rotary table against the oracle, the
oracle against hand-worked facts, and every refusal of the C ABI and the binding
(checks that run before any device work)."""

import ctypes as C

import numpy as np
import pytest

from oracle import (paged_attention_ref, pages_compact_ref, pages_fork_ref, pages_grow_ref,
                    rope_frequencies_ref, rope_ref)

torch = pytest.importorskip("torch")
tq = pytest.importorskip("bit_mixed_precision_amd.binding")

SCALINGS = {"none": tq.TQ_ROPE_NONE, "linear": tq.TQ_ROPE_LINEAR, "base": tq.TQ_ROPE_BASE,
            "parts": tq.TQ_ROPE_PARTS}


@pytest.mark.parametrize("scaling", list(SCALINGS))
@pytest.mark.parametrize("n_pos,rot,theta", [(1, 2, 1e4), (7, 6, 5e5), (513, 80, 1e4),
                                             (9001, 128, 5e5)])
def test_rope_table(scaling, n_pos, rot, theta):
    if rot == 2 and scaling == "base":
        pytest.skip("the raised base is not defined for one pair")
    got = tq.tq_rope_table(n_pos, rot, theta, SCALINGS[scaling], 4.0, 256.0, 32.0, 1.0, 1.25)
    ang = np.arange(n_pos)[:, None] * rope_frequencies_ref(rot, theta, scaling, 4.0, 256.0)
    want = np.stack([np.cos(ang), np.sin(ang)], -1) * 1.25
    assert got.shape == (n_pos, rot // 2, 2)
    # one rounding to fp32 (2^-25 of at most 1.25, half an ulp) and the angle's fp64
    # error (2^-51 of at most 9001, its own and the frequency's)
    assert np.abs(got - want).max() <= 1.25 * (2.0 ** -24 + 9001 * 2.0 ** -50)


def test_rope_table_threads_agree():
    """A table large enough for several threads holds the same rows as a small one."""
    big = tq.tq_rope_table(20000, 64)
    assert np.array_equal(big[:100], tq.tq_rope_table(100, 64))
    ang = np.arange(20000)[:, None] * rope_frequencies_ref(64, 5e5)
    assert np.abs(big[..., 0] - np.cos(ang)).max() <= 2.0 ** -24 + 20000 * 2.0 ** -50


def test_rope_table_refusals():
    buf = np.empty(64, np.float32)

    def call(n_pos=4, rot=4, theta=1e4, scaling=0, factor=1.0, trained=1.0, fast=2.0, slow=1.0,
             gain=1.0, table=buf.ctypes.data):
        return tq.raw_call("tq_rope_table", n_pos, rot, theta, scaling, factor, trained, fast,
                           slow, gain, table)

    assert call() == tq.TQ_OK
    assert call(table=None) == tq.TQ_ERR_NULL
    assert call(n_pos=0, table=None) == tq.TQ_OK
    for bad in (dict(n_pos=-1), dict(rot=3), dict(rot=0), dict(rot=(1 << 16) + 2),
                dict(n_pos=(1 << 30) + 1), dict(rot=2, scaling=2)):
        assert call(**bad) == tq.TQ_ERR_SHAPE, bad
    for bad in (dict(theta=0.0), dict(theta=float("nan")), dict(scaling=4), dict(scaling=-1),
                dict(gain=float("inf")), dict(scaling=1, factor=0.0),
                dict(scaling=3, factor=2.0, fast=1.0, slow=1.0),
                dict(scaling=3, factor=2.0, trained=-1.0)):
        assert call(**bad) == tq.TQ_ERR_VALUE, bad


def test_oracle_rotation_facts():
    # a quarter turn takes (1, 0) to (0, 1); layouts name different partners
    X = np.zeros((1, 1, 4))
    X[0, 0, 0] = 1
    f = np.array([np.pi / 2, 0.0])
    assert np.allclose(rope_ref(X, [1], f), [[[0, 0, 1, 0]]])
    assert np.allclose(rope_ref(X, [1], f, interleaved=True), [[[0, 1, 0, 0]]])
    # scores depend on the distance only, and turning back undoes a turn
    rng = np.random.default_rng(1)
    q, k = rng.normal(size=(2, 1, 1, 8))
    f = rope_frequencies_ref(8, 1e4)
    dots = [(rope_ref(q, [a], f) * rope_ref(k, [a + 5], f)).sum() for a in (0, 3, 400)]
    assert np.allclose(dots, dots[0])
    assert np.allclose(rope_ref(rope_ref(q, [9], f), [9], f, inverse=True), q)


def test_oracle_attention_facts():
    # equal scores average the values of the tokens in the window
    k = np.zeros((2, 2, 1, 8))
    v = np.arange(4).reshape(2, 2, 1, 1) * np.ones((2, 2, 1, 8))
    q = np.ones((1, 2, 8))
    out, lse, _, _ = paged_attention_ref(q, k, v, np.array([[1, 0]]), [3], 1.0)
    assert np.allclose(out, (2 + 3 + 0) / 3) and np.allclose(lse, np.log(3))
    out, _, _, _ = paged_attention_ref(q, k, v, np.array([[1, 0]]), [3], 1.0, window=2)
    assert np.allclose(out, (3 + 0) / 2)
    out, lse, _, _ = paged_attention_ref(q, k, v, np.array([[1, 0]]), [0], 1.0)
    assert np.all(out == 0) and np.all(lse == -np.inf)


def test_oracle_pages_facts():
    table, lens = np.array([[4, 2, -1], [0, -1, -1]], np.int32), [6, 4]
    t, n, refs, short, copies = pages_fork_ref(table, lens, [0, 0, 1], 6, 4)
    assert t.tolist() == [[4, 2, -1], [4, 1, -1], [0, -1, -1]] and n.tolist() == [6, 6, 4]
    assert refs.tolist() == [1, 1, 1, 0, 2, 0] and short == 0 and copies == [(2, 1)]
    t, n, refused = pages_grow_ref(table, lens, [3, 1], 6, 4)
    assert t.tolist() == [[4, 2, 1], [0, 3, -1]] and n.tolist() == [9, 5] and refused == 0
    t, used, moves = pages_compact_ref(table, lens, 6, 4)
    assert t.tolist() == [[1, 2, -1], [0, -1, -1]] and used == 3 and moves == [(4, 1)]


A = 0x10000  # 16-byte aligned, never dereferenced: every call below is refused first


def _rope(dtype=0, X=A, xt=64, xh=16, Y=A * 2, yt=64, yh=16, table=A, n_pos=8, rot=16, pos=A, T=3,
          H=4, D=16, inter=0, inv=0):
    return tq.raw_call("tq_rope", dtype, X, xt, xh, Y, yt, yh, table, n_pos, rot, pos, T, H, D,
                       inter, inv, None)


def test_rope_refusals():
    for k in ("X", "Y", "table", "pos"):
        assert _rope(**{k: None}) == tq.TQ_ERR_NULL
        assert _rope(**{k: None}, T=0) == tq.TQ_OK and _rope(**{k: None}, H=0) == tq.TQ_OK
    for bad in (dict(T=-1), dict(rot=15), dict(rot=18), dict(rot=0), dict(n_pos=-1), dict(xt=-1),
                dict(yh=8), dict(yt=0), dict(yt=48), dict(yt=16, yh=47), dict(T=1 << 30, H=4),
                dict(D=(1 << 16) + 2, yh=1 << 20, yt=1 << 24), dict(X=A, Y=A, xt=128),
                dict(xt=(1 << 46) + 1)):
        assert _rope(**bad) == tq.TQ_ERR_SHAPE, bad
    for bad in (dict(X=A + 1), dict(Y=2 * A + 1), dict(table=A + 4), dict(pos=A + 2),
                dict(dtype=2, X=A + 2)):
        assert _rope(**bad) == tq.TQ_ERR_ALIGN, bad
    for bad in (dict(dtype=3), dict(dtype=-1), dict(inter=2), dict(inv=-1)):
        assert _rope(**bad) == tq.TQ_ERR_VALUE, bad


def _append(dtype=0, X=A, xt=128, table=A, n_pos=8, rot=16, pos=A, seqs=None, pt=A, n_seqs=3,
            width=4, k=A, v=A, P=9, ps=16, pst=512, rst=32, hst=16, Q=A, T=3, Hq=4, Hkv=2, D=16,
            inter=0):
    return tq.raw_call("tq_rope_append", dtype, X, xt, table, n_pos, rot, pos, seqs, pt, n_seqs,
                       width, k, v, P, ps, pst, rst, hst, Q, T, Hq, Hkv, D, inter, None)


def test_rope_append_refusals():
    for k in ("X", "table", "pos", "pt", "k", "v", "Q"):
        assert _append(**{k: None}) == tq.TQ_ERR_NULL
    assert _append(X=None, T=0) == tq.TQ_OK
    for bad in (dict(T=-1), dict(rot=17), dict(Hq=0), dict(Hkv=0), dict(P=0), dict(ps=0),
                dict(width=0), dict(width=1 << 20, ps=1 << 11), dict(n_seqs=0), dict(pst=-8),
                dict(hst=-1), dict(pst=1 << 46, P=1 << 30), dict(hst=0), dict(hst=15),
                dict(rst=16), dict(pst=0), dict(pst=511), dict(hst=512, rst=16, pst=767)):
        assert _append(**bad) == tq.TQ_ERR_SHAPE, bad
    # heads outside slots, slots outside pages: any nesting is a cache (refused later)
    for good in (dict(hst=256, rst=16, pst=512), dict(hst=144, rst=9 * 2 * 16, pst=16),
                 dict(pst=513), dict(P=1, pst=0)):
        assert _append(**good, dtype=2) == tq.TQ_ERR_VALUE, good
    for bad in (dict(X=A + 1), dict(k=A + 1), dict(pt=A + 2), dict(seqs=A + 1)):
        assert _append(**bad) == tq.TQ_ERR_ALIGN, bad
    for bad in (dict(dtype=2), dict(inter=3)):
        assert _append(**bad) == tq.TQ_ERR_VALUE, bad


def _attn(dtype=0, Q=A, qt=512, qh=64, k=A, v=A, P=9, ps=16, pst=2048, rst=128, hst=64, pt=A,
          width=40, lens=A, B=2, Hq=8, Hkv=2, D=64, scale=1.0, window=0, out=A, lse=None, ws=A,
          wsb=1 << 40):
    return tq.raw_call("tq_paged_attention", dtype, Q, qt, qh, k, v, P, ps, pst, rst, hst, pt,
                       width, lens, B, Hq, Hkv, D, scale, window, out, lse, ws, wsb, None)


def test_paged_attention_refusals():
    for k in ("Q", "k", "v", "pt", "lens", "out", "ws"):
        assert _attn(**{k: None}) == tq.TQ_ERR_NULL, k
    assert _attn(Q=None, B=0) == tq.TQ_OK
    for bad in (dict(B=-1), dict(D=12), dict(D=264), dict(D=0), dict(Hq=7), dict(Hkv=0),
                dict(Hq=1 << 13), dict(qt=4), dict(rst=132), dict(rst=(1 << 24) + 8),
                dict(pst=-8), dict(P=0), dict(width=0), dict(ps=1 << 30), dict(wsb=1024),
                dict(width=1 << 25, ps=32, Hq=512)):
        assert _attn(**bad) == tq.TQ_ERR_SHAPE, bad
    for bad in (dict(Q=A + 8), dict(k=A + 2), dict(out=A + 4), dict(ws=A + 8), dict(lens=A + 1),
                dict(lse=A + 2)):
        assert _attn(**bad) == tq.TQ_ERR_ALIGN, bad
    for bad in (dict(dtype=2), dict(dtype=-1), dict(scale=float("inf")), dict(window=-1)):
        assert _attn(**bad) == tq.TQ_ERR_VALUE, bad
    assert tq.lib.tq_paged_attention_workspace(2, 8, 2, 12, 16, 4) == tq.TQ_ERR_SHAPE
    # short tables need no workspace
    assert tq.tq_paged_attention_workspace(2, 8, 2, 64, 16, 32) == 0
    assert tq.tq_paged_attention_workspace(2, 8, 2, 64, 16, 33) > 0
    assert tq.tq_paged_attention_workspace(2, 8, 2, 256, 16, 16) == 0
    assert tq.tq_paged_attention_workspace(2, 8, 2, 256, 16, 17) > 0


def test_pages_refusals():
    wsb = tq.tq_pages_workspace(4, 100)

    def fork(pool=A, planes=2, P=100, pb=1024, t=A, n=A, rows_in=4, parent=A, rows=4, width=8,
             ps=16, to=A, no=A, refs=None, short=A, ws=A, b=wsb):
        return tq.raw_call("tq_pages_fork", pool, planes, P, pb, t, n, rows_in, parent, rows, width,
                           ps, to, no, refs, short, ws, b, None)

    for k in ("pool", "t", "n", "parent", "to", "no", "short", "ws"):
        assert fork(**{k: None}) == tq.TQ_ERR_NULL, k
    for bad in (dict(planes=-1), dict(P=0), dict(pb=1000), dict(pb=0), dict(rows=-1),
                dict(rows_in=-1), dict(width=0), dict(ps=0), dict(b=wsb - 1), dict(P=(1 << 24) + 1),
                dict(rows=(1 << 16) + 1), dict(width=1 << 20, ps=1 << 12)):
        assert fork(**bad) == tq.TQ_ERR_SHAPE, bad
    for bad in (dict(pool=A + 8), dict(ws=A + 4), dict(parent=A + 1), dict(refs=A + 2)):
        assert fork(**bad) == tq.TQ_ERR_ALIGN, bad

    def grow(t=A, n=A, add=A, rows=4, width=8, ps=16, P=100, to=A, no=A, short=A, ws=A, b=wsb):
        return tq.raw_call("tq_pages_grow", t, n, add, rows, width, ps, P, to, no, short, ws, b,
                           None)

    for k in ("t", "n", "add", "to", "no", "short", "ws"):
        assert grow(**{k: None}) == tq.TQ_ERR_NULL, k
    assert grow(b=wsb - 1) == tq.TQ_ERR_SHAPE and grow(ps=0) == tq.TQ_ERR_SHAPE
    assert grow(add=A + 2) == tq.TQ_ERR_ALIGN

    def compact(pool=A, planes=2, P=100, pb=1024, t=A, n=A, rows=4, width=8, ps=16, to=A, used=A,
                ws=A, b=wsb):
        return tq.raw_call("tq_pages_compact", pool, planes, P, pb, t, n, rows, width, ps, to, used,
                           ws, b, None)

    for k in ("pool", "t", "n", "to", "used", "ws"):
        assert compact(**{k: None}) == tq.TQ_ERR_NULL, k
    assert compact(pb=24) == tq.TQ_ERR_SHAPE and compact(b=0) == tq.TQ_ERR_SHAPE
    assert compact(to=A + 2) == tq.TQ_ERR_ALIGN

    def copy(pool=A, planes=2, P=100, pb=1024, src=A, dst=A, n=5):
        return tq.raw_call("tq_pages_copy", pool, planes, P, pb, src, dst, n, None)

    for k in ("pool", "src", "dst"):
        assert copy(**{k: None}) == tq.TQ_ERR_NULL, k
        assert copy(**{k: None}, n=0) == tq.TQ_OK
    assert copy(n=-1) == tq.TQ_ERR_SHAPE and copy(pb=8) == tq.TQ_ERR_SHAPE
    assert copy(src=A + 1) == tq.TQ_ERR_ALIGN
    assert tq.lib.tq_pages_workspace(-1, 5) == tq.TQ_ERR_SHAPE
    assert tq.lib.tq_pages_workspace(4, 0) == tq.TQ_ERR_SHAPE


def _status(fn, *a, **k):
    with pytest.raises(tq.TQError) as e:
        fn(*a, **k)
    return e.value.status


def test_binding_refusals():
    """Types, shapes, strides, then the device, all with CPU tensors."""
    h = torch.float16
    X, pos = torch.zeros(3, 4, 16, dtype=h), torch.zeros(3, dtype=torch.int32)
    tab = torch.zeros(8, 8, 2)
    V, S, D = tq.TQ_ERR_VALUE, tq.TQ_ERR_SHAPE, tq.TQ_ERR_DEVICE
    assert _status(tq.tq_rope, X, tab, pos) == D
    assert _status(tq.tq_rope, X.int(), tab, pos) == V
    assert _status(tq.tq_rope, X[0], tab, pos) == S
    assert _status(tq.tq_rope, X.transpose(1, 2), tab, pos) == S
    assert _status(tq.tq_rope, X, tab.double(), pos) == V
    assert _status(tq.tq_rope, X, tab[:, :, 0], pos) == S
    assert _status(tq.tq_rope, X, tab, pos.long()) == V
    assert _status(tq.tq_rope, X, tab, pos[:2]) == S
    assert _status(tq.tq_rope, X, tab, pos, Y=X.bfloat16()) == V
    assert _status(tq.tq_rope, X, tab, pos, Y=X[:2]) == S

    qkv = torch.zeros(3, 8, 16, dtype=h)  # 4 query, 2 key, 2 value heads
    k = torch.zeros(5, 16, 2, 16, dtype=h)
    pt = torch.zeros(3, 4, dtype=torch.int32)
    ok = (qkv, tab, pos, pt, k, k)
    assert _status(tq.tq_rope_append, *ok) == D
    assert _status(tq.tq_rope_append, qkv.float(), *ok[1:]) == V
    assert _status(tq.tq_rope_append, torch.zeros(3, 8, 32, dtype=h)[:, :, ::2], *ok[1:]) == S
    assert _status(tq.tq_rope_append, qkv[:, :4], *ok[1:]) == S
    assert _status(tq.tq_rope_append, *ok[:4], k.bfloat16(), k) == V
    assert _status(tq.tq_rope_append, *ok[:4], k, k[:4]) == S
    assert _status(tq.tq_rope_append, *ok[:4], k[..., :8], k[..., :8]) == S
    assert _status(tq.tq_rope_append, *ok, seqs=pos.long()) == V

    q = torch.zeros(3, 4, 16, dtype=h)
    lens = torch.zeros(3, dtype=torch.int32)
    ok = (q, k, k, pt, lens)
    assert _status(tq.tq_paged_attention, *ok) == D
    assert _status(tq.tq_paged_attention, q.float(), *ok[1:]) == V
    assert _status(tq.tq_paged_attention, q, k, k, pt[:2], lens) == S
    assert _status(tq.tq_paged_attention, q, k, k, pt, lens[:2]) == S
    assert _status(tq.tq_paged_attention, q, k, k, pt.long(), lens) == V
    assert _status(tq.tq_paged_attention, *ok, out=q[:2]) == S
    assert _status(tq.tq_paged_attention, *ok, workspace=torch.zeros(4)) == V

    pool = torch.zeros(2, 5, 16, 16, dtype=h)
    assert _status(tq.tq_pages_fork, pool, pt, lens, pos, 16) == D
    assert _status(tq.tq_pages_fork, pool.transpose(0, 1), pt, lens, pos, 16) == S
    assert _status(tq.tq_pages_fork, pool, pt, lens[:2], pos, 16) == S
    assert _status(tq.tq_pages_fork, pool, pt, lens, pos.float(), 16) == V
    assert _status(tq.tq_pages_grow, pt, lens, pos[:2], 5, 16) == S
    assert _status(tq.tq_pages_grow, pt, lens, pos, 5, 16) == D
    assert _status(tq.tq_pages_compact, pool, pt.long(), lens, 16) == V
    assert _status(tq.tq_pages_compact, pool, pt, lens, 16) == D
    assert _status(tq.tq_pages_copy, pool, pos, pos[:2]) == S
    assert _status(tq.tq_pages_copy, pool, pos, pos) == D


def test_compiled_calls_leave_the_rest_to_python():
    """The compiled functions return None, and do nothing, for anything but tensors
    on the current GPU: the Python path then words the refusal."""
    f = tq._fast
    X, pos = torch.zeros(3, 4, 16, dtype=torch.float16), torch.zeros(3, dtype=torch.int32)
    tab, pt = torch.zeros(8, 8, 2), torch.zeros(3, 4, dtype=torch.int32)
    k, pool = torch.zeros(5, 16, 2, 16, dtype=torch.float16), torch.zeros(2, 5, 16, 16)
    assert f.rope(X, tab, pos, False, False) is None
    assert f.rope(None, tab, pos, False, False) is None
    assert f.rope(X, tab) is None and f.rope() is None
    assert f.rope_append(X, tab, pos, pt, k, k, False, None) is None
    assert f.rope_append(X, tab, pos, pt, k, k, False, 3) is None
    assert f.paged_attention(X, k, k, pt, pos, None, 0, True) is None
    assert f.paged_attention(X, k, k, pt, pos, "a", 0, True) is None
    assert f.pages_fork(pool, pt, pos, pos, 16) is None
    assert f.pages_grow(pt, pos, pos, 5, 16) is None
    assert f.pages_compact(pool, pt, pos, 16) is None
    with pytest.raises(TypeError):
        f.bind()
    with pytest.raises(KeyError):
        f.bind(lambda i: 0, {"tq_rope": 1})
    # what was bound before still is
    assert f.rope(X, tab, pos, False, False) is None


def test_division_constants():
    """The multiply-and-shift divisions of the kernels, t / d for t < 2^30 and n / d
    for n < 2^31, at every divisor's most critical dividends."""
    rng = np.random.default_rng(2)
    for bits in (30, 31):
        ds = np.unique(np.concatenate([np.arange(1, 300), 2 ** np.arange(0, bits),
                                       2 ** np.arange(1, bits) - 1, 2 ** np.arange(1, bits) + 1,
                                       rng.integers(1, 2 ** bits, 300)]))
        for d in ds[(ds >= 1) & (ds < 2 ** bits)].tolist():
            s = max(0, (d - 1).bit_length())
            m = -(-(1 << (bits + s)) // d)
            assert m < 1 << 32
            top = ((1 << bits) - 1) // d
            for q in {0, 1, 2, top - 1, top, top // 2}:
                for n in (q * d - 1, q * d, q * d + d - 1):
                    if 0 <= n < 1 << bits:
                        assert n * m < 1 << 64 and (n * m) >> (bits + s) == n // d, (n, d)


def test_abi_types():
    assert C.sizeof(C.c_int) == 4 and tq.TQ_BF16 == 1 and tq.TQ_F32 == 2
