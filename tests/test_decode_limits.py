"""Argument checks of the decode-side entry points at the ends of their ranges.

Every call is refused (by an unknown type, if by nothing before it), so that none
reaches a device; addresses are never dereferenced."""

import pytest

torch = pytest.importorskip("torch")
tq = pytest.importorskip("bit_mixed_precision_amd.binding")

A = 0x10000
S, V = tq.TQ_ERR_SHAPE, tq.TQ_ERR_VALUE


def rope(X=A, xt=64, xh=16, Y=A * 2, yt=64, yh=16, n_pos=8, rot=16, T=3, H=4, D=16):
    return tq.raw_call("tq_rope", 9, X, xt, xh, Y, yt, yh, A, n_pos, rot, A, T, H, D, 0, 0, None)


def append(xt=128, n_pos=8, rot=16, n_seqs=3, width=4, P=9, ps=16, pst=512, rst=32, hst=16, T=3,
           Hq=4, Hkv=2, D=16):
    return tq.raw_call("tq_rope_append", 9, A, xt, A, n_pos, rot, A, None, A, n_seqs, width, A, A,
                       P, ps, pst, rst, hst, A, T, Hq, Hkv, D, 0, None)


def attn(qt=512, qh=64, P=9, ps=16, pst=2048, rst=128, hst=64, width=40, B=2, Hq=8, Hkv=2, D=64,
         scale=1.0, dtype=9):
    return tq.raw_call("tq_paged_attention", dtype, A, qt, qh, A, A, P, ps, pst, rst, hst, A, width,
                       A, B, Hq, Hkv, D, scale, 0, A, None, A, 1 << 40, None)


def test_strides_that_leave_64_bits():
    """Offsets of the last element have to stay in 64 bits: a stride that fits one
    step, taken 2^29 times, does not."""
    assert rope() == V and append() == V and attn() == V  # nothing but the type is wrong
    big = dict(T=1 << 29, H=2)
    for bad in (dict(yt=1 << 40, yh=1 << 46, xt=0), dict(yt=1 << 40, yh=1 << 41, xt=0),
                dict(yt=1 << 46, yh=1 << 4, xt=0), dict(yt=64, yh=16, xt=1 << 46),
                dict(yt=64, yh=16, xt=1 << 30)):
        assert rope(**big, **bad) == S, bad
    assert rope(**big, yt=1 << 28, yh=16, xt=1 << 28) == V  # 2^57 numbers apart
    assert append(T=1 << 28, xt=1 << 40) == S
    assert append(Hkv=1 << 15, hst=1 << 46, rst=1 << 45, pst=1 << 46, Hq=1, T=1) == S
    for bad in (dict(P=1 << 20, pst=1 << 46), dict(B=1 << 18, qt=1 << 46, width=1),
                dict(Hq=1 << 12, Hkv=1 << 12, hst=1 << 46 | 8), dict(P=1 << 30, pst=1 << 30)):
        assert attn(**bad) == S, bad
    assert attn(P=1 << 30, pst=1 << 27) == V


def test_scale_past_fp32():
    """The kernels hold scale log2(e) in fp32: a finite scale that leaves its range would
    make 0 * inf of a score of zero."""
    for bad in (3e38, -3e38, 1e39, 1e308, float("nan")):
        assert attn(scale=bad, dtype=0) == V, bad


def test_tokens_times_heads():
    """Both sides of the documented limit T H < 2^31, appending with Hq + 2 Hkv heads."""
    far = dict(yt=1 << 20, yh=16)
    assert rope(T=1 << 16, H=(1 << 15) - 1, **far) == V and rope(T=1 << 16, H=1 << 15, **far) == S
    assert rope(T=(1 << 30), H=1, yt=16) == V and rope(T=(1 << 30), H=2, yt=32) == S
    assert append(T=1 << 28, Hq=5, Hkv=1, xt=112) == V
    assert append(T=1 << 28, Hq=6, Hkv=1, xt=128) == S


def test_strides_of_single_entries():
    """The stride of a dimension of one entry is never taken, so it need not fit."""
    assert rope(T=1, xt=-1, yt=(1 << 46) + 1) == V and rope(H=1, xh=-1, yh=-5) == V
    assert append(T=1, xt=-1) == V and append(ps=1, rst=-1, width=64, pst=32) == V
    assert append(P=1, pst=-1) == V and append(Hkv=1, Hq=6, hst=-1) == V
    assert attn(B=1, qt=3) == V and attn(ps=1, rst=(1 << 24) + 8) == V and attn(P=1, pst=-4) == V
    assert attn(Hq=1, Hkv=1, qh=3, hst=5) == V
    # of two entries it is
    assert attn(B=2, qt=3) == S and attn(ps=2, rst=(1 << 24) + 8) == S and attn(P=2, pst=-4) == S
