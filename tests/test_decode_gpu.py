"""GPU parity of the decode-side operators against the fp64 oracle.

Tolerances are derived, not fitted.  half_ulp(y) is half the distance of
neighbouring numbers of the output type at y: 2^(e - p) for 2^e <= |y| < 2^(e+1)
and p significant bits (fp16 11, bf16 8, fp32 24).

* rotation: cos and sin rounded once to fp32, a product and a fused multiply-add
  in fp32, one rounding to the type: |err| <= 4 * 2^-24 gain (|a| + |b|) +
  half_ulp(y);
* attention: a score is an fp32 sum of D exact products, off by at most
  ds = (D + 4) 2^-24 smag (smag = scale sum |q k|, the scaling's own rounding
  included), which moves each weight by a factor e^(2 ds) at most; the weight as
  two 16-bit numbers is off by 2^-20 (fp16) or 2^-14 (bf16) of itself, and below
  the fp16 range by 2^-38 of the largest weight; exponentials and the fp32 sums
  over n tokens add (n + 16) 2^-23 in the worst case.  All are relative to
  sum w |v|; then one rounding, half_ulp(out).
"""

import math

import numpy as np
import pytest

from oracle import (paged_attention_ref, pages_compact_ref, pages_fork_ref, pages_grow_ref,
                    rope_frequencies_ref, rope_ref)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
tq = pytest.importorskip("bit_mixed_precision_amd.binding")

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BITS = {"f16": (11, -14), "bf16": (8, -126), "f32": (24, -126)}  # significant, lowest exponent
NAN = float("nan")


def half_ulp(y, dtype):
    """Half an ulp at |y|, half the smallest subnormal near zero."""
    p, low = BITS[dtype]
    e = np.maximum(np.frexp(np.abs(y))[1] - 1, low)
    return np.ldexp(1.0, e - p)


def f64(t):
    return t.detach().double().cpu().numpy()


def randn(seed, dtype, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(DT[dtype]).cuda()


def i32(a):
    return torch.as_tensor(np.asarray(a, dtype=np.int32)).cuda()


# ------------------------------------------------------------------ rotary

def rope_bound(X, want, dtype, gain, rot, interleaved):
    X = np.abs(f64(X))
    pair = X.copy()
    if interleaved:
        s = X[..., 0:rot:2] + X[..., 1:rot:2]
        pair[..., 0:rot:2] = pair[..., 1:rot:2] = s
    else:
        s = X[..., :rot // 2] + X[..., rot // 2:rot]
        pair[..., :rot // 2] = pair[..., rot // 2:rot] = s
    before = 4 * 2.0 ** -24 * gain * pair
    return before + half_ulp(np.abs(want) + before, dtype)


def check_rope(Y, X, pos, freq, dtype, interleaved, inverse, gain=1.0, n_pos=None):
    want = rope_ref(f64(X), f64(pos).astype(np.int64), freq, interleaved, inverse, gain, n_pos)
    err = np.abs(f64(Y) - want)
    bound = rope_bound(X, want, dtype, gain, 2 * len(freq), interleaved)
    assert np.all(err <= bound), float((err / bound).max())


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("T,H,D,rot", [
    (1, 1, 2, 2),        # one pair
    (1, 72, 128, 128),   # one token of a decode step
    (3, 5, 80, 32),      # part of the head
    (7, 3, 80, 40),      # 20 pairs: vectors of 4
    (5, 2, 37, 6),       # an odd head: single numbers
    (33, 9, 64, 64),
    (130, 17, 96, 96),   # more rows than a workgroup's
    (4, 3, 600, 594),    # more units than threads
])
def test_rope(dtype, interleaved, inverse, T, H, D, rot):
    freq = rope_frequencies_ref(rot, 1e4)
    table = torch.from_numpy(tq.tq_rope_table(5000, rot, 1e4)).cuda()
    X = randn(T + D, dtype, T, H, D)
    pos = i32(np.random.default_rng(D).integers(0, 5000, T))
    Y = tq.tq_rope(X, table, pos, interleaved=interleaved, inverse=inverse)
    check_rope(Y, X, pos, freq, dtype, interleaved, inverse)
    # in place
    Z = X.clone()
    assert tq.tq_rope(Z, table, pos, interleaved=interleaved, inverse=inverse, Y=Z) is Z
    assert torch.equal(Z, Y)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_rope_many_rows(dtype):
    """Enough rows for several per thread, a scaled table with a gain."""
    T, H, D = 1203, 24, 64
    freq = rope_frequencies_ref(64, 5e5, "parts", 8.0, 512.0)
    table = torch.from_numpy(tq.tq_rope_table(1000, 64, 5e5, tq.TQ_ROPE_PARTS, 8.0, 512.0,
                                              gain=1.25)).cuda()
    X = randn(3, dtype, T, H, D)
    pos = i32(np.arange(T) % 1000)
    for inter in (False, True):
        check_rope(tq.tq_rope(X, table, pos, interleaved=inter), X, pos, freq, dtype, inter, False,
                   1.25)


@pytest.mark.parametrize("D,off", [(64, 0), (64, 4), (64, 1)])
def test_rope_strides_and_alignment(D, off):
    """Views: heads inside a wider row, [H][T][D] order in and out, a broadcast
    token, and bases that are not 16-byte aligned."""
    freq = rope_frequencies_ref(D, 1e4)
    table = torch.from_numpy(tq.tq_rope_table(64, D, 1e4)).cuda()
    T, H = 9, 6
    pos = i32(np.arange(T) * 5)
    flat = randn(1, "f16", T * (H + 3) * D + off)[off:]
    X = flat.view(T, H + 3, D)[:, 2:2 + H]
    check_rope(tq.tq_rope(X, table, pos), X, pos, freq, "f16", False, False)
    out = torch.zeros(H, T, D, dtype=torch.float16, device="cuda").transpose(0, 1)
    check_rope(tq.tq_rope(X, table, pos, Y=out), X, pos, freq, "f16", False, False)
    Xt = flat[:H * T * D].view(H, T, D).transpose(0, 1)
    check_rope(tq.tq_rope(Xt, table, pos), Xt, pos, freq, "f16", False, False)
    Xb = flat[:H * D].view(1, H, D).expand(T, H, D)
    check_rope(tq.tq_rope(Xb, table, pos), Xb, pos, freq, "f16", False, False)
    # what lies between the heads of Y stays
    room = torch.full((T, H + 3, D), 7.0, dtype=torch.float16, device="cuda")
    tq.tq_rope(X, table, pos, Y=room[:, 1:1 + H])
    assert torch.all(room[:, 0] == 7) and torch.all(room[:, 1 + H:] == 7)


def test_rope_positions_outside_the_table():
    table = torch.from_numpy(tq.tq_rope_table(10, 16, 1e4)).cuda()
    X = torch.full((5, 2, 24), NAN, dtype=torch.float16, device="cuda")
    X[1] = 1
    Y = tq.tq_rope(X, table, i32([-1, 9, 10, 2 ** 31 - 1, -2 ** 31]))
    assert torch.all(Y[[0, 2, 3, 4]] == 0) and torch.all(torch.isfinite(Y[1]))
    check_rope(Y[1:2], X[1:2], i32([9]), rope_frequencies_ref(16, 1e4), "f16", False, False)
    # no position is valid in an empty table
    assert torch.all(tq.tq_rope(X[1:2], table[:0], i32([0])) == 0)
    assert tq.tq_rope(X[:0], table, i32([])).shape == (0, 2, 24)


def test_rope_non_finite_values_stay_in_their_pair():
    table = torch.from_numpy(tq.tq_rope_table(10, 16, 1e4)).cuda()
    X = torch.ones(1, 1, 24, dtype=torch.float16, device="cuda")
    X[0, 0, 3], X[0, 0, 20] = float("inf"), NAN
    Y = f64(tq.tq_rope(X, table, i32([5])))[0, 0]
    assert not np.isfinite(Y[[3, 11]]).any() and np.isnan(Y[20])
    assert np.isfinite(np.delete(Y, [3, 11, 20])).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_gradient(interleaved):
    """The inverse call against the formula's transpose and against differences of
    the forward call (a linear map: differences of any step are exact up to
    rounding, 2^-20 of the summed magnitudes)."""
    T, H, D, rot = 6, 3, 40, 24
    table = torch.from_numpy(tq.tq_rope_table(100, rot, 1e4, gain=1.5)).cuda()
    pos = i32([0, 1, 17, 99, 3, 50])
    X, dY = randn(1, "f32", T, H, D), randn(2, "f32", T, H, D)
    fwd = lambda x: tq.tq_rope(x, table, pos, interleaved=interleaved)  # noqa: E731
    dX = tq.tq_rope(dY, table, pos, interleaved=interleaved, inverse=True)
    freq = rope_frequencies_ref(rot, 1e4)
    # transpose of the oracle's map, column by column
    want = np.zeros((T, H, D))
    for d in range(D):
        e = np.zeros((T, H, D))
        e[..., d] = 1
        want[..., d] = (rope_ref(e, f64(pos).astype(int), freq, interleaved, False, 1.5)
                        * f64(dY)).sum(-1)
    bound = rope_bound(dY, want, "f32", 1.5, rot, interleaved)
    assert np.all(np.abs(f64(dX) - want) <= bound)
    for seed in (5, 6):
        step = randn(seed, "f32", T, H, D)
        diff = (f64(fwd(X + step)) - f64(fwd(X - step))) / 2
        lhs, rhs = (diff * f64(dY)).sum(), (f64(step) * f64(dX)).sum()
        mag = 3 * ((np.abs(f64(X)) + np.abs(f64(step))) .max() ** 2) * np.abs(f64(dY)).sum()
        assert abs(lhs - rhs) <= 2.0 ** -20 * mag


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,size,order", [
    (1, 64, 8, 128, 128, 16, "tokens"),
    (5, 6, 3, 80, 32, 24, "heads"),
    (37, 4, 4, 64, 64, 1, "tokens"),
    (3, 2, 1, 36, 12, 5, "heads"),
    (300, 4, 2, 64, 64, 16, "tokens"),
])
def test_rope_append(dtype, interleaved, T, Hq, Hkv, D, rot, size, order):
    rng = np.random.default_rng(T + D)
    P, width, n_pos = 2 * T + 3, 9, 8 * size
    freq = rope_frequencies_ref(rot, 1e4)
    table = torch.from_numpy(tq.tq_rope_table(n_pos, rot, 1e4)).cuda()
    shape = (P, size, Hkv, D) if order == "tokens" else (P, Hkv, size, D)
    k, v = (randn(s, dtype, *shape) for s in (1, 2))
    kv, vv = (x if order == "tokens" else x.transpose(1, 2) for x in (k, v))
    row = torch.zeros(T, Hq + 2 * Hkv + 1, D, dtype=DT[dtype], device="cuda")
    qkv = row[:, :-1]  # rows with room behind them
    qkv.copy_(randn(3, dtype, T, Hq + 2 * Hkv, D))
    pos = rng.integers(0, n_pos, T)
    seqs = rng.permutation(T + 2)[:T]
    pt = np.full((T + 2, width), -1)
    pages = rng.permutation(P)[:T]
    pt[seqs, pos // size] = pages
    k0, v0 = f64(kv), f64(vv)
    Q = tq.tq_rope_append(qkv, table, i32(pos), i32(pt), kv, vv, interleaved=interleaved,
                          seqs=i32(seqs))
    check_rope(Q, qkv[:, :Hq], i32(pos), freq, dtype, interleaved, False)
    got = kv[torch.as_tensor(pages), torch.as_tensor(pos % size)]
    check_rope(got, qkv[:, Hq:Hq + Hkv], i32(pos), freq, dtype, interleaved, False)
    assert torch.equal(vv[torch.as_tensor(pages), torch.as_tensor(pos % size)], qkv[:, Hq + Hkv:])
    # every other slot is as it was
    k1, v1 = f64(kv), f64(vv)
    k1[pages, pos % size] = k0[pages, pos % size]
    v1[pages, pos % size] = v0[pages, pos % size]
    assert np.array_equal(k1, k0) and np.array_equal(v1, v0)
    # the queries are tq_rope's bits
    assert torch.equal(Q, tq.tq_rope(qkv[:, :Hq], table, i32(pos), interleaved=interleaved))


def test_rope_append_leaves_out_what_has_no_slot():
    table = torch.from_numpy(tq.tq_rope_table(64, 16, 1e4)).cuda()
    T = 7
    qkv = randn(1, "f16", T, 4, 16)
    k = torch.zeros(3, 8, 1, 16, dtype=torch.float16, device="cuda")
    v = torch.zeros_like(k)
    #           ok  no position  past table  past width  bad page  bad row  ok
    pos = i32([0, -1, 64, 40, 9, 0, 17])
    seqs = i32([0, 0, 0, 0, 0, 9, 0])
    pt = i32([[2, 7, 1, -1], [0, 0, 0, 0]])
    Q = tq.tq_rope_append(qkv, table, pos, pt, k, v, seqs=seqs)
    assert torch.all(Q[[1, 2]] == 0) and torch.all(Q[[0, 3, 4, 5, 6]].abs().sum((1, 2)) > 0)
    written = (v.abs().sum((2, 3)) > 0).nonzero().tolist()
    assert written == [[1, 1], [2, 0]]
    assert torch.equal(v[2, 0], qkv[0, 3:]) and torch.equal(v[1, 1], qkv[6, 3:])


# ------------------------------------------------------------------ attention

def paged(seed, dtype, lens, Hq, Hkv, D, size, order="tokens", extra=3, poison=True, spread=1.0):
    """Q, cache and table of random values; slots that no sequence uses hold NaN."""
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, dtype=np.int64)
    need = -(-lens // size)
    width = max(1, int(need.max())) + 1
    P = int(need.sum()) + extra
    pt = np.full((len(lens), width), -1, np.int32)
    pt[np.arange(width)[None] < need[:, None]] = rng.permutation(P)[:need.sum()]
    shape = (P, size, Hkv, D)
    k, v = randn(seed, dtype, *shape), randn(seed + 1, dtype, *shape)
    if poison:
        used = np.zeros((P, size), bool)
        for b, n in enumerate(lens):
            for t in range(n):
                used[pt[b, t // size], t % size] = True
        off = torch.from_numpy(~used).cuda()
        k[off], v[off] = NAN, NAN
    if order == "heads":
        k, v = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (k, v))
    q = randn(seed + 2, dtype, len(lens), Hq, D) * spread
    return q, k, v, i32(pt), i32(lens)


def check_attention(got, lse, ref, dtype, D, n):
    out, lref, smag, vmag = ref
    ds = (D + 4) * 2.0 ** -24 * smag
    split = {"f16": 2.0 ** -20, "bf16": 2.0 ** -14}[dtype]
    rel = np.expm1(2 * ds) + split + (n + 16) * 2.0 ** -23 + n * 2.0 ** -38
    # the weight below the fp16 range is relative to the largest, times the largest |v|
    before = rel[..., None] * vmag
    bound = before + half_ulp(np.abs(out) + before, dtype)
    err = np.abs(f64(got) - out)
    assert np.all(err <= bound), float((err / np.maximum(bound, 1e-300)).max())
    if lse is not None:
        lg = f64(lse)
        assert np.array_equal(np.isfinite(lg), np.isfinite(lref))
        fin = np.isfinite(lref)
        lb = 2 * ds + (n + 16) * 2.0 ** -23 + 2.0 ** -21 * np.abs(lref)
        assert np.all(np.abs(lg[fin] - lref[fin]) <= lb[fin])


def run_attention(q, k, v, pt, lens, dtype, window=0, scale=None, **kw):
    D = q.shape[2]
    scale = D ** -0.5 if scale is None else scale
    out, lse = tq.tq_paged_attention(q, k, v, pt, lens, scale=scale, window=window,
                                     return_lse=True, **kw)
    ref = paged_attention_ref(f64(q), f64(k), f64(v), pt.cpu().numpy(), lens.cpu().numpy(), scale,
                              window)
    check_attention(out, lse, ref, dtype, D, max(1, int(lens.max())))
    return out, lse


EDGE = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 0, 300]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 1, 128), (4, 4, 64), (6, 2, 80), (16, 1, 96),
                                      (3, 3, 256), (5, 1, 200), (2, 2, 8), (7, 7, 32), (4, 2, 40)])
@pytest.mark.parametrize("size,order", [(16, "tokens"), (64, "heads"), (24, "tokens"), (1, "heads")])
def test_attention_edges(dtype, Hq, Hkv, D, size, order):
    q, k, v, pt, lens = paged(D + size, dtype, EDGE, Hq, Hkv, D, size, order)
    run_attention(q, k, v, pt, lens, dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("n,D", [(1, 128), (5, 64), (31, 128), (32, 80), (33, 128), (96, 128), (128, 64),
                                 (129, 128), (300, 128), (512, 128), (511, 64), (256, 256), (250, 192)])
def test_attention_short_tables(dtype, n, D):
    """Short tables: one workgroup per head, no joining."""
    size = 32
    q, k, v, pt, lens = paged(n, dtype, [n, max(0, n - 3), 0, n, n // 2], 8, 2, D, size)
    pt = pt[:, :max(1, -(-n // size))].contiguous()
    assert tq.tq_paged_attention_workspace(5, 8, 2, D, size, pt.shape[1]) == 0
    run_attention(q, k, v, pt, lens, dtype)


@pytest.mark.parametrize("Hq,Hkv", [(17, 1), (40, 1), (64, 2), (24, 24), (48, 16)])
def test_attention_head_groups(Hq, Hkv):
    """More query heads than one tile of 16, groups that do not fill it."""
    q, k, v, pt, lens = paged(Hq, "f16", [70, 1, 0, 200], Hq, Hkv, 64, 16)
    run_attention(q, k, v, pt, lens, "f16")


@pytest.mark.parametrize("window", [1, 2, 31, 32, 33, 100, 299, 300, 5000])
@pytest.mark.parametrize("size", [16, 24])
def test_attention_window(window, size):
    q, k, v, pt, lens = paged(window, "f16", EDGE, 4, 2, 64, size)
    run_attention(q, k, v, pt, lens, "f16", window=window)


def test_attention_freed_pages_before_the_window():
    """Pages that a window has left behind may be gone from the table."""
    q, k, v, pt, lens = paged(4, "bf16", [200, 90], 4, 2, 64, 16)
    pt[0, :8] = -1  # tokens 0..127
    pt[1, :1] = 10 ** 9
    run_attention(q, k, v, pt, lens, "bf16", window=60)
    run_attention(q, k, v, pt, lens, "bf16")  # without a window: their tokens are left out


def test_attention_absent_pages_everywhere():
    q, k, v, pt, lens = paged(5, "f16", [100, 100], 4, 2, 64, 24)
    pt[0] = -1
    out, lse = run_attention(q, k, v, pt, lens, "f16")
    assert torch.all(out[0] == 0) and torch.all(lse[0] == -math.inf)


def test_attention_lengths_outside_the_table():
    q, k, v, pt, lens = paged(6, "f16", [40, 33, 20], 4, 2, 64, 16)
    lens = i32([-5, 10 ** 9, 20])  # row 1: 33 tokens of two full pages and one named page
    pt[1, 3] = -1
    k, v = torch.nan_to_num(k), torch.nan_to_num(v)
    run_attention(q, k, v, pt, lens, "f16")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("spread", [0.0, 30.0])
def test_attention_flat_and_peaked(dtype, spread):
    """Equal scores, and scores of some hundreds that leave one token all weight."""
    q, k, v, pt, lens = paged(7, dtype, [700, 65, 1], 8, 2, 128, 16, spread=spread)
    run_attention(q, k, v, pt, lens, dtype, scale=0.5)


def test_attention_rising_scores():
    """A running maximum that grows at every tile, and one that never does."""
    for sign in (1, -1):
        q, k, v, pt, lens = paged(8, "f16", [1000], 2, 1, 64, 16, poison=False)
        order = pt[0, :63].long()
        ramp = sign * torch.arange(63 * 16, device="cuda").view(63, 16, 1, 1) / 64
        k[order] = (ramp * torch.ones(64, device="cuda")).half()
        q[:] = 0.25
        run_attention(q, k, v, pt, lens, "f16", scale=1.0)


def test_attention_extreme_values():
    """Scores at the type's lowest value, infinite keys and values, NaN."""
    q, k, v, pt, lens = paged(9, "f16", [50], 1, 1, 64, 16, poison=False)
    row = pt[0].long()
    base, _ = tq.tq_paged_attention(q, k, v, pt, lens, return_lse=True)
    # -inf scores leave their tokens out, also where it is every token
    q[:] = 1
    k2 = k.clone()
    k2[row[:3]] = -float("inf")
    out, lse = tq.tq_paged_attention(q, k2, v, pt, lens, return_lse=True)
    k3, n3 = k.clone(), k.clone()
    ref = paged_attention_ref(f64(q), f64(k3)[f64(row[3:4]).astype(int)], f64(v)[f64(row[3:4]).astype(int)],
                              np.array([[0]]), [2], 64 ** -0.5)
    check_attention(out, lse, ref, "f16", 64, 50)
    k2[:] = -float("inf")
    out, lse = tq.tq_paged_attention(q, k2, v, pt, lens, return_lse=True)
    assert torch.all(out == 0) and torch.all(lse == -math.inf)
    # the lowest finite score everywhere: the mean
    k2[:] = -65504
    out = tq.tq_paged_attention(q, k2, v, pt, lens, scale=1.0)
    mean = f64(v)[f64(row[:4]).astype(int)].reshape(-1, 1, 64)[:50].mean(0)
    assert np.abs(f64(out)[0] - mean).max() <= 2.0 ** -9 * np.abs(f64(v)).max()
    # infinite values count, and only in their number of the head
    v2 = v.clone()
    v2[row[0], 0, 0, 5] = float("inf")
    out = f64(tq.tq_paged_attention(q, k, v2, pt, lens))[0, 0]
    assert out[5] == np.inf and np.isfinite(np.delete(out, 5)).all()
    # one token: its weight is exactly 1, nothing remains for the low part
    for dt in (torch.float16, torch.bfloat16):
        one = tq.tq_paged_attention(q.to(dt), k.to(dt), v2.to(dt), pt, i32([1]))
        assert torch.equal(one[0, 0], v2[row[0], 0, 0].to(dt))
    n3[row[0], 0, 0, 5] = NAN
    assert torch.all(torch.isnan(tq.tq_paged_attention(q, n3, v, pt, lens)))


# Rows kept to a workgroup each, and rows split over all of them: either side of the
# number of rows, of the table's length and of the window's at which that changes;
# one, a few and many lengths a lane.
@pytest.mark.parametrize("B,Hq,Hkv,D,longest,window", [
    (150, 8, 8, 128, 60, 0), (128, 64, 8, 128, 40, 0), (129, 64, 8, 128, 40, 0),
    (33, 32, 2, 256, 40, 0), (300, 8, 8, 64, 50, 0), (700, 8, 8, 64, 40, 0),
    (1500, 2, 1, 64, 30, 0), (1200, 1, 1, 256, 30, 0), (2, 48, 3, 128, 512, 0),
    (2, 48, 3, 128, 513, 0), (6, 8, 2, 128, 1500, 482), (6, 8, 2, 128, 1500, 483),
    (6, 8, 2, 256, 1500, 226), (6, 8, 2, 256, 1500, 227), (70, 16, 1, 64, 400, 33),
    (64, 2, 2, 128, 1024, 0), (64, 2, 2, 128, 1025, 0), (128, 3, 1, 80, 1024, 900),
    (63, 2, 2, 64, 1000, 0),
    (5, 5, 5, 80, 900, 1)])
def test_attention_many_rows(B, Hq, Hkv, D, longest, window):
    rng = np.random.default_rng(B + D)
    lens = rng.integers(0, longest + 1, B)
    lens[rng.integers(0, B, B // 5)] = 0
    lens[-1] = longest
    q, k, v, pt, lens = paged(13, "bf16" if D == 64 else "f16", lens, Hq, Hkv, D, 16)
    run_attention(q, k, v, pt[:, :-(-longest // 16)].contiguous(), lens,
                  "bf16" if D == 64 else "f16", window=window)


@pytest.mark.parametrize("D,size", [(64, 16), (128, 24), (256, 32)])
def test_attention_weight_of_zero(D, size):
    """A bf16 token of weight e^-400 leaves no trace, however large its value."""
    q, k, v, pt, lens = paged(12, "bf16", [70], 3, 1, D, size)
    q[:] = 1
    k.zero_()
    v[pt[0, 0].long(), 3] = 3e38
    k[pt[0, 0].long(), 3] = -400 / D  # exact in bf16
    assert torch.all(k[pt[0, 0].long(), 3].float() == -400 / D)
    run_attention(q, k, v, pt, lens, "bf16", scale=1.0)


@pytest.mark.parametrize("dtype,size,D", [("f16", 64, 128), ("bf16", 16, 128), ("f16", 24, 128),
                                          ("f16", 16, 256), ("bf16", 32, 64), ("f16", 16, 80)])
def test_attention_long(dtype, size, D):
    """One sequence over every workgroup (the split and its joining), against fp64
    on the GPU; the oracle's loops would take minutes."""
    n, Hq, Hkv = 70001, 8, 2
    q, k, v, pt, lens = paged(10, dtype, [n], Hq, Hkv, D, size, poison=False)
    out, lse = tq.tq_paged_attention(q, k, v, pt, lens, return_lse=True)
    ids = pt[0, :-(-n // size)].long()
    kk = k[ids].flatten(0, 1)[:n].double()
    vv = v[ids].flatten(0, 1)[:n].double()
    for h in range(Hq):
        qh = q[0, h].double()
        s = kk[:, h // 4] @ qh / math.sqrt(D)
        w = torch.softmax(s, 0)
        smag = float((kk[:, h // 4].abs() @ qh.abs()).max()) / math.sqrt(D)
        ref = (f64(vv[:, h // 4].t().contiguous() @ w)[None, None],
               f64(torch.logsumexp(s, 0))[None, None], np.array([[smag]]),
               f64(vv[:, h // 4].abs().t().contiguous() @ w)[None, None])
        check_attention(out[:, h:h + 1], lse[:, h:h + 1], ref, dtype, D, n)


def test_attention_many_sequences():
    """More sequences than a workgroup has threads, most of them short or empty."""
    lens = np.random.default_rng(0).integers(0, 40, 700)
    lens[[5, 300, 699]] = [0, 1500, 900]
    lens[600:650] = 0
    q, k, v, pt, lens = paged(11, "f16", lens, 4, 2, 64, 16)
    run_attention(q, k, v, pt, lens, "f16")


def test_attention_all_empty():
    q, k, v, pt, lens = paged(12, "f16", [300] * 5, 4, 2, 64, 16)
    out, lse = tq.tq_paged_attention(q, k, v, pt, torch.zeros_like(lens), return_lse=True)
    assert torch.all(out == 0) and torch.all(lse == -math.inf)
    assert tq.tq_paged_attention(q[:0], k, v, pt[:0], lens[:0]).shape == (0, 4, 64)


def test_attention_query_strides():
    """Queries inside the rows of a q/k/v product, and [Hq][B][D] order."""
    q, k, v, pt, lens = paged(13, "f16", [70, 3, 129], 4, 2, 64, 16)
    want = tq.tq_paged_attention(q, k, v, pt, lens)
    wide = torch.zeros(3, 8, 64, dtype=torch.float16, device="cuda")
    wide[:, :4] = q
    assert torch.equal(tq.tq_paged_attention(wide[:, :4], k, v, pt, lens), want)
    turned = q.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(tq.tq_paged_attention(turned, k, v, pt, lens), want)
    out = torch.empty_like(want)
    assert tq.tq_paged_attention(q, k, v, pt, lens, out=out) is out and torch.equal(out, want)


def test_attention_offsets_past_32_bits():
    """Pages that lie more than 4 GiB apart, for both kinds of page size, and the
    append that writes them."""
    for size in (16, 24):
        far = 1200 * 1000 * 1000  # numbers between pages: 2.4 GB
        base = torch.empty(2 * far + 4096 * 8, dtype=torch.float16, device="cuda")
        k = base.as_strided((3, size, 2, 64), (far, 128, 64, 1))
        v = base.as_strided((3, size, 2, 64), (far, 128, 64, 1), 8192)
        k.copy_(randn(1, "f16", 3, size, 2, 64))
        v.copy_(randn(2, "f16", 3, size, 2, 64))
        pt, lens = i32([[2, 0, 1], [1, -1, -1]]), i32([3 * size - 2, 5])
        q = randn(3, "f16", 2, 4, 64)
        run_attention(q, k, v, pt, lens, "f16")
        table = torch.from_numpy(tq.tq_rope_table(100, 64, 1e4)).cuda()
        qkv = randn(4, "f16", 2, 8, 64)
        tq.tq_rope_append(qkv, table, i32([1, 6]), pt, k, v)
        assert torch.equal(v[2, 1], qkv[0, 6:]) and torch.equal(v[1, 6], qkv[1, 6:])
        del base, k, v


def test_attention_repeats_and_streams():
    """The same bits on every call, on another stream, and with a shared workspace."""
    q, k, v, pt, lens = paged(14, "f16", [3000, 1, 777, 64], 8, 2, 128, 16)
    want, lw = tq.tq_paged_attention(q, k, v, pt, lens, return_lse=True)
    n = tq.tq_paged_attention_workspace(4, 8, 2, 128, 16, pt.shape[1])
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for i in range(5):
        out, lse = tq.tq_paged_attention(q, k, v, pt, lens, return_lse=True, workspace=ws)
        assert torch.equal(out, want) and torch.equal(lse, lw)
    torch.cuda.synchronize()
    got = [tq.tq_paged_attention(q, k, v, pt, lens, stream=side.cuda_stream) for _ in range(5)]
    side.synchronize()
    assert all(torch.equal(g, want) for g in got)
    with torch.cuda.stream(side):  # stream 0 while another one is current
        out = tq.tq_paged_attention(q, k, v, pt, lens, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_compiled_and_python_calls_agree():
    """The compiled form of each call and the Python one (taken when a stream is
    named) give the same bits, and a refusal of the C ABI reaches the caller from both."""
    q, k, v, pt, lens = paged(16, "bf16", [100, 700, 0], 8, 2, 64, 16, poison=False)
    table = torch.from_numpy(tq.tq_rope_table(1024, 64)).cuda()
    qkv, pool, parent = randn(2, "bf16", 3, 12, 64), torch.stack([k, v]), i32([1, 1, 0])
    s = torch.cuda.current_stream().cuda_stream

    def calls(**kw):
        kc, vc = k.clone(), v.clone()
        pc, pd = pool.clone(), pool.clone()
        out = [tq.tq_rope(qkv[:, :10], table, lens, interleaved=True, **kw),
               tq.tq_rope(qkv.float(), table, lens, inverse=True, **kw),
               tq.tq_rope_append(qkv, table, i32([0, 1, 2]), pt, kc, vc, **kw), kc, vc,
               tq.tq_rope_append(qkv, table, i32([0, 1, 2]), pt, kc, vc, True, i32([1, 0, 1]), **kw),
               tq.tq_paged_attention(q, k, v, pt, lens, **kw),
               *tq.tq_paged_attention(q, k, v, pt, lens, 0.5, 50, return_lse=True, **kw),
               *tq.tq_pages_fork(pc, pt, lens, parent, 16, **kw), pc,
               *tq.tq_pages_grow(pt, lens, i32([1, 90, 5]), k.shape[0], 16, **kw),
               *tq.tq_pages_compact(pd, pt, lens, 16, **kw), pd]
        return out

    a, b = calls(), calls(stream=s)
    assert len(a) == len(b)
    for x, y in zip(a, b):
        assert x.dtype == y.dtype and x.shape == y.shape and torch.equal(x, y)
    for kw in ({}, {"stream": s}):
        for bad in (lambda: tq.tq_pages_fork(pool, pt, lens, parent, 0, **kw),
                    lambda: tq.tq_pages_grow(pt, lens, lens, 0, 16, **kw),
                    lambda: tq.tq_pages_compact(pool, pt, lens, -1, **kw),
                    lambda: tq.tq_paged_attention(q, k, v, pt, lens, window=-1, **kw),
                    lambda: tq.tq_paged_attention(q, k, v, pt, lens, float("nan"), **kw),
                    lambda: tq.tq_paged_attention(q.cpu(), k, v, pt, lens, **kw),
                    lambda: tq.tq_rope(qkv, table, lens.cpu(), **kw),
                    lambda: tq.tq_rope(qkv.double(), table, lens, **kw),
                    lambda: tq.tq_rope_append(qkv, table, lens, pt, k, v.half(), **kw)):
            with pytest.raises(tq.TQError):
                bad()


def test_decode_ops_in_a_graph():
    """Append, attention and the page operators captured once and replayed, against
    the eager results, with eager work between the replays."""
    q, k, v, pt, lens = paged(15, "f16", [500, 33, 0], 8, 2, 64, 16, poison=False)
    pool = torch.stack([k, v])
    table = torch.from_numpy(tq.tq_rope_table(1024, 64, 1e4)).cuda()
    qkv = randn(1, "f16", 3, 12, 64)
    add, parent = i32([1, 1, 1]), i32([0, 0, 1])

    def step():
        t1, n1, short = tq.tq_pages_grow(pt, lens, add, pool.shape[1], 16)
        Q = tq.tq_rope_append(qkv, table, lens, t1, pool[0], pool[1])
        out = tq.tq_paged_attention(Q, pool[0], pool[1], t1, n1)
        t2, n2, refs, _ = tq.tq_pages_fork(pool, t1, n1, parent, 16)
        t3, used = tq.tq_pages_compact(pool, t2, n2, 16)
        return t1, n1, short, Q, out, t2, n2, refs, t3, used

    start = pool.clone()
    eager = [x.clone() for x in step()]
    pool_after = pool.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pool.copy_(start)
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(4):
        pool.copy_(start)
        for x in held:
            x.fill_(77)
        torch.cuda.synchronize()
        graph.replay()
        assert torch.equal(pool, pool_after), i
        for a, b in zip(held, eager):
            assert torch.equal(a, b), i
        _ = torch.randn(1000, device="cuda").sum().item()


# ------------------------------------------------------------------ pages

def random_state(rng, rows, width, P, size, share=True):
    """A table whose rows share some full pages, plus stale entries past the held ones."""
    table = rng.integers(-1, P, (rows, width)).astype(np.int32)
    lens = np.zeros(rows, np.int32)
    free = list(rng.permutation(P))
    for r in range(rows):
        n = int(rng.integers(0, width + 1))
        n = min(n, len(free))
        tokens = max(0, n * size - int(rng.integers(0, size))) if n else 0
        n = -(-tokens // size)
        for j in range(n):
            if share and r and rng.random() < 0.4 and (j + 1) * size <= tokens:
                other = int(rng.integers(0, r))
                if j < lens[other] // size:
                    table[r, j] = table[other, j]
                    continue
            table[r, j] = free.pop()
        lens[r] = tokens
    return table, lens


def make_pool(seed, planes, P, size, dtype="f16", D=8):
    return randn(seed, dtype, planes, P, size, 1, D)


@pytest.mark.parametrize("rows,width,P,size", [(1, 1, 1, 1), (3, 4, 33, 16), (8, 6, 40, 5),
                                               (20, 9, 300, 16), (1100, 3, 5000, 2)])
def test_pages_fork(rows, width, P, size):
    for seed in range(4):
        rng = np.random.default_rng(seed)
        table, lens = random_state(rng, rows, width, P, size)
        new = int(rng.integers(1, 2 * rows + 1))
        parent = rng.integers(-1, rows + 1, new)
        if seed == 3:
            parent[:] = 0  # everyone continues the first
        pool = make_pool(seed, 3, P, size)
        want_t, want_n, refs, short, copies = pages_fork_ref(table, lens, parent, P, size)
        want_pool = pool.clone()
        for s, d in copies:
            want_pool[:, d] = pool[:, s]
        t, n, r, sh = tq.tq_pages_fork(pool, i32(table), i32(lens), i32(parent), size)
        assert np.array_equal(t.cpu().numpy(), want_t)
        assert np.array_equal(n.cpu().numpy(), want_n)
        assert np.array_equal(r.cpu().numpy(), refs) and int(sh) == short
        assert torch.equal(pool, want_pool)


def test_pages_fork_shortage_and_odd_entries():
    # four pages, all held: a copy finds none until a row is dropped
    table, lens = [[0, 1], [2, 3]], [5, 8]
    pool = make_pool(1, 2, 4, 4)
    for parent in ([0, 0, 1], [0, 0, -1], [0, 0, 0, 0], [0, 7, 0]):
        want = pages_fork_ref(table, lens, parent, 4, 4)
        before = pool.clone()
        t, n, r, sh = tq.tq_pages_fork(pool, i32(table), i32(lens), i32(parent), 4)
        assert np.array_equal(t.cpu().numpy(), want[0]) and np.array_equal(n.cpu(), want[1])
        assert np.array_equal(r.cpu().numpy(), want[2]) and int(sh) == want[3]
        for s, d in want[4]:
            before[:, d] = before[:, s]
        assert torch.equal(pool, before)
    # entries that name no page are kept and never followed; lengths are clamped
    table, lens = [[9, -3], [1, 10 ** 9]], [7, 100]
    want = pages_fork_ref(table, lens, [0, 0, 1, 1], 4, 4)
    t, n, r, sh = tq.tq_pages_fork(pool, i32(table), i32(lens), i32([0, 0, 1, 1]), 4)
    assert np.array_equal(t.cpu().numpy(), want[0]) and np.array_equal(n.cpu(), want[1])
    assert np.array_equal(r.cpu().numpy(), want[2])
    # no rows: everything is free
    t, n, r, sh = tq.tq_pages_fork(pool, i32(table), i32(lens), i32([]), 4)
    assert t.shape == (0, 2) and torch.all(r == 0) and int(sh) == 0


@pytest.mark.parametrize("rows,width,P,size", [(1, 2, 3, 4), (5, 8, 64, 16), (9, 7, 31, 3),
                                               (1500, 4, 4000, 2), (70, 40, 1000, 1)])
def test_pages_grow(rows, width, P, size):
    for seed in range(4):
        rng = np.random.default_rng(seed)
        table, lens = random_state(rng, rows, width, P, size)
        add = rng.integers(-1, 3 * size, rows) if seed else np.ones(rows)
        if seed == 2:
            add[rng.integers(0, rows)] = 2 ** 31 - 1
        want = pages_grow_ref(table, lens, add, P, size)
        t, n, refused = tq.tq_pages_grow(i32(table), i32(lens), i32(add), P, size)
        assert np.array_equal(t.cpu().numpy(), want[0])
        assert np.array_equal(n.cpu().numpy(), want[1]) and int(refused) == want[2]


@pytest.mark.parametrize("rows,width,P,size", [(1, 1, 1, 4), (4, 5, 33, 16), (30, 9, 64, 3),
                                               (900, 5, 6001, 2)])
def test_pages_compact(rows, width, P, size):
    for seed in range(4):
        rng = np.random.default_rng(seed + 50)
        table, lens = random_state(rng, rows, width, P, size)
        if seed == 1:
            lens[:] = 0
        pool = make_pool(seed, 2, P, size, "bf16")
        want_t, used, moves = pages_compact_ref(table, lens, P, size)
        want_pool = pool.clone()
        for s, d in moves:
            want_pool[:, d] = pool[:, s]
        t, u = tq.tq_pages_compact(pool, i32(table), i32(lens), size)
        assert np.array_equal(t.cpu().numpy(), want_t) and int(u) == used
        assert torch.equal(pool, want_pool)
        # a compact pool stays as it is
        t2, u2 = tq.tq_pages_compact(pool, t, i32(lens), size)
        assert torch.equal(t2, t) and int(u2) == used and torch.equal(pool, want_pool)


# Either side of the sizes at which the bookkeeping changes its form (one launch for
# everything, one workgroup in LDS, three kernels), with pages of one and two pieces.
@pytest.mark.parametrize("rows,width,P,size,planes,D", [
    (64, 12, 1000, 4, 2, 8), (65, 12, 1000, 4, 2, 8), (64, 12, 1000, 4, 9, 8),
    (256, 5, 1500, 3, 1, 8), (257, 5, 1500, 3, 1, 8), (64, 128, 600, 2, 1, 8),
    (63, 131, 600, 2, 1, 8), (10, 40, 4096, 2, 1, 8), (10, 40, 4097, 2, 1, 8),
    (10, 40, 8192, 2, 1, 8), (10, 40, 8193, 2, 1, 8), (12, 4, 60, 33, 3, 1000),
    (70, 4, 350, 33, 2, 1000), (3, 400, 1100, 1, 1, 8)])
def test_pages_forms(rows, width, P, size, planes, D):
    rng = np.random.default_rng(rows + P)
    table, lens = random_state(rng, rows, width, P, size)
    table_dev, lens_dev = i32(table), i32(lens)
    pool = make_pool(5, planes, P, size, D=D)
    want_t, used, moves = pages_compact_ref(table, lens, P, size)
    want_pool = pool.clone()
    for s, d in moves:
        want_pool[:, d] = pool[:, s]
    t, u = tq.tq_pages_compact(pool, table_dev, lens_dev, size)
    assert np.array_equal(t.cpu().numpy(), want_t) and int(u) == used
    assert torch.equal(pool, want_pool)
    parent = rng.integers(0, max(1, rows // 2), rows)
    want_t, want_n, refs, short, copies = pages_fork_ref(table, lens, parent, P, size)
    for s, d in copies:
        want_pool[:, d] = pool[:, s]
    t, n, r, sh = tq.tq_pages_fork(pool, table_dev, lens_dev, i32(parent), size)
    assert np.array_equal(t.cpu().numpy(), want_t) and np.array_equal(n.cpu().numpy(), want_n)
    assert np.array_equal(r.cpu().numpy(), refs) and int(sh) == short
    assert torch.equal(pool, want_pool)
    add = rng.integers(0, 2 * size + 1, rows)
    want = pages_grow_ref(table, lens, add, P, size)
    t, n, refused = tq.tq_pages_grow(table_dev, lens_dev, i32(add), P, size)
    assert np.array_equal(t.cpu().numpy(), want[0])
    assert np.array_equal(n.cpu().numpy(), want[1]) and int(refused) == want[2]


@pytest.mark.parametrize("shape", [(1, 2, 8), (3, 9, 16, 1, 24), (2, 5, 64, 4, 128), (1, 300, 8)])
def test_pages_copy(shape):
    pool = randn(1, "f16", *shape)
    P = shape[1]
    rng = np.random.default_rng(P)
    pages = rng.permutation(P)
    n = P // 2
    src, dst = pages[:n].copy(), pages[n:2 * n].copy()
    if n > 2:
        src[0], dst[1] = -1, P  # left out
    want = pool.clone()
    for s, d in zip(src, dst):
        if 0 <= s < P and 0 <= d < P:
            want[:, d] = want[:, s]
    tq.tq_pages_copy(pool, i32(src), i32(dst))
    assert torch.equal(pool, want)
    tq.tq_pages_copy(pool, i32([]), i32([]))
    assert torch.equal(pool, want)


def test_pages_past_32_bits():
    """A pool of more than 4 GiB: the last page to the first of each plane."""
    pool = torch.empty(2, 5, 300 * 1000 * 1000, dtype=torch.float16, device="cuda")
    pool[:, 0] = 0
    pool[:, 4] = randn(1, "f16", 2, 1000).repeat(1, 300 * 1000)
    tq.tq_pages_copy(pool, i32([4]), i32([0]))
    assert torch.equal(pool[:, 0], pool[:, 4])
    pool[:, 0] = 0
    t, used = tq.tq_pages_compact(pool, i32([[4]]), i32([3]), 16)
    assert t.tolist() == [[0]] and int(used) == 1 and torch.equal(pool[:, 0], pool[:, 4])
