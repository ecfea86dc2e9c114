"""GPU parity of the operators on drafted trees against the fp64 oracle.

Bounds as derived in test_decode_gpu.py, with the rounding of a weight: where up to 32
rows share a key-value head (nodes times heads of the group) as in tq_paged_attention,
with more of them one 16-bit number, rounded to nearest: of p significant bits, so that
half a step at 2^e is 2^(e - p), off by 2^-p of itself at most (fp16 2^-11, bf16 2^-8).
fp16's least step is 2^-24, and the row's largest weight enters as 2^9 at least (so that the
sum of the others stays below fp16's range while the maximum that they are measured from lags
by a factor of 2^6): a small weight is off by 2^-25 / 2^9 = 2^-34 of the largest at most,
n of them by n 2^-34 of the sum, which holds the largest.
"""

import numpy as np
import pytest

from oracle import mask_words_ref, tree_attention_ref, tree_paths_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
tq = pytest.importorskip("bit_mixed_precision_amd.binding")

from test_decode_gpu import DT, NAN, f64, half_ulp, i32, randn  # noqa: E402


def parents_of(seed, B, T, deep=2.0):
    rng = np.random.default_rng(seed)
    back = 1 + np.floor(rng.exponential(deep, (B, T))).astype(int) if deep else np.ones((B, T), int)
    return np.maximum(np.arange(T) - back, -1).astype(np.int32)


def tree(seed, dtype, lens, nodes, T, Hq, Hkv, D, size, poison=True, extra=3, spread=1.0):
    """Q [B][T][Hq][D], cache, table, lens, nodes; slots of no token hold NaN."""
    rng = np.random.default_rng(seed)
    lens, nodes = np.asarray(lens), np.asarray(nodes)
    total = lens + nodes
    need = -(-total // size)
    width = max(1, int(need.max())) + 1
    P = int(need.sum()) + extra
    pt = np.full((len(lens), width), -1, np.int32)
    pt[np.arange(width)[None] < need[:, None]] = rng.permutation(P)[:need.sum()]
    k, v = randn(seed, dtype, P, size, Hkv, D), randn(seed + 1, dtype, P, size, Hkv, D)
    if poison:
        used = np.zeros((P, size), bool)
        for b, n in enumerate(total):
            t = np.arange(n)
            used[pt[b, t // size], t % size] = True
        off = torch.from_numpy(~used).cuda()
        k[off], v[off] = NAN, NAN
    q = randn(seed + 2, dtype, len(lens), T, Hq, D) * spread
    return q, k, v, i32(pt), i32(lens), i32(nodes)


def words(sees):
    return torch.from_numpy(mask_words_ref(sees)).cuda()


def check(got, lse, ref, dtype, D, rows, n):
    out, lref, smag, vmag = ref
    ds = (D + 4) * 2.0 ** -24 * smag
    weight = {"f16": 2.0 ** -20 if rows <= 32 else 2.0 ** -11,
              "bf16": 2.0 ** -14 if rows <= 32 else 2.0 ** -8}[dtype]
    rel = np.expm1(2 * ds) + weight + (n + 16) * 2.0 ** -23 + n * 2.0 ** -34
    before = rel[..., None] * vmag
    bound = before + half_ulp(np.abs(out) + before, dtype)
    err = np.abs(f64(got) - out)
    assert np.all(err <= bound), float(np.nanmax(err / np.maximum(bound, 1e-300)))
    lg = f64(lse)
    assert np.array_equal(lg == -np.inf, lref == -np.inf)
    fin = np.isfinite(lref)
    lb = 2 * ds + (n + 16) * 2.0 ** -23 + 2.0 ** -21 * np.abs(lref)
    assert np.all(np.abs(lg[fin] - lref[fin]) <= lb[fin])


def run(q, k, v, pt, lens, nodes, sees, dtype, window=0, scale=None, chain=False, **kw):
    B, T, Hq, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    mask = None if chain else words(sees)
    out, lse = tq.tq_tree_attention(q, k, v, pt, lens, mask=mask, nodes=nodes, scale=scale,
                                    window=window, return_lse=True, **kw)
    m = np.full(B, T) if nodes is None else nodes.cpu().numpy()
    ref = tree_attention_ref(f64(q), f64(k), f64(v), pt.cpu().numpy(), lens.cpu().numpy(), m, sees,
                             scale, window)
    check(out, lse, ref, dtype, D, T * (Hq // k.shape[2]), max(1, int(lens.max()) + T))
    return out, lse


@pytest.mark.parametrize("B,T", [(1, 1), (1, 2), (3, 24), (5, 63), (2, 64), (4, 65), (7, 130), (2, 256)])
@pytest.mark.parametrize("deep", [0.0, 1.0, 20.0])
def test_mask(B, T, deep):
    p = parents_of(T, B, T, deep)
    mask, depth = tq.tq_tree_mask(torch.from_numpy(p).cuda())
    sees = tree_paths_ref(p)
    assert np.array_equal(mask.cpu().numpy(), mask_words_ref(sees))
    assert np.array_equal(depth.cpu().numpy(), sees.sum(-1) - 1)


def test_mask_parents_that_are_no_nodes():
    """Itself, a later node, numbers far out: all of them roots."""
    p = np.array([[5, 1, 7, -9, 2 ** 31 - 1, -2 ** 31, 3, 6]], np.int32)
    mask, depth = tq.tq_tree_mask(torch.from_numpy(p).cuda())
    assert np.array_equal(mask.cpu().numpy(), mask_words_ref(tree_paths_ref(p)))
    assert depth.tolist() == [[0, 0, 0, 0, 0, 0, 1, 2]]


EDGE = [0, 1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,Hq,Hkv,D,size", [
    (1, 4, 4, 64, 16), (3, 8, 1, 128, 16), (4, 16, 2, 128, 32), (24, 8, 1, 128, 16),
    (13, 6, 6, 64, 24), (17, 6, 2, 80, 5), (9, 4, 1, 256, 16), (40, 6, 3, 96, 1),
    (2, 5, 5, 8, 16), (65, 4, 2, 128, 64), (7, 33, 1, 192, 16), (3, 4, 4, 256, 24)])
def test_lengths_around_tiles(dtype, T, Hq, Hkv, D, size):
    B = len(EDGE)
    rng = np.random.default_rng(T)
    nodes = rng.integers(0, T + 1, B)
    nodes[:2] = T
    args = tree(T + D, dtype, EDGE, nodes, T, Hq, Hkv, D, size)
    run(*args, tree_paths_ref(parents_of(D, B, T)), dtype)


@pytest.mark.parametrize("dtype,T,Hq,Hkv,D,lens", [
    ("f16", 24, 64, 8, 128, [97]), ("f16", 16, 16, 2, 128, [9000]), ("bf16", 2, 8, 8, 64, [7000, 5, 2300]),
    ("bf16", 40, 8, 1, 128, [3000, 0, 1, 4000]), ("f16", 5, 16, 8, 256, [2500]), ("bf16", 70, 2, 1, 80, [1500, 900]),
    ("f16", 256, 8, 2, 64, [700, 20])])
def test_long(dtype, T, Hq, Hkv, D, lens):
    """Rows cut between workgroups; nodes NULL, and the chain that no mask gives."""
    B = len(lens)
    q, k, v, pt, lens, nodes = tree(T, dtype, lens, [T] * B, T, Hq, Hkv, D, 16)
    sees = tree_paths_ref(parents_of(T, B, T))
    out, lse = run(q, k, v, pt, lens, None, sees, dtype)
    again = tq.tq_tree_attention(q, k, v, pt, lens, mask=words(sees), return_lse=True)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    chain = np.tril(np.ones((1, T, T), bool)).repeat(B, 0)
    run(q, k, v, pt, lens, nodes, chain, dtype, chain=True)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,Hq,Hkv,D", [(4, 8, 2, 64), (30, 8, 2, 128)])
def test_any_bits(dtype, T, Hq, Hkv, D):
    """Masks that are no trees: random bits, bits past the nodes, rows of none, one mask for
    all sequences, and rows without a single token."""
    lens = [0, 0, 1, 40, 200, 64]
    B = len(lens)
    rng = np.random.default_rng(1)
    sees = rng.random((B, T, T)) < 0.4
    sees[:, 1] = False
    sees[0, :] = False
    nodes = [T, T - 1, 1, T, T - 2, 0]
    args = tree(5, dtype, lens, nodes, T, Hq, Hkv, D, 16)
    out, lse = run(*args, sees, dtype)
    assert not out[0].any() and torch.all(lse[0] == -np.inf)
    one = words(sees[3:4])
    got = tq.tq_tree_attention(*args[:5], mask=one[0], nodes=args[5], return_lse=True)
    same = tq.tq_tree_attention(*args[:5], mask=one.expand(B, -1, -1).contiguous(), nodes=args[5], return_lse=True)
    third = tq.tq_tree_attention(*args[:5], mask=one, nodes=args[5], return_lse=True)
    for x, y, z in zip(got, same, third):
        assert torch.equal(x, y) and torch.equal(x, z)


@pytest.mark.parametrize("window", [12, 13, 50, 64, 200, 1 << 40])
@pytest.mark.parametrize("Hq", [2, 16])
def test_window(window, Hq):
    lens = [0, 3, 40, 64, 129, 300]
    T = 12
    args = tree(window % 97, "f16", lens, [12, 12, 3, 12, 7, 12], T, Hq, 1, 64, 16)
    run(*args, tree_paths_ref(parents_of(3, len(lens), T)), "f16", window=window)


@pytest.mark.parametrize("T,Hq", [(4, 8), (20, 8)])
@pytest.mark.parametrize("scale", [0.0, -0.2, 30.0])
def test_scales(T, Hq, scale):
    args = tree(9, "bf16", [100, 0, 257], [T, T, T], T, Hq, 1, 64, 16)
    run(*args, tree_paths_ref(parents_of(4, 3, T)), "bf16", scale=scale)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,Hq,D", [(4, 8, 64), (20, 8, 128), (6, 2, 96)])
def test_what_is_not_seen_has_no_influence(dtype, T, Hq, D):
    """Infinite and undefined keys and values of drafted tokens, and of tokens before
    the windows: rows that do not see them keep their bits."""
    lens = [70, 5, 0]
    q, k, v, pt, lens, nodes = tree(11, dtype, lens, [T] * 3, T, Hq, 1, D, 16, poison=False)
    p = parents_of(8, 3, T, 3.0)
    sees = tree_paths_ref(p)
    for window in (0, T + 20):
        kw = dict(mask=words(sees), nodes=nodes, window=window, return_lse=True)
        want = tq.tq_tree_attention(q, k, v, pt, lens, **kw)
        for bad in (float("inf"), -float("inf"), NAN):
            kk, vv = k.clone(), v.clone()
            for b in range(3):
                t = int(lens[b]) + 2
                kk[pt[b, t // 16].long(), t % 16] = bad
                vv[pt[b, t // 16].long(), t % 16] = bad
            if window:  # tokens that only some of the first sequence's nodes see
                kk[pt[0, 3].long(), 2:8], vv[pt[0, 3].long(), 2:8] = bad, bad
            got = tq.tq_tree_attention(q, kk, vv, pt, lens, **kw)
            clean = torch.from_numpy(~sees[:, :, 2]).cuda()
            if window:
                low = 70 + sees[0].sum(-1) - window
                clean[0] &= torch.from_numpy(low > 55).cuda()
            assert clean.any() and not clean.all()
            for x, y in zip(got, want):
                assert torch.equal(x[clean], y[clean])
            assert not torch.isfinite(got[1][~clean]).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,Hq", [(4, 8), (20, 8)])
def test_infinite_values_reach_those_who_see_them(dtype, T, Hq):
    q, k, v, pt, lens, nodes = tree(12, dtype, [40, 0], [T, T], T, Hq, 1, 64, 16)
    sees = tree_paths_ref(parents_of(5, 2, T))
    for b, n in enumerate((40, 0)):
        t = n + 1
        v[pt[b, t // 16].long(), t % 16, 0, 3] = float("inf")
        v[pt[b, t // 16].long(), t % 16, 0, 4] = -float("inf")
        v[pt[b, t // 16].long(), t % 16, 0, 9] = NAN
    out = tq.tq_tree_attention(q, k, v, pt, lens, mask=words(sees), nodes=nodes)
    on = torch.from_numpy(sees[:, :, 1]).cuda()
    assert torch.all(out[on][..., 3] == float("inf")) and torch.all(out[on][..., 4] == -float("inf"))
    assert torch.isnan(out[on][..., 9]).all()
    rest = [d for d in range(64) if d not in (3, 4, 9)]
    assert torch.isfinite(out[on][..., rest]).all() and torch.isfinite(out[~on]).all()


def test_absent_pages_and_lengths_out_of_range():
    T = 5
    q, k, v, pt, lens, nodes = tree(13, "f16", [100, 40, 70, 16], [T] * 4, T, 8, 2, 64, 16, poison=False)
    pt[0, 1], pt[0, 3], pt[2, 4], pt[3, 1] = -1, 10 ** 6, -5, 2 ** 31 - 1
    sees = tree_paths_ref(parents_of(6, 4, T))
    run(q, k, v, pt, lens, nodes, sees, "f16")
    # negative and too long lengths, more nodes than there are rows or slots
    pt[1] = torch.arange(pt.shape[1], device="cuda")
    lens[0], lens[1], nodes[2], nodes[3] = -7, 10 ** 9, 99, -3
    ref = tree_attention_ref(f64(q), f64(k), f64(v), pt.cpu().numpy(), lens.cpu().numpy(),
                             np.clip(nodes.cpu().numpy(), 0, T), sees, 0.125)
    out, lse = tq.tq_tree_attention(q, k, v, pt, lens, mask=words(sees), nodes=nodes, return_lse=True)
    check(out, lse, ref, "f16", 64, T * 4, 200)


@pytest.mark.parametrize("rows", [8, 64])
def test_strides(rows):
    """Queries inside the rows of a fused product, [Hq][T] order, caches by heads and
    interleaved with each other."""
    T, Hq, Hkv, D = rows // 4, 8, 2, 64
    q, k, v, pt, lens, nodes = tree(14, "bf16", [33, 200], [T, T], T, Hq, Hkv, D, 16, poison=False)
    sees = tree_paths_ref(parents_of(7, 2, T))
    want, _ = run(q, k, v, pt, lens, nodes, sees, "bf16")
    wide = torch.full((2, T, Hq + 2 * Hkv, D), NAN, dtype=q.dtype, device="cuda")
    wide[:, :, :Hq] = q
    both = torch.stack([k, v], 2)
    turned = q.permute(2, 1, 0, 3).contiguous().permute(2, 1, 0, 3)
    by_heads = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in (k, v)]
    for qq, kk, vv in ((wide[:, :, :Hq], k, v), (turned, k, v), (q, both[:, :, 0], both[:, :, 1]),
                       (q, *by_heads)):
        out = tq.tq_tree_attention(qq, kk, vv, pt, lens, mask=words(sees), nodes=nodes)
        assert torch.equal(out, want)
    out = torch.empty_like(q)
    ws = torch.empty(tq.tq_tree_attention_workspace(2, T, Hq, Hkv, D, 16, pt.shape[1]) + 16,
                     dtype=torch.uint8, device="cuda")
    assert tq.tq_tree_attention(q, k, v, pt, lens, mask=words(sees), nodes=nodes, out=out, workspace=ws) is out
    assert torch.equal(out, want)


@pytest.mark.parametrize("T,Hq,Hkv", [(3, 8, 2), (48, 8, 2)])
def test_one_node_is_paged_attention(T, Hq, Hkv):
    """The first node of a chain against the single-token operator; and a cache whose
    pages lie more than 2^31 bytes apart."""
    q, k, v, pt, lens, nodes = tree(15, "f16", [500, 1, 90], [T] * 3, T, Hq, Hkv, 64, 16, poison=False)
    a, la = tq.tq_tree_attention(q, k, v, pt, lens, return_lse=True)
    b, lb = tq.tq_paged_attention(q[:, 0], k, v, pt, lens + 1, return_lse=True)
    assert (a[:, 0].float() - b.float()).abs().max() < 2.0 ** -8
    assert (la[:, 0] - lb).abs().max() < 2.0 ** -16


def test_a_cache_of_more_than_4_gib():
    T, P = 9, 3
    page = (1 << 31) // 2 + 8 * 16  # elements: pages 2 GiB apart
    pool = torch.empty(P * page, dtype=torch.float16, device="cuda")
    shape, strides = (P, 16, 1, 64), (page, 64, 64, 1)
    k = torch.as_strided(pool, shape, strides)
    v = torch.as_strided(pool, shape, strides, 16 * 64)
    g = torch.Generator().manual_seed(0)
    k.copy_(torch.randn(shape, generator=g).half())
    v.copy_(torch.randn(shape, generator=g).half())
    q = randn(1, "f16", 1, T, 8, 64)
    pt, lens, nodes = i32([[2, 0, 1]]), i32([30]), i32([T])
    sees = tree_paths_ref(parents_of(1, 1, T))
    run(q, k, v, pt, lens, nodes, sees, "f16")


@pytest.mark.parametrize("T,Hq,Hkv,lens", [(24, 8, 1, [300, 0, 4000]), (3, 8, 8, [5000, 17, 2])])
def test_captured(T, Hq, Hkv, lens):
    """Captured with its mask, replayed with other contents and lengths, on a side stream."""
    q, k, v, pt, lens, nodes = tree(16, "bf16", lens, [T] * len(lens), T, Hq, Hkv, 128, 16, poison=False)
    p = torch.from_numpy(parents_of(9, len(lens), T)).cuda()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        for _ in range(2):
            tq.tq_tree_attention(q, k, v, pt, lens, mask=tq.tq_tree_mask(p)[0], nodes=nodes)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            mask, depth = tq.tq_tree_mask(p)
            out, lse = tq.tq_tree_attention(q, k, v, pt, lens, mask=mask, nodes=nodes, return_lse=True)
    full = lens.clone()
    for i in range(4):
        torch.cuda.synchronize()
        q.copy_(randn(20 + i, "bf16", *q.shape))
        lens.copy_((full.float() * (1 - 0.3 * i)).int().clamp(min=0))
        nodes.fill_(max(1, T - i))
        p.copy_(torch.from_numpy(parents_of(30 + i, len(lens), T)))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = tq.tq_tree_attention(q, k, v, pt, lens, mask=tq.tq_tree_mask(p)[0], nodes=nodes, return_lse=True)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]), i


def test_streams_and_empty_calls():
    T = 6
    q, k, v, pt, lens, nodes = tree(17, "f16", [400, 30], [T, T], T, 8, 2, 64, 16, poison=False)
    p = torch.from_numpy(parents_of(2, 2, T)).cuda()
    want = tq.tq_tree_attention(q, k, v, pt, lens, mask=tq.tq_tree_mask(p)[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    mask, _ = tq.tq_tree_mask(p, stream=side.cuda_stream)
    out = tq.tq_tree_attention(q, k, v, pt, lens, mask=mask, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(out, want)
    assert tq.tq_tree_attention(q[:0], k, v, pt[:0], lens[:0]).shape == (0, T, 8, 64)
    assert tq.tq_tree_attention(q[:, :0], k, v, pt, lens).shape == (2, 0, 8, 64)
    assert tq.tq_tree_mask(p[:0])[0].shape == (0, T, 1) and tq.tq_tree_mask(p[:, :0])[0].shape == (2, 0, 0)
