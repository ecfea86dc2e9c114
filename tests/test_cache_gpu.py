"""GPU parity of the operators on caches that are kept short against the fp64 oracle.

Weights: with ds = (D + 4) 2^-24 smag for a score (as in test_decode_gpu.py) and the
exponent's own rounding, 2^-22 (smag + |lse|) at most (the sum in base 2, the scaled
lse), a term is off by a factor e^(ds + ..); fp32 sums of R terms and the hardware's
exponential add (R + 8) 2^-23.  All relative to the weight; the running sum is multiplied,
added and rounded once: 2^-23 of each.  Choices and moves are exact.
"""

import numpy as np
import pytest

from oracle import (cache_select_ref, cache_weights_ref, pages_keep_ref, tree_attention_ref,
                    tree_paths_ref)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
tq = pytest.importorskip("bit_mixed_precision_amd.binding")

from test_decode_gpu import DT, NAN, f64, i32, randn  # noqa: E402
from test_tree_gpu import parents_of, tree, words  # noqa: E402


# ------------------------------------------------------------------ weights

def check_weights(q, k, v, pt, lens, nodes, sees, S, decay=1.0, window=0, scale=None, chain=False, lse=None):
    B, T, Hq, D = q.shape
    Hkv = k.shape[2]
    scale = D ** -0.5 if scale is None else scale
    m = np.clip(nodes.cpu().numpy(), 0, T)
    a = (f64(q), f64(k))
    if lse is None:
        lse = torch.from_numpy(tree_attention_ref(*a, np.nan_to_num(f64(v)), pt.cpu().numpy(), lens.cpu().numpy(), m, sees,
                                                  scale, window)[1]).float().cuda()
    room = torch.rand(B, Hkv + 1, S + 5, generator=torch.Generator().manual_seed(3)).cuda() * 4
    scores = room[:, :Hkv, 2:2 + S]
    before = room.clone()
    want, add, smag = cache_weights_ref(*a, pt.cpu().numpy(), lens.cpu().numpy(), m, sees,
                                        f64(lse), f64(scores), decay, scale, window)
    got = tq.tq_cache_weights(q, k, pt, lens, lse, scores, mask=None if chain else words(sees), nodes=nodes,
                              scale=scale, window=window, decay=decay)
    assert got is scores
    fin = np.where(np.isfinite(f64(lse)), np.abs(f64(lse)), 0).max()
    ds = ((D + 4) * 2.0 ** -24 * smag + 2.0 ** -22 * (smag + fin))[:, None, None]
    bound = add * (np.expm1(ds) + (T * Hq // Hkv + 8) * 2.0 ** -23) + 2.0 ** -22 * np.abs(want)
    err = np.abs(f64(scores) - want)
    assert np.all(err <= bound), float((err / np.maximum(bound, 1e-300)).max())
    # what lies around the sums, and past the last token
    mine = torch.zeros_like(room, dtype=torch.bool)
    cap = min(S, pt.shape[1] * k.shape[1])
    for b in range(B):
        n = min(max(int(lens[b]), 0), pt.shape[1] * k.shape[1])
        mine[b, :Hkv, 2:2 + min(n + int(m[b]), cap)] = True
    assert torch.equal(room[~mine], before[~mine])
    return scores


EDGE = [0, 1, 31, 32, 33, 127, 128, 129, 300]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,Hq,Hkv,D,size", [
    (1, 8, 1, 128, 16), (1, 3, 3, 64, 24), (5, 16, 2, 80, 16), (17, 8, 4, 128, 32), (70, 4, 2, 64, 16),
    (3, 34, 2, 256, 16), (2, 5, 5, 8, 1), (9, 6, 2, 192, 5)])
@pytest.mark.parametrize("decay", [1.0, 0.75])
def test_weights(dtype, T, Hq, Hkv, D, size, decay):
    B = len(EDGE)
    nodes = np.random.default_rng(T).integers(0, T + 1, B)
    nodes[:2] = T
    args = tree(T + D, dtype, EDGE, nodes, T, Hq, Hkv, D, size)
    check_weights(*args, tree_paths_ref(parents_of(D, B, T)), 340, decay)


@pytest.mark.parametrize("T,Hq,Hkv,D,lens,S", [
    (1, 64, 8, 128, [9000, 1, 700, 0, 12345], 13000), (16, 8, 2, 128, [5000, 8000], 8100),
    (1, 1, 1, 64, [30] * 700, 64), (200, 4, 1, 128, [900], 800), (4, 8, 8, 256, [3000], 2000)])
def test_weights_long(T, Hq, Hkv, D, lens, S):
    """Runs of tiles that cross heads and sequences; sums shorter than the cache."""
    B = len(lens)
    args = tree(T, "bf16", lens, [T] * B, T, Hq, Hkv, D, 16, poison=False)
    chain = np.tril(np.ones((1, T, T), bool)).repeat(B, 0)
    check_weights(*args, chain, S, 0.5, chain=True)


@pytest.mark.parametrize("window", [6, 40, 150, 1 << 40])
@pytest.mark.parametrize("decay", [1.0, 0.5])
def test_weights_window(window, decay):
    lens, T = [0, 3, 64, 129, 300], 6
    args = tree(1, "f16", lens, [6, 6, 2, 6, 0], T, 4, 2, 64, 16)
    check_weights(*args, tree_paths_ref(parents_of(3, 5, T)), 320, decay, window)


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_weights_scale(scale):
    args = tree(2, "bf16", [90, 200], [3, 3], 3, 4, 2, 64, 16)
    check_weights(*args, tree_paths_ref(parents_of(3, 2, 3)), 210, scale=scale)


def test_weights_rows_left_out():
    """Rows with an infinite or undefined lse add nothing, whatever they hold; bits that
    are no tree; absent pages."""
    T = 5
    q, k, v, pt, lens, nodes = tree(4, "f16", [100, 40], [T, 4], T, 4, 2, 64, 16)
    sees = np.random.default_rng(0).random((2, T, T)) < 0.5
    pt[0, 2] = -1
    lse = randn(8, "f16", 2, T, 4).float() + 5
    lse[0, 1], lse[0, 3, 2], lse[1, 0, 1] = -float("inf"), NAN, float("inf")
    q[0, 1], q[1, 4] = NAN, NAN  # the second is no node
    qq = q.clone()
    qq[0, 1], qq[1, 4] = 0, 0
    got = check_weights(qq, k, v, pt, lens, nodes, sees, 120, lse=lse)
    room = torch.rand(2, 3, 125, generator=torch.Generator().manual_seed(3)).cuda() * 4
    again = tq.tq_cache_weights(q, k, pt, lens, lse, room[:, :2, 2:122], mask=words(sees), nodes=nodes)
    assert torch.equal(got, again)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,Hq", [(1, 2), (3, 14), (9, 4)])
def test_weights_of_infinite_keys(dtype, T, Hq):
    """A score of -inf is a weight of zero for every row, also where the rows do not fill a
    tile of the matrix instruction."""
    q, k, v, pt, lens, nodes = tree(9, dtype, [300, 40], [T, T], T, Hq, 2, 64, 16)
    q[..., 0] = -q[..., 0].abs() - 1
    chain = np.tril(np.ones((2, T, T), bool))
    hit = [(0, 70), (0, 130), (1, 3)]
    for b, t in hit:
        k[pt[b, t // 16].long(), t % 16, :, 0] = float("inf")
    out, lse = tq.tq_tree_attention(q, k, v, pt, lens, nodes=nodes, return_lse=True)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    scores = torch.zeros(2, 2, 330, device="cuda")
    tq.tq_cache_weights(q, k, pt, lens, lse, scores, nodes=nodes)
    for b, t in hit:  # the same without these tokens, whose keys are then finite
        k[pt[b, t // 16].long(), t % 16, :, 0] = 0
        assert torch.equal(scores[b, :, t], torch.zeros(2, device="cuda"))
    want = torch.zeros_like(scores)
    tq.tq_cache_weights(q, k, pt, lens, lse, want, nodes=nodes)
    for b, t in hit:
        want[b, :, t] = 0
    assert torch.equal(scores, want)


def test_weights_add_up_and_repeat():
    """One token's weights over a whole cache add up to the heads of a group."""
    q, k, v, pt, lens, nodes = tree(5, "bf16", [4000, 77], [1, 1], 1, 16, 4, 128, 16)
    out, lse = tq.tq_tree_attention(q, k, v, pt, lens, return_lse=True)
    first = torch.zeros(2, 4, 4096, device="cuda")
    tq.tq_cache_weights(q, k, pt, lens, lse, first)
    assert (first.double().sum(-1) - 4).abs().max() < 1e-3
    for _ in range(3):
        again = torch.zeros_like(first)
        tq.tq_cache_weights(q, k, pt, lens, lse, again)
        assert torch.equal(first, again)


# ------------------------------------------------------------------ the choice

def check_select(scores, lens, budget, recent, sinks):
    keep, counts, sums = tq.tq_cache_select(scores, i32(lens), budget, recent, sinks)
    want = cache_select_ref(scores.cpu().numpy(), lens, budget, recent, sinks)
    assert np.array_equal(counts.cpu().numpy(), want[1])
    assert np.array_equal(keep.cpu().numpy(), want[0])
    assert np.array_equal(sums.cpu().numpy(), want[2], equal_nan=True)


@pytest.mark.parametrize("budget,recent,sinks", [(1, 0, 0), (1, 1, 0), (7, 2, 1), (64, 16, 4), (64, 60, 4),
                                                 (200, 0, 0), (300, 100, 0), (1000, 10, 10)])
def test_select(budget, recent, sinks):
    lens = [0, 1, 7, 8, 63, 64, 65, 200, 299, 300, 1023, 1024, 1025]
    g = torch.Generator().manual_seed(budget)
    x = torch.exp(3 * torch.randn(len(lens), 3, 1030, generator=g))
    x = torch.where(torch.rand(x.shape, generator=g) < 0.3, (x * 2).round() / 2, x).cuda()
    check_select(x, lens, budget, recent, sinks)


@pytest.mark.parametrize("n,budget", [(5000, 512), (40000, 20000), (70001, 64), (131072, 131071)])
def test_select_long(n, budget):
    g = torch.Generator().manual_seed(n)
    x = torch.exp(2 * torch.randn(2, 2, n, generator=g))
    x = torch.where(torch.rand(x.shape, generator=g) < 0.2, (x * 2).round() / 2, x).cuda()
    check_select(x, [n, n // 3], budget, budget // 8, 4)


def test_select_equal_and_odd_numbers():
    """All equal, zeros of both signs, negative numbers, infinities, NaN; the first ones of
    equal weight stay."""
    inf = float("inf")
    rows = [[1.0] * 40, [0.0, -0.0] * 20, [-1.0, -2.0, -1.0, 5e-324, -5e-324] * 8,
            [inf, 1.0, -inf, NAN] * 10, [NAN] * 40, [-inf, NAN] * 20, [1e-45, 0, 1e-38, -1e-45] * 10]
    x = torch.tensor(rows, dtype=torch.float32).view(len(rows), 1, 40).cuda()
    for budget, recent, sinks in ((1, 0, 0), (13, 0, 0), (13, 3, 2), (20, 0, 1), (39, 0, 0)):
        check_select(x, [40] * len(rows), budget, recent, sinks)


def test_select_strides_lengths_and_empty_calls():
    room = torch.rand(4, 6, 300, generator=torch.Generator().manual_seed(1)).cuda()
    x = room[:, 1:5:2, 3:253]
    check_select(x, [-5, 10 ** 6, 250, 100], 50, 5, 1)
    check_select(room.transpose(0, 1)[:2], [300, 200, 100, 1][:2], 50, 5, 1)
    check_select(room[:1, :1].expand(3, 2, -1), [300, 20, 77], 30, 0, 0)
    keep, counts, sums = tq.tq_cache_select(room, i32([5, 6, 7, 8]), 0)
    assert keep.shape == (4, 6, 0) and counts.tolist() == [0] * 4
    assert tq.tq_cache_select(room[:0], i32([]), 9)[0].shape == (0, 6, 9)
    keep, counts, sums = tq.tq_cache_select(room[:, :, :0], i32([5, 6, 7, 8]), 3)
    assert torch.all(keep == -1) and counts.tolist() == [0] * 4 and not sums.any()


# ------------------------------------------------------------------ the move

def pool_of(seed, planes, pages, size, H, D, dtype=torch.float16):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(planes, pages, size, H, D, generator=g).to(dtype).cuda()


def check_keep(pool, pt, lens, keep, counts, base, size):
    planes, P = pool.shape[:2]
    k4 = keep if keep.dim() == 4 else keep[None] if keep.dim() == 3 else keep[None, :, None]
    groups, rows, heads, n = k4.shape
    want = pool.clone().view(planes, P, size, heads, -1)
    old = want.clone()
    table, out, short, moves = pages_keep_ref(pt.cpu().numpy(), lens.cpu().numpy(), k4.cpu().numpy(),
                                              counts.cpu().numpy(), None if base is None else base.cpu().numpy(), P, size)
    each = planes // groups
    for g, h, sp, ss, dp, ds in moves:
        want[g * each:(g + 1) * each, dp, ds, h] = old[g * each:(g + 1) * each, sp, ss, h]
    got = tq.tq_pages_keep(pool, pt, lens, keep, counts, size, base=base)
    assert np.array_equal(got[0].cpu().numpy(), table)
    assert np.array_equal(got[1].cpu().numpy(), out)
    assert got[2].tolist() == [short]
    assert torch.equal(pool, want.view(pool.shape))
    return got


def dealt(seed, lens, size, extra, width=None):
    """A table that holds these lengths in shuffled pages, `extra` pages free."""
    rng = np.random.default_rng(seed)
    need = -(-np.asarray(lens) // size)
    width = width or max(1, int(need.max()))
    P = int(need.sum()) + extra
    pt = np.full((len(lens), width), -1, np.int32)
    pt[np.arange(width)[None] < need[:, None]] = rng.permutation(P)[:need.sum()]
    return i32(pt), i32(lens), P


def some(rng, groups, rows, heads, lens, base, counts, n):
    keep = np.full((groups, rows, heads, n), -1, np.int32)
    for g in range(groups):
        for r in range(rows):
            for h in range(heads):
                keep[g, r, h, :counts[r]] = base[r] + np.sort(rng.permutation(lens[r] - base[r])[:counts[r]])
    return i32(keep)


@pytest.mark.parametrize("size", [1, 5, 16, 64])
@pytest.mark.parametrize("groups,planes,heads,H,D", [(1, 2, 1, 3, 16), (2, 4, 4, 4, 64), (1, 1, 2, 4, 40),
                                                     (3, 3, 8, 8, 128), (1, 3, 1, 8, 72)])
def test_keep(size, groups, planes, heads, H, D):
    lens = [0, 1, 16, 17, 100, 333, 700]
    rng = np.random.default_rng(size)
    base = [0, 0, 3, 17, 40, 1, 128]
    counts = [0, 1, 5, 0, 60, 200, 570]
    pt, ln, P = dealt(size, lens, size, 2)
    pool = pool_of(1, planes, P, size, H, D)
    keep = some(rng, groups, len(lens), heads, lens, base, counts, 600)
    check_keep(pool, pt, ln, keep, i32(counts), i32(base), size)
    if groups == 1:
        check_keep(pool, pt, ln, keep[0].contiguous(), i32(counts), i32(base), size)
        if heads == 1:
            check_keep(pool, pt, ln, keep[0, :, 0].contiguous(), i32(counts), i32(base), size)
    counts = [min(c, n) for c, n in zip([0, 1, 9, 10, 64, 100, 512], lens)]
    keep = some(rng, groups, len(lens), heads, lens, [0] * 7, counts, 512)
    check_keep(pool, pt, ln, keep, i32(counts), None, size)


@pytest.mark.parametrize("free", [0, 1, 3, 5, 20])
def test_keep_shared_pages(free):
    """Pages that several rows hold: replaced where they would change, kept where they do
    not, and rows that find too few free pages stay as they are."""
    size, lens = 8, [40, 50, 23, 64, 40, 9]
    pt, ln, P = dealt(3, lens, size, free, width=9)
    pt[1, :3], pt[3, :2], pt[4, :5], pt[5, 0] = pt[0, :3], pt[2, :2], pt[0, :5], pt[2, 0]
    rng = np.random.default_rng(0)
    base, counts = [0, 8, 4, 0, 40, 0], [20, 30, 10, 64, 0, 4]
    pool = pool_of(2, 2, P, size, 2, 32)
    keep = some(rng, 1, 6, 2, lens, base, counts, 64)
    keep[0, 5] = torch.arange(64, device="cuda")  # keeps its first tokens where they are
    check_keep(pool, pt, ln, keep, i32(counts), i32(base), size)


@pytest.mark.parametrize("rows,width,pages", [(300, 3, 900), (40, 1300, 52000), (3, 40, 70000)])
def test_keep_large_states(rows, width, pages):
    size = 2
    rng = np.random.default_rng(rows)
    lens = rng.integers(0, width * size // 2, rows)
    pt, ln, P = dealt(4, lens, size, 0, width)
    extra = max(0, pages - P)
    pool = pool_of(3, 1, P + extra, size, 1, 8)
    pt[1::2, :1] = pt[0::2, :1][:rows // 2]  # first pages shared where they are held
    counts = np.minimum(lens, 40)
    keep = some(rng, 1, rows, 1, lens, np.zeros(rows, int), counts, 40)
    check_keep(pool, pt, ln, keep, i32(counts), None, size)


def test_keep_odd_arguments():
    """Lengths, bases and counts out of range, entries that name no page, lists that do
    not ascend or leave the row: nothing outside the row's slots changes."""
    size = 4
    pt, ln, P = dealt(5, [30, 20, 17, 12, 8], size, 4, width=8)
    pt[0, 2], pt[1, 0], pt[2, 4] = -7, 10 ** 6, -1
    ln[3], ln[4] = -3, 10 ** 9
    base, counts = i32([-5, 100, 3, 0, 2]), i32([10, 3, 99, 5, -2])
    keep = np.tile(np.arange(12) * 2, (5, 2, 1)).astype(np.int32)
    keep[0, 0] = [0, 9, 3, 3, 5, 100, -1, 7, 2 ** 31 - 1, 9, 10, 11]
    keep[2, 1, :4] = [5, 5, 5, 6]
    pool = pool_of(4, 2, P, size, 2, 16)
    before = pool.clone()
    table, lens, short = tq.tq_pages_keep(pool, pt, ln, i32(keep), counts, size, base=base)
    want = pages_keep_ref(pt.cpu().numpy(), ln.cpu().numpy(), keep[None], counts.cpu().numpy(),
                          base.cpu().numpy(), P, size)
    assert np.array_equal(table.cpu().numpy(), want[0]) and np.array_equal(lens.cpu().numpy(), want[1])
    touched = {(d, s) for _, _, _, _, d, s in want[3]}
    same = torch.ones(P, size, dtype=torch.bool)
    for d, s in touched:
        same[d, s] = False
    assert torch.equal(pool[:, same.cuda()], before[:, same.cuda()])


def test_keep_entries_that_name_no_token_of_a_shared_page():
    """A slot whose list entry names no token keeps its token, also where the row gets another
    page for it."""
    size = 8
    pt, ln, P = dealt(9, [20, 20], size, 3, width=4)
    pt[1, :2] = pt[0, :2]
    keep = np.array([[-1, 3, 2 ** 31 - 1, 9, 2, 11, 12, 13, 14, -5], list(range(10))], np.int32)
    pool = pool_of(8, 2, P, size, 2, 16)
    table, lens, short = check_keep(pool, pt, ln, i32(keep), i32([10, 10]), None, size)
    assert short.tolist() == [0] and table[1].tolist() == pt[1, :2].tolist() + [-1, -1]
    mine, old = pool[:, table[0, 0].long()], pool[:, pt[0, 0].long()]
    assert torch.equal(mine[:, [0, 1, 2, 4]], old[:, [0, 3, 2, 4]])


def test_keep_no_rows_of_many_pages():
    pool = torch.zeros(1, 70000, 1, 8, dtype=torch.float16, device="cuda")
    none = torch.zeros(0, 4, dtype=torch.int32, device="cuda")
    table, lens, short = tq.tq_pages_keep(pool, none, none[:, 0].contiguous(), none, none[:, 0].contiguous(), 1)
    assert table.shape == (0, 4) and short.tolist() == [0]


def test_keep_empty_calls():
    pt, ln, P = dealt(6, [30, 20], 4, 1)
    pool = pool_of(5, 2, P, 4, 2, 16)
    before = pool.clone()
    none = torch.zeros(2, 0, dtype=torch.int32, device="cuda")
    table, lens, short = tq.tq_pages_keep(pool, pt, ln, none, i32([9, 9]), 4, base=i32([12, 20]))
    assert lens.tolist() == [12, 20] and table[0].tolist() == pt[0, :3].tolist() + [-1] * 5
    assert torch.equal(pool, before)
    table, lens, short = tq.tq_pages_keep(pool, pt[:0], ln[:0], none[:0], ln[:0], 4)
    assert table.shape == (0, 8) and short.tolist() == [0]


def test_keep_in_place_over_a_long_row():
    """A row of many parts, moved forward by one token: every part reads what the part
    after it overwrites."""
    n, size = 20000, 16
    pt, ln, P = dealt(7, [n], size, 0)
    pool = pool_of(6, 2, P, size, 2, 64)
    keep = torch.arange(1, n, device="cuda", dtype=torch.int32).view(1, 1, n - 1).repeat(1, 2, 1)
    for gap in (1, 2, 63, 64, 65, 1000):
        keep = torch.arange(gap, n, device="cuda", dtype=torch.int32).view(1, 1, -1).repeat(1, 2, 1).contiguous()
        want = pool.clone()
        flat = want[:, pt[0].long()].reshape(2, -1, 2, 64)
        flat[:, :n - gap] = flat[:, gap:n].clone()
        want[:, pt[0].long()] = flat.view(2, -1, size, 2, 64)
        tq.tq_pages_keep(pool, pt, ln, keep, i32([n - gap]), size)
        assert torch.equal(pool, want), gap


def test_append_at_slots():
    """Slots apart from positions; slots out of range are not written."""
    D, Hq, Hkv = 64, 4, 2
    table = torch.from_numpy(tq.tq_rope_table(100, D)).cuda()
    qkv = randn(1, "f16", 6, Hq + 2 * Hkv, D)
    pt = i32([[3, 1], [0, 2]])
    k, v = (torch.zeros(4, 8, Hkv, D, dtype=torch.float16, device="cuda") for _ in range(2))
    pos, seqs = i32([40, 40, 41, 99, 100, 7]), i32([0, 0, 1, 1, 1, 0])
    slots = i32([2, 9, 15, 16, 3, -1])
    q = tq.tq_rope_append(qkv, table, pos, pt, k, v, seqs=seqs, slots=slots)
    turned = tq.tq_rope(qkv[:, :Hq + Hkv], table, pos)
    assert torch.equal(q, turned[:, :Hq])
    want_k, want_v = torch.zeros_like(k), torch.zeros_like(v)
    for t, page, slot in ((0, 3, 2), (1, 1, 1), (2, 2, 7)):
        want_k[page, slot], want_v[page, slot] = turned[t, Hq:], qkv[t, Hq + Hkv:]
    assert torch.equal(k, want_k) and torch.equal(v, want_v)
    k2, v2 = torch.zeros_like(k), torch.zeros_like(v)
    q2 = tq.tq_rope_append(qkv, table, pos, pt, k2, v2, seqs=seqs, slots=slots,
                           stream=torch.cuda.current_stream().cuda_stream)
    assert torch.equal(q, q2) and torch.equal(k, k2) and torch.equal(v, v2)
    # slots that are the positions
    low = pos.clamp(max=15)
    for x in (k, v, k2, v2):
        x.zero_()
    assert torch.equal(tq.tq_rope_append(qkv, table, low, pt, k, v, seqs=i32([0, 1, 0, 1, 0, 1]), slots=low),
                       tq.tq_rope_append(qkv, table, low, pt, k2, v2, seqs=i32([0, 1, 0, 1, 0, 1])))


# ------------------------------------------------------------------ together

def test_captured_steps():
    """Weights, choice and move captured as one step, replayed over changing contents."""
    B, Hq, Hkv, D, size = 3, 8, 2, 64, 16
    lens0 = [150, 90, 200]
    pt, lens, P = dealt(8, lens0, size, 6, width=14)
    pool = pool_of(7, 2, P, size, Hkv, D)
    q = randn(2, "f16", B, 1, Hq, D)
    scores = torch.rand(B, Hkv, 14 * size, device="cuda")

    def step():
        before = lens - 1
        _, lse = tq.tq_tree_attention(q, pool[0], pool[1], pt, before, return_lse=True)
        tq.tq_cache_weights(q, pool[0], pt, before, lse, scores, decay=0.5)
        keep, counts, sums = tq.tq_cache_select(scores, lens, 64, 8, 2)
        table, left, short = tq.tq_pages_keep(pool, pt, lens, keep, counts, size)
        return lse, keep, sums, table, left, short

    start = [x.clone() for x in (pool, scores)]
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            got = step()
    for i in range(3):
        torch.cuda.synchronize()
        q.copy_(randn(10 + i, "f16", *q.shape))
        lens.copy_(i32([n - 20 * i for n in lens0]))
        results = []
        for run in (step, graph.replay):
            pool.copy_(start[0]), scores.copy_(start[1])
            torch.cuda.synchronize()
            r = run()
            torch.cuda.synchronize()
            results.append([x.clone() for x in (r or got)] + [pool.clone(), scores.clone()])
        for x, y in zip(*results):
            assert torch.equal(x, y), i


def test_other_streams():
    """Calls on a stream of their own, handed over or current, give what the first stream does."""
    q, k, v, pt, lens, nodes = tree(6, "f16", [500, 90], [3, 2], 3, 8, 2, 64, 16, poison=False)
    _, lse = tq.tq_tree_attention(q, k, v, pt, lens, nodes=nodes, return_lse=True)
    pool = torch.stack([k, v])

    def run(**kw):
        s, p = torch.zeros(2, 2, 520, device="cuda"), pool.clone()
        torch.cuda.synchronize()
        tq.tq_cache_weights(q, k, pt, lens, lse, s, nodes=nodes, **kw)
        keep, counts, sums = tq.tq_cache_select(s, lens, 64, 8, 2, **kw)
        got = tq.tq_pages_keep(p, pt, lens, keep, counts, 16, **kw)
        torch.cuda.synchronize()
        return [s, p, keep, counts, sums, *got]

    want = run()
    stream = torch.cuda.Stream()
    given = run(stream=stream.cuda_stream)
    with torch.cuda.stream(stream):
        current = run()
    for x, y, z in zip(want, given, current):
        assert torch.equal(x, y) and torch.equal(x, z)
