"""More decode-side operators of this library as measurable cases: several new
tokens per sequence, and caches that are kept short.

* the ancestors of the nodes of drafted trees, as bits (``mask``);
* attention of the nodes of a drafted tree over the paged cache (``tree``);
* the attention weight that each cached token receives, added to a running sum
  (``weights``);
* the choice of the tokens that a cache keeps by those sums (``select``);
* moving kept tokens together in the pages: the accepted path of a tree, or what an
  eviction leaves (``keep``).

``own`` chooses between the plain torch form (False) and the library (True).
Sizes: 64 query / 8 key-value heads of 128 are the library's 70B-shaped decode
stack; the others are generic.
"""

import math

import numpy as np
import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- the cases

def listed():
    stack = dict(Hq=64, Hkv=8, D=128, page=16)
    return [
        # one user's drafted tree
        dict(name="mask_1x24", op="mask", B=1, T=24, deep=2),
        # large trees of a full batch
        dict(name="mask_96x255", op="mask", B=96, T=255, deep=8),
        # verifying a small tree in a short chat: latency
        dict(name="tree_1x24", op="tree", dtype="f16", B=1, T=24, lo=97, hi=97, ragged=False, deep=2,
             empty=0, window=0, **stack),
        # heads that share nothing, trees of 1 to 13 nodes, short and ragged sequences, two unused slots
        dict(name="tree_37_ragged", op="tree", dtype="bf16", B=37, T=13, lo=1, hi=4096, ragged=True, deep=2,
             empty=2, window=0, Hq=24, Hkv=24, D=64, page=32),
        # one very long document and a large tree
        dict(name="tree_1x131072", op="tree", dtype="f16", B=1, T=64, lo=131072, hi=131072, ragged=False, deep=4,
             empty=0, window=0, **stack),
        # a serving batch of long chats, drafted chains and trees of 32
        dict(name="tree_24_long", op="tree", dtype="bf16", B=24, T=32, lo=2048, hi=8192, ragged=True, deep=3,
             empty=0, window=0, **stack),
        # one decoded token of one user
        dict(name="weights_1x2000", op="weights", dtype="f16", B=1, T=1, lo=2000, hi=2000, ragged=False, deep=1,
             empty=0, window=0, decay=1.0, **stack),
        # the last 16 tokens of prompts decide what is kept of them
        dict(name="weights_16_prompt", op="weights", dtype="bf16", B=16, T=16, lo=4096, hi=16384, ragged=False,
             deep=0, empty=0, window=0, decay=1.0, **stack),
        # one user's cache of one layer
        dict(name="select_1x1009", op="select", B=1, H=8, lo=1009, hi=1009, budget=512, recent=64, sinks=4),
        # a layer of a serving batch, short and long
        dict(name="select_48_long", op="select", B=48, H=8, lo=1024, hi=32768, budget=1024, recent=128, sinks=4),
        # accepted paths of eight trees, sixteen layers, all heads alike
        dict(name="keep_path_8", op="keep", kind="path", dtype="f16", B=8, T=24, lo=100, hi=1500, budget=0,
             groups=1, planes=32, shared=0, Hkv=8, D=128, page=16),
        # eviction to half, each head of eight layers its own tokens; prompts of two pages shared by pairs
        dict(name="keep_evict_16", op="keep", kind="evict", dtype="bf16", B=16, T=0, lo=1100, hi=2048, budget=1024,
             groups=8, planes=16, shared=2, Hkv=8, D=128, page=16),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "weights", "weights", "select", "keep", "keep", "mask"])
    if op == "mask":
        return dict(op=op, B=_log(rng, 1, 96), T=_log(rng, 1, 256), deep=rng.choice([0, 1, 2, 4, 8]))
    if op == "select":
        H = rng.choice([1, 2, 8, 8, 24])
        B = _log(rng, 1, 384 // H)
        hi = _log(rng, 1, min(131072, 48 * 8 * 9000 // (B * H)))
        budget = _log(rng, 1, max(1, hi))
        recent = rng.choice([0, budget // 8, rng.randint(0, budget)])
        return dict(op=op, B=B, H=H, lo=_log(rng, 1, hi), hi=hi, budget=budget, recent=recent,
                    sinks=rng.randint(0, min(4, budget - recent)))
    D = rng.choice([64, 80, 96, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8, 8, 12])
    page = rng.choice([16, 16, 32, 64, 128, 24])
    dtype = rng.choice(["f16", "bf16"])
    if op == "keep":
        kind = rng.choice(["path", "evict"])
        T = _log(rng, 1, 64) if kind == "path" else 0
        hi = _log(rng, 2, 4096)
        B = _log(rng, 1, 32)
        pages = B * (-(-(hi + T) // page) + 2)
        most = 16 * 16 * 2048 * 8 * 128 // (pages * page * Hkv * D)
        if most < 1:
            B, pages, most = 1, -(-(hi + T) // page) + 2, 4
        groups = 1 if kind == "path" else rng.choice([1, 2, 4])
        planes = 2 * groups * max(1, _log(rng, 1, max(1, min(32, most // (2 * groups)))))
        return dict(op=op, kind=kind, dtype=dtype, B=B, T=T, lo=_log(rng, 1, hi), hi=hi, budget=_log(rng, 1, hi),
                    groups=groups, planes=planes, shared=rng.choice([0, 0, 1, 3]), Hkv=Hkv, D=D, page=page)
    group = rng.choice([1, 2, 3, 4, 8, 8, 16])
    Hq = Hkv * group
    T = rng.choice([1, _log(rng, 1, 16), _log(rng, 2, 64), _log(rng, 2, 256)])
    B = _log(rng, 1, 64)
    # of all sequences together: the keys read, the products, and the scores that the plain form holds
    room = min(24 * 8192 * 8 * 128 // (Hkv * D), 64 * 131072 * 64 * 128 // (T * Hq * D), 64 * 131072 * 64 // (T * Hq))
    B = max(1, min(B, room // (T + 1)))
    hi = _log(rng, 1, max(1, min(131072, room // B)))
    c = dict(op=op, dtype=dtype, B=B, T=T, lo=_log(rng, 1, hi), hi=hi, ragged=rng.random() < 0.5,
             deep=rng.choice([0, 1, 2, 4]), empty=rng.choice([0, 0, 1]) if B > 1 else 0,
             window=rng.choice([0, 0, 0, T + _log(rng, 1, hi)]), Hq=Hq, Hkv=Hkv, D=D, page=page)
    if op == "weights":
        c["decay"] = rng.choice([1.0, 0.97])
    return c


def _lens(c):
    """The lengths of a batch, in rising order: even over the logarithm."""
    n = c["B"] - c.get("empty", 0)
    q = np.arange(n) / max(1, n - 1) if n > 1 else np.ones(1)
    x = np.rint(np.exp(math.log(c["lo"]) + q * (math.log(c["hi"]) - math.log(c["lo"]))))
    return np.concatenate([np.zeros(c.get("empty", 0)), x]).astype(np.int64)


def work(c):
    if c["op"] == "mask":
        words = -(-c["T"] // 64)
        return {"bytes": c["B"] * c["T"] * (4 + 8 * words + 4), "flops": 0}
    n = _lens(c)
    if c["op"] == "select":
        kept = np.minimum(n, c["budget"]).sum()
        return {"bytes": int(4 * c["H"] * (n.sum() + 2 * kept)), "flops": 0}
    row = 2 * c["Hkv"] * c["D"]
    if c["op"] == "keep":
        # a few tokens of each path, about what the eviction keeps behind the first hole
        moved = 3 * c["B"] if c["kind"] == "path" else int(np.where(n > c["budget"], c["budget"], 0).sum())
        return {"bytes": 2 * moved * row * c["planes"] + 4 * moved * (1 if c["kind"] == "path" else c["Hkv"] * c["groups"])
                + 8 * int((n // c["page"] + 1).sum()), "flops": 0}
    seen = np.minimum(n, c["window"]) if c["window"] else n
    tokens = int(seen.sum()) + (c["B"] - c["empty"]) * c["T"]
    q = 2 * c["B"] * c["T"] * c["Hq"] * c["D"]
    flops = 2 * tokens * c["T"] * c["Hq"] * c["D"]
    if c["op"] == "weights":
        return {"bytes": tokens * row + q + 8 * tokens * c["Hkv"] + 4 * c["B"] * c["T"] * c["Hq"], "flops": flops}
    return {"bytes": 2 * tokens * row + 2 * q + 4 * c["B"] * c["T"] * c["Hq"], "flops": 2 * flops}


# ---------------------------------------------------------------- the inputs

def _normal(gen, dtype, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float16).to(_DT[dtype])


def _parents(c, rng):
    """Drafted trees [B][T]: node i hangs on one of the nodes before it, mostly on a
    recent one; deep = 0 is a chain, the larger it is the more nodes branch off."""
    i = np.arange(c["T"])
    back = 1 + np.floor(rng.exponential(max(c["deep"], 1e-9), (c["B"], c["T"]))).astype(np.int64)
    return np.maximum(i - back, -1).astype(np.int32)


def _bits(parents):
    """The mask of trees as int64 words [B][T][ceil(T / 64)] (host, node by node)."""
    B, T = parents.shape
    words = -(-T // 64)
    mask = np.zeros((B, T, words), np.uint64)
    for i in range(T):
        p = parents[:, i]
        mask[:, i] = np.where((p >= 0)[:, None], mask[np.arange(B), np.maximum(p, 0)], np.uint64(0))
        mask[:, i, i // 64] |= np.uint64(1 << (i % 64))
    return mask.view(np.int64)


def _cached(c, gen, rng, lens, tokens, both):
    """A page table for `tokens` cached tokens per sequence, in shuffled pages."""
    need = -(-tokens // c["page"])
    width, total = max(1, int(need.max())), int(need.sum())
    pages = total + 3
    table = np.full((c["B"], width), -1, np.int32)
    table[np.arange(width)[None, :] < need[:, None]] = rng.permutation(pages)[:total]
    shape = (pages, c["page"], c["Hkv"], c["D"])
    s = {"c": c, "k": _normal(gen, c["dtype"], *shape), "pages": torch.from_numpy(table).cuda(),
         "lens": torch.from_numpy(lens).int().cuda()}
    if both:
        s["v"] = _normal(gen, c["dtype"], *shape)
    return s


def _prepare_attn(c, gen, rng):
    lens = rng.permutation(_lens(c))
    nodes = np.full(c["B"], c["T"], np.int64)
    if c["ragged"]:
        nodes = rng.integers(1, c["T"] + 1, c["B"])
    nodes[lens == 0] = 0
    s = _cached(c, gen, rng, lens, lens + nodes, c["op"] == "tree")
    s["parents"] = _parents(c, rng)
    s["nodes"] = torch.from_numpy(nodes).int().cuda()
    s["mask"] = torch.from_numpy(_bits(s["parents"])).cuda() if c["deep"] else None
    s["q"] = _normal(gen, c["dtype"], c["B"], c["T"], c["Hq"], c["D"]) * 2
    if c["op"] == "weights":
        # what the attention before returned, and the sums of the steps so far
        s["lse"] = torch.stack([_scores64(s, b)[0].logsumexp(-1).float() for b in range(c["B"])])
        L = s["pages"].shape[1] * c["page"]
        old = torch.rand(c["B"], c["Hkv"], L, generator=gen, device="cuda") ** 4
        s["scores"] = old * (torch.arange(L, device="cuda") < s["lens"][:, None, None])
    return s


def _prepare_select(c, gen, rng):
    lens = rng.permutation(_lens(c))
    L = c["hi"] + 13
    x = torch.randn(c["B"], c["H"], L, generator=gen, device="cuda")
    # sums of softmax weights: over many orders of magnitude, with equal ones among them
    x = torch.exp(3 * x)
    coarse = torch.rand(x.shape, generator=gen, device="cuda") < 0.1
    x = torch.where(coarse, (x * 4).round() / 4, x)
    return {"c": c, "scores": x, "lens": torch.from_numpy(lens).int().cuda()}


def _prepare_keep(c, gen, rng):
    B, page, T = c["B"], c["page"], c["T"]
    lens = rng.permutation(_lens(c))
    full = lens + T
    need = -(-full // page)
    width = int(need.max()) + 1
    table = np.full((B, width), -1, np.int32)
    # pairs of rows share their first pages
    pairs = np.arange(B) % 2 == 1
    pairs[pairs] = np.minimum(lens[1::2], lens[:B // 2 * 2:2]) >= c["shared"] * page
    own_from = np.where(pairs, c["shared"], 0)
    mine = (np.arange(width) >= own_from[:, None]) & (np.arange(width) < need[:, None])
    pages = int(mine.sum()) + B * (c["shared"] + 1)
    table[mine] = rng.permutation(pages)[:int(mine.sum())]
    follow = np.nonzero(pairs)[0]
    table[follow, :c["shared"]] = table[follow - 1, :c["shared"]]
    s = {"c": c, "pool": _normal(gen, c["dtype"], c["planes"], pages, page, c["Hkv"], c["D"]),
         "pages": torch.from_numpy(table).cuda(), "lens": torch.from_numpy(full).int().cuda()}
    if c["kind"] == "path":
        # a path from a root: each node of a random tree goes on with one of its children
        parents = _parents(dict(B=B, T=T, deep=2), rng)
        keep = np.full((1, B, 1, T), -1, np.int32)
        counts = np.zeros(B, np.int64)
        for b in range(B):
            at = -1
            while counts[b] < 6:
                kids = np.nonzero(parents[b] == at)[0]
                if not len(kids):
                    break
                at = int(rng.choice(kids))
                keep[0, b, 0, counts[b]] = lens[b] + at
                counts[b] += 1
        s["base"] = torch.from_numpy(lens).int().cuda()
        s["keep"] = torch.from_numpy(keep).cuda()
    else:
        # the newest eighth, the first tokens, and some of the rest, another choice for every head
        n = torch.from_numpy(full).cuda()[None, :, None, None]
        L = int(full.max())
        at = torch.arange(L, device="cuda")
        x = torch.rand(c["groups"], B, c["Hkv"], L, generator=gen, device="cuda")
        x = torch.where((at < 4) | (at >= n - c["budget"] // 8), x + 2, x)
        x = torch.where(at < n, x, x - 9)
        got = x.topk(min(c["budget"], L), -1).indices.sort(-1).values
        counts = np.minimum(full, c["budget"])
        # rows that keep everything: their tokens in order
        got = torch.where(n <= c["budget"], torch.arange(got.shape[-1], device="cuda"), got)
        held = torch.arange(got.shape[-1], device="cuda") < torch.from_numpy(counts).cuda()[:, None, None]
        s["keep"] = torch.where(held, got, -1).int().contiguous()
        s["base"] = None
    s["counts"] = torch.from_numpy(counts).int().cuda()
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = np.random.default_rng(seed)
    if case["op"] == "mask":
        parents = _parents(case, rng)
        return {"c": case, "parents": torch.from_numpy(parents).cuda()}
    return {"tree": _prepare_attn, "weights": _prepare_attn, "select": _prepare_select,
            "keep": _prepare_keep}[case["op"]](case, gen, rng)


# ---------------------------------------------------------------- the plain forms

def _plain_mask(s):
    parents = s["parents"].long()
    B, T = parents.shape
    words = -(-T // 64)
    at = torch.arange(T, device="cuda")
    # seen[i][j]: j is on the path from the root to i; up: the node above everything seen so far
    seen = (at[:, None] == at).expand(B, T, T)
    up = parents
    for _ in range(max(1, (T - 1).bit_length())):
        on = (up >= 0)[..., None]
        seen = seen | (on & seen.gather(1, up.clamp(min=0)[..., None].expand(B, T, T)))
        up = torch.where(up >= 0, up.gather(1, up.clamp(min=0)), up)
    bits = torch.zeros(B, T, words * 64, dtype=torch.int64, device="cuda")
    bits[..., :T] = seen.long()
    mask = (bits.view(B, T, words, 64) << torch.arange(64, device="cuda")).sum(-1)
    return {"mask": mask, "depth": seen.sum(-1).int() - 1}


def _seen(s, L):
    """Which cached tokens each node sees, [B][T][L], and which of them are cached."""
    c = s["c"]
    T = c["T"]
    at = torch.arange(L, device="cuda")
    j = torch.arange(T, device="cuda")
    lens, nodes = s["lens"].long()[:, None], s["nodes"].long()[:, None]
    if s["mask"] is None:
        sees = (j <= j[:, None]).expand(c["B"], T, T)
    else:
        sees = (s["mask"][..., j // 64] >> (j % 64)) & 1 != 0
    sees = sees & (j < nodes)[:, None, :] & (j < nodes)[:, :, None]
    drafted = (at >= lens) & (at < lens + nodes)
    place = (at - lens).clamp(0, T - 1)
    late = sees.gather(2, place[:, None, :].expand(-1, T, -1)) & drafted[:, None, :]
    early = (at < lens)[:, None, :] & (j < nodes)[:, :, None]
    if c["window"]:
        early = early & (at >= (lens - c["window"])[:, None, :] + sees.sum(-1, keepdim=True))
    return early | late


def _plain_scores(s, seen):
    """Scores [B][Hkv][T * G][L] in 32 bits, -inf where not seen."""
    c = s["c"]
    B, T, G = c["B"], c["T"], c["Hq"] // c["Hkv"]
    held = seen.any(1)[:, None, :, None]
    k = s["k"][s["pages"].clamp(min=0).long()].view(B, -1, c["Hkv"], c["D"]).transpose(1, 2).float()
    q = s["q"].float().view(B, T, c["Hkv"], G, c["D"]).transpose(1, 2).reshape(B, c["Hkv"], T * G, c["D"])
    x = torch.matmul(q, k.masked_fill(~held, 0.0).transpose(2, 3)) * (c["D"] ** -0.5)
    x = x.view(B, c["Hkv"], T, G, -1).masked_fill(~seen[:, None, :, None], -math.inf)
    return x.view(B, c["Hkv"], T * G, -1), held


def _plain_tree(s):
    c = s["c"]
    B, T, G = c["B"], c["T"], c["Hq"] // c["Hkv"]
    seen = _seen(s, s["pages"].shape[1] * c["page"])
    x, held = _plain_scores(s, seen)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - top.clamp(min=torch.finfo(torch.float32).min))
    total = p.sum(-1, keepdim=True)
    v = s["v"][s["pages"].clamp(min=0).long()].view(B, -1, c["Hkv"], c["D"]).transpose(1, 2).float()
    out = torch.matmul(p, v.masked_fill(~held, 0.0)) / total.where(total > 0, torch.ones_like(total))
    out = out.view(B, c["Hkv"], T, G, c["D"]).transpose(1, 2).reshape(B, T, c["Hq"], c["D"])
    lse = (top + torch.log(total)).view(B, c["Hkv"], T, G).transpose(1, 2).reshape(B, T, c["Hq"])
    return {"out": out.to(s["q"].dtype), "lse": lse}


def _plain_weights(s):
    c = s["c"]
    B, T, G = c["B"], c["T"], c["Hq"] // c["Hkv"]
    L = s["pages"].shape[1] * c["page"]
    x, _ = _plain_scores(s, _seen(s, L))
    lse = s["lse"].view(B, T, c["Hkv"], G).transpose(1, 2).reshape(B, c["Hkv"], T * G, 1)
    w = torch.exp(x - lse).masked_fill(~torch.isfinite(lse), 0.0).sum(2)
    at, lens, nodes = torch.arange(L, device="cuda"), s["lens"][:, None, None], s["nodes"][:, None, None]
    w = torch.where(at < lens, s["scores"] * c["decay"] + w, w)
    return {"scores": w.masked_fill(at >= lens + nodes, 0.0)}


def _plain_select(s):
    c = s["c"]
    x, n = s["scores"], s["lens"].long()[:, None, None]
    at = torch.arange(x.shape[-1], device="cuda")
    # scores as whole numbers of the same order; NaN the least
    i = (x.nan_to_num(nan=-math.inf, posinf=math.inf, neginf=-math.inf) + 0.0).view(torch.int32).long()
    i = torch.where(i < 0, -2147483648 - i, i)
    i = torch.where((at < c["sinks"]) | (at >= n - c["recent"]), 1 << 40, i)
    i = torch.where(at < n, i, -(1 << 40))
    count = n.clamp(max=c["budget"])
    width = min(c["budget"], x.shape[-1])
    best = i.sort(dim=-1, descending=True, stable=True).indices[..., :width]
    held = torch.arange(width, device="cuda") < count
    best = torch.where(held, best, x.shape[-1]).sort(-1).values
    keep = torch.full((c["B"], c["H"], c["budget"]), -1, dtype=torch.int32, device="cuda")
    keep[..., :width] = torch.where(held, best, -1).int()
    out = torch.zeros_like(x)
    out[..., :width] = x.gather(2, best.clamp(max=x.shape[-1] - 1)).masked_fill(~held, 0.0)
    return {"keep": keep, "counts": count.view(-1).int(), "scores": out}


def _plain_keep(s):
    c = s["c"]
    pool, table, page, keep = s["pool"], s["pages"], c["page"], s["keep"].long()
    planes, n_pages = pool.shape[:2]
    rows, width = table.shape
    lens, counts = s["lens"].long(), s["counts"].long()
    base = s["base"].long() if s["base"] is not None else torch.zeros_like(lens)
    total = base + counts
    col = torch.arange(width, device="cuda")
    held = col < ((lens + page - 1) // page)[:, None]
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    refs.index_add_(0, table[held].long(), torch.ones_like(table[held]))
    # slots that receive another token, and the shared pages that they lie in
    i = base[:, None] + torch.arange(keep.shape[-1], device="cuda")
    real = i < total[:, None]
    moves = (real[:, None] & (keep != i[:, None])).any(2).any(0)
    written = torch.zeros(rows, width + 1, dtype=torch.int32, device="cuda")
    written.scatter_reduce_(1, torch.where(real, i // page, width), moves.int(), "amax")
    fresh = (written[:, :width] > 0) & held & (refs[table.clamp(min=0).long()] > 1)
    want = fresh.sum(1)
    free = (refs == 0).nonzero()[:, 0]
    ok = want.cumsum(0) <= free.numel()
    fresh = fresh & ok[:, None]
    rank = fresh.view(-1).long().cumsum(0).view(rows, width) - 1
    new = torch.where(fresh, free[rank.clamp(0, max(0, free.numel() - 1))].int() if free.numel() else table, table)
    lens_out = torch.where(ok, total, lens)
    new = torch.where(col < ((lens_out + page - 1) // page)[:, None], new, -1)
    # every slot of the written rows: its token's old place, whole pages where they are fresh
    t = torch.arange(width * page, device="cuda")
    k = (t - base[:, None]).clamp(0, keep.shape[-1] - 1)
    src = keep.gather(3, k[:, None, :].expand(keep.shape[0], rows, keep.shape[2], -1))
    src = torch.where(t < base[:, None, None], t, src)
    act = (ok[:, None] & (t < total[:, None]))[:, None] & ((src != t) | fresh.repeat_interleave(page, 1)[:, None])
    g, r, h, slot = act.nonzero(as_tuple=True)
    from_ = src[g, r, h, slot]
    sp, sl = table[r, from_ // page].long(), from_ % page
    dp, dl = new[r, slot // page].long(), slot % page
    # [groups][planes of a group][pages][slots][choices of tokens][rest]
    view = pool.view(keep.shape[0], planes // keep.shape[0], n_pages, page, keep.shape[2], -1)
    view[g, :, dp, dl, h] = view[g, :, sp, sl, h]
    return {"pages": new, "lens": lens_out.int(), "short": (~ok).sum().int().view(1), "pool": pool}


# ---------------------------------------------------------------- one pass

def _own(s):
    from bit_mixed_precision_amd import binding as tq
    c = s["c"]
    if c["op"] == "mask":
        mask, depth = tq.tq_tree_mask(s["parents"])
        return {"mask": mask, "depth": depth}
    if c["op"] == "tree":
        out, lse = tq.tq_tree_attention(s["q"], s["k"], s["v"], s["pages"], s["lens"], mask=s["mask"],
                                        nodes=s["nodes"], window=c["window"], return_lse=True)
        return {"out": out, "lse": lse}
    if c["op"] == "weights":
        # the library adds in place: to a copy, since the sums so far are an input
        return {"scores": tq.tq_cache_weights(s["q"], s["k"], s["pages"], s["lens"], s["lse"],
                                              s["scores"].clone(), mask=s["mask"], nodes=s["nodes"],
                                              window=c["window"], decay=c["decay"])}
    if c["op"] == "select":
        keep, counts, sums = tq.tq_cache_select(s["scores"], s["lens"], c["budget"], recent=c["recent"],
                                                sinks=c["sinks"])
        # the library's sums are as long as the budget: at the front of new rows
        width = min(c["budget"], s["scores"].shape[-1])
        scores = torch.zeros_like(s["scores"])
        scores[..., :width] = sums[..., :width]
        return {"keep": keep, "counts": counts, "scores": scores}
    pages, lens, short = tq.tq_pages_keep(s["pool"], s["pages"], s["lens"], s["keep"], s["counts"], c["page"],
                                          base=s["base"])
    return {"pages": pages, "lens": lens, "short": short, "pool": s["pool"]}


def run(state):
    if own:
        return _own(state)
    return {"mask": _plain_mask, "tree": _plain_tree, "weights": _plain_weights, "select": _plain_select,
            "keep": _plain_keep}[state["c"]["op"]](state)


# ---------------------------------------------------------------- in 64 bits

def _scores64(s, b):
    """Scores of sequence b [T][Hq][tokens] in fp64, -inf where a node does not see a
    token, and the places of its tokens; paths walked node by node from the parents."""
    c = s["c"]
    n, m, T, G = int(s["lens"][b]), int(s["nodes"][b]), c["T"], c["Hq"] // c["Hkv"]
    total = max(1, n + m)
    sees = np.zeros((T, total), bool)
    for i in range(m):
        path, at = [], i
        while at >= 0:
            path.append(at)
            at = at - 1 if not c["deep"] else int(s["parents"][b, at])
        start = max(0, n + len(path) - c["window"]) if c["window"] else 0
        sees[i, min(start, n):n] = True
        sees[i, n + np.array(path)] = True
    ids = s["pages"][b, :-(-total // c["page"])].long().clamp(min=0)
    k = s["k"][ids].flatten(0, 1)[:total].double().permute(1, 2, 0).contiguous()
    q = s["q"][b].double().view(T, c["Hkv"], G * c["D"]).transpose(0, 1).reshape(c["Hkv"], T * G, c["D"])
    x = torch.bmm(q, k) / math.sqrt(c["D"])
    x = x.view(c["Hkv"], T, G, total).transpose(0, 1).reshape(T, c["Hq"], total)
    return x.masked_fill(~torch.from_numpy(sees).cuda()[:, None], -math.inf), ids


def exact(case, seed):
    c = case
    if c["op"] not in ("tree", "weights"):
        return None  # nothing is computed: tokens and bits are chosen, numbered and moved
    s = prepare(c, seed)
    B, T, G, Hkv = c["B"], c["T"], c["Hq"] // c["Hkv"], c["Hkv"]
    if c["op"] == "weights":
        L = s["pages"].shape[1] * c["page"]
        got = torch.zeros(B, Hkv, L, dtype=torch.float64, device="cuda")
        for b in range(B):
            n, m = int(s["lens"][b]), int(s["nodes"][b])
            if m == 0:
                got[b, :, :n] = s["scores"][b, :, :n].double() * c["decay"]
                continue
            x, _ = _scores64(s, b)
            lse = s["lse"][b].double()[..., None]
            w = torch.where(torch.isfinite(lse), torch.exp(x - lse), 0.0)
            got[b, :, :n + m] = w.view(T, Hkv, G, -1).sum((0, 2))
            got[b, :, :n] += s["scores"][b, :, :n].double() * c["decay"]
        return {"scores": got}
    out = torch.zeros(B, T, c["Hq"], c["D"], dtype=torch.float64, device="cuda")
    lse = torch.full((B, T, c["Hq"]), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        m = int(s["nodes"][b])
        if m == 0:
            continue
        x, ids = _scores64(s, b)
        x = x[:m]
        v = s["v"][ids].flatten(0, 1)[:x.shape[-1]].double().transpose(0, 1).contiguous()
        lse[b, :m] = torch.logsumexp(x, -1)
        p = torch.softmax(x, -1).view(m, Hkv, G, -1).transpose(0, 1).reshape(Hkv, m * G, -1)
        out[b, :m] = torch.bmm(p, v).view(Hkv, m, G, c["D"]).transpose(0, 1).reshape(m, c["Hq"], c["D"])
    return {"out": out, "lse": lse}
