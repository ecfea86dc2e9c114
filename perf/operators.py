"""The decode-side operators of this library as measurable cases.

Three operators that stand between the ternary products of one decoder layer:

* rotary positions: applied to the query and key heads of the fused q/k/v
  product (prompts, and their gradient), and applied while the new keys and
  values are written into a paged cache (decoding);
* attention of one new token over a paged key-value cache;
* the pages of that cache: forking sequences (beams) and compacting the pool.

``own`` chooses between the plain torch form (False) and the library (True).
Sizes: 64 query / 8 key-value heads of 128 and the 10240-wide q/k/v product are
the library's 70B-shaped decode stack; the others are generic.
"""

import math

import numpy as np
import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"f16": 2, "bf16": 2, "f32": 4}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one user, one new token: q/k/v of the 70B-shaped layer; latency only
        dict(name="append_1", op="append", dtype="f16", T=1, Hq=64, Hkv=8, D=128, rot=128,
             interleaved=False, scaling="none", n_pos=8192, page=16, pages=64),
        # a full decode batch with an odd number of sequences, interleaved pairs
        dict(name="append_251", op="append", dtype="bf16", T=251, Hq=32, Hkv=8, D=128, rot=128,
             interleaved=True, scaling="parts", n_pos=16384, page=16, pages=1024),
        # packed prompts: the q and k heads of the q/k/v product, scaled for a long context
        dict(name="rope_prompt_8192", op="rope", dtype="f16", T=8192, Hq=64, Hkv=8, D=128, rot=128,
             interleaved=False, scaling="linear", n_pos=32768, inverse=False),
        # training: the gradient through a rotation of part of a small head, ragged batch
        dict(name="rope_grad_4093", op="rope", dtype="f32", T=4093, Hq=20, Hkv=20, D=80, rot=32,
             interleaved=True, scaling="none", n_pos=4096, inverse=True),
        # one short chat: latency
        dict(name="attn_1x97", op="attn", dtype="f16", B=1, Hq=64, Hkv=8, D=128, page=16,
             lo=97, hi=97, empty=0, window=0),
        # heads that share nothing, small heads, short and ragged sequences, two unused slots
        dict(name="attn_37_ragged", op="attn", dtype="bf16", B=37, Hq=24, Hkv=24, D=64, page=32,
             lo=1, hi=4096, empty=2, window=0),
        # one very long document: the split over the cache's length
        dict(name="attn_1x131072", op="attn", dtype="f16", B=1, Hq=64, Hkv=8, D=128, page=64,
             lo=131072, hi=131072, empty=0, window=0),
        # a full serving batch of long chats
        dict(name="attn_96_long", op="attn", dtype="f16", B=96, Hq=64, Hkv=8, D=128, page=16,
             lo=2048, hi=8192, empty=0, window=0),
        # four beams of one request, four layers
        dict(name="fork_4", op="fork", dtype="f16", groups=1, beams=4, dup=1, prompt=100, own=20,
             planes=8, Hkv=8, D=128, page=16, pages=64),
        # sixteen requests of four beams, sixteen layers
        dict(name="fork_64", op="fork", dtype="f16", groups=16, beams=4, dup=2, prompt=500, own=75,
             planes=32, Hkv=8, D=128, page=16, pages=1024),
        # a small pool after one request ended
        dict(name="compact_128", op="compact", dtype="f16", S=3, used=61, moves=20, planes=4,
             Hkv=8, D=128, page=16, pages=128),
        # a large pool, under half in use and scattered
        dict(name="compact_2048", op="compact", dtype="bf16", S=48, used=930, moves=500, planes=16,
             Hkv=8, D=128, page=16, pages=2048),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "rope", "attn", "attn", "fork", "compact"])
    D = rng.choice([64, 80, 96, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8, 8, 12])
    group = rng.choice([1, 2, 3, 4, 8, 8, 16])
    dtype = rng.choice(["f16", "bf16"])
    page = rng.choice([16, 16, 32, 64, 128, 24])
    if op in ("append", "rope"):
        rot = rng.choice([D, D, D // 2 // 8 * 8, 32])
        c = dict(op=op, dtype=dtype, Hq=Hkv * group, Hkv=Hkv, D=D, rot=rot,
                 interleaved=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "parts"]),
                 n_pos=rng.choice([2048, 8192, 32768]))
        if op == "append":
            c.update(T=_log(rng, 1, 509), page=page, pages=max(512, 1024 * 16 // page))
        else:
            most = int(8192 * 72 * 128 / ((c["Hq"] + Hkv) * D))
            if rng.random() < 0.3:
                c["dtype"], most = "f32", most // 2
            c.update(T=_log(rng, 1, max(2, min(16384, most))), inverse=rng.random() < 0.5)
        return c
    if op == "attn":
        B = _log(rng, 1, 128)
        # the keys of the largest listed case, fewer where more heads read each
        room = 96 * 4400 * 8 * 128 * 8 // (B * Hkv * D * max(8, group))
        hi = _log(rng, 1, max(1, min(131072, room)))
        lo = _log(rng, 1, hi)
        return dict(op="attn", dtype=dtype, B=B, Hq=Hkv * group, Hkv=Hkv, D=D, page=page, lo=lo,
                    hi=hi, empty=rng.choice([0, 0, 1]) if B > 1 else 0,
                    window=rng.choice([0, 0, 0, _log(rng, 1, hi)]))
    if op == "fork":
        beams = rng.choice([2, 3, 4, 8])
        groups = _log(rng, 1, 64 // beams)
        own_tok = _log(rng, 1, 90)
        prompt = _log(rng, 1, 600)
        need = groups * (-(-prompt // page) + beams * (-(-own_tok // page) + 2))
        pages = need + rng.randint(groups * beams, 200)
        most = (32 * 1024 * 16 * 8 * 128) // (pages * page * Hkv * D)
        return dict(op="fork", dtype=dtype, groups=groups, beams=beams, dup=rng.randint(0, beams - 1),
                    prompt=prompt, own=own_tok, planes=max(1, _log(rng, 1, max(1, min(32, most)))),
                    Hkv=Hkv, D=D, page=page, pages=pages)
    pages = _log(rng, 16, 2048)
    used = rng.randint(1, pages)
    most = (32 * 1024 * 16 * 8 * 128) // (pages * page * Hkv * D)
    return dict(op="compact", dtype=dtype, S=min(used, _log(rng, 1, 64)), used=used,
                moves=rng.randint(0, min(used, pages - used)),
                planes=max(1, _log(rng, 1, max(1, min(32, most)))), Hkv=Hkv, D=D, page=page,
                pages=pages)


def _lens(c):
    """The lengths of an attention batch, in rising order: even over the logarithm."""
    n = c["B"] - c["empty"]
    q = np.arange(n) / max(1, n - 1) if n > 1 else np.ones(1)
    x = np.rint(np.exp(math.log(c["lo"]) + q * (math.log(c["hi"]) - math.log(c["lo"]))))
    return np.concatenate([np.zeros(c["empty"]), x]).astype(np.int64)


def _fork_lens(c):
    """(prompt pages, tokens) of a beam: shared full pages of the prompt, then
    pages of its own that end inside a page (one token in it at least)."""
    page = c["page"]
    shared = c["prompt"] // page
    length = c["prompt"] + c["own"]
    return shared, length + 1 if length % page == 0 and page > 1 else length


def work(c):
    e = _BYTES[c["dtype"]]
    if c["op"] == "append":
        h, rows = c["Hq"] + 2 * c["Hkv"], c["T"]
        nbytes = 2 * rows * h * c["D"] * e + rows * c["rot"] * 4 + rows * 8
        return {"bytes": nbytes, "flops": 3 * rows * (c["Hq"] + c["Hkv"]) * c["rot"]}
    if c["op"] == "rope":
        h, rows = c["Hq"] + c["Hkv"], c["T"]
        table = min(rows, c["n_pos"]) * c["rot"] * 4
        return {"bytes": 2 * rows * h * c["D"] * e + table + rows * 4, "flops": 3 * rows * h * c["rot"]}
    if c["op"] == "attn":
        n = _lens(c)
        n = int((np.minimum(n, c["window"]) if c["window"] else n).sum())
        io = 2 * c["B"] * c["Hq"] * c["D"] * e + 4 * (n // c["page"] + c["B"]) + 4 * c["B"] * c["Hq"]
        return {"bytes": 2 * n * c["Hkv"] * c["D"] * e + io, "flops": 4 * n * c["Hq"] * c["D"]}
    page_bytes = c["page"] * c["Hkv"] * c["D"] * e
    if c["op"] == "fork":
        s, length = c["groups"] * c["beams"], _fork_lens(c)[1]
        tables = 8 * s * -(-length // c["page"]) + 12 * s + 4 * c["pages"]
        copies = c["groups"] * c["dup"] * (length % c["page"] != 0)
        return {"bytes": 2 * copies * c["planes"] * page_bytes + tables, "flops": 0}
    return {"bytes": 2 * c["moves"] * c["planes"] * page_bytes + 8 * c["used"], "flops": 0}


# ---------------------------------------------------------------- the inputs

def _normal(gen, dtype, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float16 if dtype == "f16" else
                       torch.float32).to(_DT[dtype])


def _angles(c, positions):
    """cos and sin of every pair of `positions`, float64: [len][rot / 2] each.
    linear: positions divided by 4.  parts: each frequency between itself and a
    quarter of itself by how often it turns in a first context of 4096 (below
    one turn: a quarter, above 32: itself), both scaled by 0.1 ln 4 + 1."""
    half = c["rot"] // 2
    freq = 500000.0 ** (-torch.arange(half, dtype=torch.float64, device=positions.device) * 2 / c["rot"])
    gain = 1.0
    if c["scaling"] == "linear":
        freq = freq / 4
    elif c["scaling"] == "parts":
        turns = 4096 * freq / (2 * math.pi)
        keep = ((turns - 1) / 31).clamp(0, 1)
        freq = freq * keep + freq / 4 * (1 - keep)
        gain = 0.1 * math.log(4.0) + 1
    a = positions.double()[:, None] * freq
    return a.cos() * gain, a.sin() * gain


def _prepare_rotary(c, gen):
    T, D = c["T"], c["D"]
    s = {"c": c}
    s["table"] = torch.stack(_angles(c, torch.arange(c["n_pos"], device="cuda")), -1).float().contiguous()
    qkv = _normal(gen, c["dtype"], T, c["Hq"] + 2 * c["Hkv"], D)
    if c["op"] == "rope":
        # the q and k heads in place in the q/k/v product's rows; packed documents
        s["x"] = qkv[:, :c["Hq"] + c["Hkv"]]
        start = int(torch.randint(0, c["n_pos"], (1,), generator=gen, device="cuda"))
        s["pos"] = ((torch.arange(T, device="cuda") + start) % c["n_pos"]).int()
        return s
    s["qkv"] = qkv
    shape = (c["pages"], c["page"], c["Hkv"], D)
    s["k"], s["v"] = _normal(gen, c["dtype"], *shape), _normal(gen, c["dtype"], *shape)
    # one page for each sequence at the place where its new token goes
    width = -(-c["n_pos"] // c["page"])
    s["pos"] = torch.randint(0, c["n_pos"], (T,), generator=gen, device="cuda").int()
    s["pages"] = torch.full((T, width), -1, dtype=torch.int32, device="cuda")
    got = torch.randperm(c["pages"], generator=gen, device="cuda")[:T].int()
    s["pages"][torch.arange(T, device="cuda"), s["pos"].long() // c["page"]] = got
    return s


def _prepare_attn(c, gen, rng):
    lens = rng.permutation(_lens(c))
    need = -(-lens // c["page"])
    width, total = max(1, int(need.max())), int(need.sum())
    pages = total + 3
    table = np.full((c["B"], width), -1, np.int32)
    table[np.arange(width)[None, :] < need[:, None]] = rng.permutation(pages)[:total]
    shape = (pages, c["page"], c["Hkv"], c["D"])
    return {"c": c, "q": _normal(gen, c["dtype"], c["B"], c["Hq"], c["D"]) * 2,
            "k": _normal(gen, c["dtype"], *shape), "v": _normal(gen, c["dtype"], *shape),
            "pages": torch.from_numpy(table).cuda(), "lens": torch.from_numpy(lens).int().cuda()}


def _prepare_fork(c, gen, rng):
    S, beams = c["groups"] * c["beams"], c["beams"]
    shared, length = _fork_lens(c)
    each = -(-length // c["page"])
    ids = rng.permutation(c["pages"])
    prompt = ids[:c["groups"] * shared].reshape(c["groups"], 1, shared)
    rest = ids[c["groups"] * shared:][:S * (each - shared)].reshape(c["groups"], beams, each - shared)
    table = np.concatenate([np.broadcast_to(prompt, (c["groups"], beams, shared)), rest], 2)
    full = np.full((S, each + 2), -1, np.int32)
    full[:, :each] = table.reshape(S, each)
    # each group keeps beams - dup of its beams; the best of them goes on dup times more
    keep = rng.permuted(np.tile(np.arange(beams), (c["groups"], 1)), axis=1)
    keep[:, beams - c["dup"]:] = keep[:, :1]
    parent = (rng.permuted(keep, axis=1) + beams * np.arange(c["groups"])[:, None]).reshape(-1)
    return {"c": c, "pool": _normal(gen, c["dtype"], c["planes"], c["pages"], c["page"], c["Hkv"], c["D"]),
            "pages": torch.from_numpy(full).cuda(),
            "lens": torch.full((S,), length, dtype=torch.int32, device="cuda"),
            "parent": torch.from_numpy(parent).int().cuda()}


def _prepare_compact(c, gen, rng):
    low = rng.permutation(c["used"])[:c["used"] - c["moves"]]
    high = c["used"] + rng.permutation(c["pages"] - c["used"])[:c["moves"]]
    ids = rng.permutation(np.concatenate([low, high]))
    # the pages dealt out to S sequences, the last page of each partly filled
    cut = np.sort(rng.permutation(c["used"] - 1)[:c["S"] - 1] + 1) if c["S"] > 1 else np.zeros(0, int)
    need = np.diff(np.concatenate([[0], cut, [c["used"]]])).astype(np.int64)
    table = np.full((c["S"], c["used"] - c["S"] + 2), -1, np.int32)
    table[np.arange(table.shape[1])[None, :] < need[:, None]] = ids
    lens = need * c["page"] - rng.integers(0, c["page"], c["S"])
    return {"c": c, "pool": _normal(gen, c["dtype"], c["planes"], c["pages"], c["page"], c["Hkv"], c["D"]),
            "pages": torch.from_numpy(table).cuda(), "lens": torch.from_numpy(lens).int().cuda()}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = np.random.default_rng(seed)
    if case["op"] in ("append", "rope"):
        return _prepare_rotary(case, gen)
    return {"attn": _prepare_attn, "fork": _prepare_fork, "compact": _prepare_compact}[case["op"]](case, gen, rng)


# ---------------------------------------------------------------- the plain forms

def _rotate(x, cos, sin, rot, interleaved, inverse):
    """Pairs of the first `rot` numbers of each head turned by their angles."""
    x = x.to(cos.dtype)
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    if inverse:
        sin = -sin
    y, z = a * cos - b * sin, a * sin + b * cos
    y = torch.stack([y, z], -1).flatten(-2) if interleaved else torch.cat([y, z], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_rope(s):
    c = s["c"]
    cs = s["table"][s["pos"].long()][:, None]
    return {"y": _rotate(s["x"], cs[..., 0], cs[..., 1], c["rot"], c["interleaved"], c["inverse"]).to(s["x"].dtype)}


def _plain_append(s):
    c = s["c"]
    qk, v = s["qkv"][:, :c["Hq"] + c["Hkv"]], s["qkv"][:, c["Hq"] + c["Hkv"]:]
    cs = s["table"][s["pos"].long()][:, None]
    y = _rotate(qk, cs[..., 0], cs[..., 1], c["rot"], c["interleaved"], False).to(qk.dtype)
    pos = s["pos"].long()
    page = s["pages"].gather(1, (pos // c["page"])[:, None])[:, 0].long()
    s["k"][page, pos % c["page"]] = y[:, c["Hq"]:]
    s["v"][page, pos % c["page"]] = v
    return {"q": y[:, :c["Hq"]].contiguous(), "k": s["k"], "v": s["v"]}


def _plain_attn(s):
    c = s["c"]
    B, width = s["pages"].shape
    at = torch.arange(width * c["page"], device="cuda")
    n = s["lens"].long()[:, None]
    seen = at < n
    if c["window"]:
        seen = seen & (at >= n - c["window"])
    ids = s["pages"].clamp(min=0).long()
    rows = seen[:, None, :, None]

    def cached(pool):  # [B][Hkv][tokens][D] in 32 bits, zero where not seen
        x = pool[ids].view(B, -1, c["Hkv"], c["D"]).transpose(1, 2).float()
        return x.masked_fill(~rows, 0.0)

    q = s["q"].float().view(B, c["Hkv"], -1, c["D"])
    scores = torch.matmul(q, cached(s["k"]).transpose(2, 3)) * (c["D"] ** -0.5)
    scores = scores.masked_fill(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - top.clamp(min=torch.finfo(torch.float32).min))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, cached(s["v"])) / total.where(total > 0, torch.ones_like(total))
    return {"out": out.reshape(B, c["Hq"], c["D"]).to(s["q"].dtype),
            "lse": (top + torch.log(total)).reshape(B, c["Hq"])}


def _held(pages, lens, page):
    """Which table entries hold a page."""
    return torch.arange(pages.shape[1], device="cuda") < ((lens.long() + page - 1) // page)[:, None]


def _refs(pages, held, n_pages):
    """How many table entries hold each page."""
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    return refs.index_add_(0, pages[held].long(), torch.ones_like(pages[held]))


def _plain_fork(s):
    c = s["c"]
    parent = s["parent"].long()
    lens = s["lens"][parent]
    pages = s["pages"][parent]
    # the first child of a parent keeps its part-filled page, the others need one of their own
    same = parent[:, None] == parent[None, :]
    later = same.tril(-1).any(1)
    copies = later & (lens % c["page"] != 0)
    last = (lens.long() // c["page"])[copies]
    src = pages[copies].gather(1, last[:, None])[:, 0].long()
    kept = pages.clone()
    kept[copies.nonzero()[:, 0], last] = -1
    held = _held(kept, lens, c["page"])
    used = torch.zeros(c["pages"], dtype=torch.bool, device="cuda")
    used[kept[held & (kept >= 0)].long()] = True
    dst = (~used).nonzero()[:src.numel(), 0]
    s["pool"][:, dst] = s["pool"][:, src]
    kept[copies.nonzero()[:, 0], last] = dst.int()
    return {"pages": kept, "lens": lens, "refs": _refs(kept, held, c["pages"]), "pool": s["pool"]}


def _plain_compact(s):
    c = s["c"]
    held = _held(s["pages"], s["lens"], c["page"])
    used = _refs(s["pages"], held, c["pages"]) > 0
    n = used.sum()
    at = torch.arange(c["pages"], device="cuda")
    src = (used & (at >= n)).nonzero()[:, 0]
    dst = (~used & (at < n)).nonzero()[:, 0]
    to = at.int()
    to[src] = dst.int()
    s["pool"][:, dst] = s["pool"][:, src]
    pages = torch.where(held, to[s["pages"].clamp(min=0).long()], torch.full_like(s["pages"], -1))
    return {"pages": pages, "used": n.int().reshape(1), "pool": s["pool"]}


# ---------------------------------------------------------------- one pass

def _own(s):
    from bit_mixed_precision_amd import binding as tq
    c = s["c"]
    if c["op"] == "rope":
        return {"y": tq.tq_rope(s["x"], s["table"], s["pos"], interleaved=c["interleaved"], inverse=c["inverse"])}
    if c["op"] == "append":
        q = tq.tq_rope_append(s["qkv"], s["table"], s["pos"], s["pages"], s["k"], s["v"],
                              interleaved=c["interleaved"])
        return {"q": q, "k": s["k"], "v": s["v"]}
    if c["op"] == "attn":
        out, lse = tq.tq_paged_attention(s["q"], s["k"], s["v"], s["pages"], s["lens"], window=c["window"],
                                         return_lse=True)
        return {"out": out, "lse": lse}
    if c["op"] == "fork":
        pages, lens, refs, _ = tq.tq_pages_fork(s["pool"], s["pages"], s["lens"], s["parent"], c["page"])
        return {"pages": pages, "lens": lens, "refs": refs, "pool": s["pool"]}
    pages, used = tq.tq_pages_compact(s["pool"], s["pages"], s["lens"], c["page"])
    return {"pages": pages, "used": used, "pool": s["pool"]}


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "append": _plain_append, "attn": _plain_attn, "fork": _plain_fork,
            "compact": _plain_compact}[state["c"]["op"]](state)


# ---------------------------------------------------------------- in 64 bits

def _exact_turn(x, c, pos, inverse):
    """Each pair as a complex number times e^(i angle), from the angle's definition."""
    rot = c["rot"]
    cos, sin = _angles(c, pos.double())
    w = torch.complex(cos, -sin if inverse else sin)[:, None]
    x = x.double().clone()
    lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if c["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
    z = torch.complex(x[..., lo].contiguous(), x[..., hi].contiguous()) * w
    x[..., lo], x[..., hi] = z.real, z.imag
    return x


def exact(case, seed):
    c = case
    if c["op"] in ("fork", "compact"):
        return None  # nothing is computed: pages are copied and numbered
    s = prepare(case, seed)
    if c["op"] == "rope":
        return {"y": _exact_turn(s["x"], c, s["pos"], c["inverse"])}
    if c["op"] == "append":
        y = _exact_turn(s["qkv"][:, :c["Hq"] + c["Hkv"]], c, s["pos"], False)
        k, v = s["k"].double(), s["v"].double()
        for t, p in enumerate(s["pos"].tolist()):
            page = int(s["pages"][t, p // c["page"]])
            k[page, p % c["page"]] = y[t, c["Hq"]:]
            v[page, p % c["page"]] = s["qkv"][t, c["Hq"] + c["Hkv"]:].double()
        return {"q": y[:, :c["Hq"]].contiguous(), "k": k, "v": v}
    out = torch.zeros(c["B"], c["Hq"], c["D"], dtype=torch.float64, device="cuda")
    lse = torch.full((c["B"], c["Hq"]), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        lo = max(0, n - c["window"]) if c["window"] else 0
        if n == lo:
            continue
        ids = s["pages"][b, :-(-n // c["page"])].long()
        k = s["k"][ids].flatten(0, 1)[lo:n].double().permute(1, 2, 0).contiguous()
        v = s["v"][ids].flatten(0, 1)[lo:n].double().transpose(0, 1).contiguous()
        x = torch.bmm(s["q"][b].double().view(c["Hkv"], -1, c["D"]), k) / math.sqrt(c["D"])
        lse[b] = torch.logsumexp(x, -1).flatten()
        out[b] = torch.bmm(torch.softmax(x, -1), v).reshape(c["Hq"], c["D"])
    return {"out": out, "lse": lse}
