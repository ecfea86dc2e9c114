"""Beam decoding with a small ternary decoder, every step on the library's operators.

One layer of the step: the fused q/k/v product (tq_gemm_tq2), rotary positions and
the write into the paged cache (tq_rope_append), attention of the new token over
the cache (tq_paged_attention), the output product, and the SwiGLU MLP
(tq_gemm_tq2_swiglu, tq_gemm_tq2).  Between steps the beams are selected, forked
(tq_pages_fork) and given room for their next token (tq_pages_grow); at the end
the pool is compacted (tq_pages_compact).

    python examples/decode_beams.py [--steps 24] [--beams 4] [--requests 2] [--check]

Random weights.  --check recomputes the last step's logits of every beam from its
whole token sequence in fp64 on the CPU, without a cache.
"""

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bit_mixed_precision_amd import binding as tq  # noqa: E402

HIDDEN, FFN, HEADS, KV_HEADS, D, LAYERS, VOCAB = 512, 1024, 8, 2, 64, 2, 300
PAGE, POSITIONS, THETA = 16, 1024, 5e5


class Linear:
    """A ternarized matrix on the GPU, and its dense values for the check."""

    def __init__(self, rng, n, k):
        W = rng.normal(0, 0.02, (n, k)).astype(np.float32)
        qs, scales, _ = tq.tq_pack_tq2(W)
        self.dense = tq.tq_unpack_tq2(qs, k) * np.repeat(scales.astype(np.float64), 256, axis=1)
        self.qs, self.scales = torch.from_numpy(qs).cuda(), torch.from_numpy(scales).cuda()

    def __call__(self, x):
        return tq.tq_gemm_tq2(x, self.qs, self.scales)


class Model:
    def __init__(self, seed):
        rng = np.random.default_rng(seed)
        self.embed = torch.from_numpy(rng.normal(0, 1, (VOCAB, HIDDEN)).astype(np.float16)).cuda()
        self.layers = [dict(qkv=Linear(rng, (HEADS + 2 * KV_HEADS) * D, HIDDEN),
                            out=Linear(rng, HIDDEN, HEADS * D), gate=Linear(rng, FFN, HIDDEN),
                            up=Linear(rng, FFN, HIDDEN), down=Linear(rng, HIDDEN, FFN))
                       for _ in range(LAYERS)]
        self.table = torch.from_numpy(tq.tq_rope_table(POSITIONS, D, THETA)).cuda()


def norm(x):
    x = x.float()
    return (x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-5)).half()


def step(model, tokens, pool, pages, lens, positions):
    """Logits [rows][VOCAB] of one new token per row; lens count it already."""
    x = model.embed[tokens.long()]
    for i, w in enumerate(model.layers):
        k, v = pool[2 * i], pool[2 * i + 1]
        qkv = w["qkv"](norm(x)).view(len(tokens), HEADS + 2 * KV_HEADS, D)
        q = tq.tq_rope_append(qkv, model.table, positions, pages, k, v)
        a = tq.tq_paged_attention(q, k, v, pages, lens)
        x = x + w["out"](a.view(len(tokens), HEADS * D))
        h = tq.tq_gemm_tq2_swiglu(norm(x), w["gate"].qs, w["gate"].scales, w["up"].qs, w["up"].scales)
        x = x + w["down"](h)
    return norm(x).float() @ model.embed.float().t() * (4 / HIDDEN)


def decode(model, prompts, beams, steps):
    """Beam search from prompts [requests][length]; returns a dict of its state."""
    requests, length = prompts.shape
    rows = requests * beams
    if rows > 16:
        raise ValueError("the fused gate / up product takes 16 rows")
    each = -(-(length + steps) // PAGE)
    n_pages = rows * (each + 1)
    # uninitialised on purpose: what lies in unused slots has no influence
    pool = torch.empty(2 * LAYERS, n_pages, PAGE, KV_HEADS, D, dtype=torch.float16, device="cuda")
    pages = torch.full((rows, each), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
    # the prompts go into the first row of each request, which the beams then fork
    lead = (torch.arange(rows, device="cuda") % beams == 0).int()
    history = torch.zeros(rows, 0, dtype=torch.long, device="cuda")
    score = torch.zeros(rows, device="cuda")
    mine = torch.arange(rows, device="cuda") // beams
    for t in range(length):
        tokens = prompts[:, t].cuda()[mine]
        positions = torch.where(lead > 0, lens, torch.full_like(lens, -1))
        pages, lens, short = tq.tq_pages_grow(pages, lens, lead, n_pages, PAGE)
        logits = step(model, tokens, pool, pages, lens, positions)
        history = torch.cat([history, tokens[:, None]], 1)
    pages, lens, refs, short = tq.tq_pages_fork(pool, pages, lens, (mine * beams).int(), PAGE)
    logits = logits.view(requests, beams, VOCAB)[:, :1].expand(-1, beams, -1).reshape(rows, VOCAB)
    refused = short.clone()
    for t in range(steps):
        total = score[:, None] + torch.log_softmax(logits, -1)
        total = total.view(requests, beams, VOCAB)
        if t == 0:  # equal beams: take the best tokens of one
            total[:, 1:] = -float("inf")
        score, best = total.view(requests, -1).topk(beams, -1)
        parent = (best // VOCAB + beams * torch.arange(requests, device="cuda")[:, None]).view(-1)
        tokens, score = (best % VOCAB).view(-1), score.view(-1)
        pages, lens, refs, short = tq.tq_pages_fork(pool, pages, lens, parent.int(), PAGE)
        refused = refused + short
        history = torch.cat([history[parent], tokens[:, None]], 1)
        positions = lens.clone()
        pages, lens, short = tq.tq_pages_grow(pages, lens, torch.ones_like(lens), n_pages, PAGE)
        refused = refused + short
        logits = step(model, tokens, pool, pages, lens, positions)
    pages, used = tq.tq_pages_compact(pool, pages, lens, PAGE)
    # the last token once more on the compacted pool: the same keys in other pages
    again = step(model, tokens, pool, pages, lens, lens - 1)
    return dict(history=history, score=score, logits=logits, again=again, pages=pages, lens=lens,
                used=used, refused=refused, n_pages=n_pages)


def recompute(model, tokens):
    """Logits after the last of `tokens`, in fp64 from the whole sequence."""
    n = len(tokens)
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    rms = lambda x: x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-5)  # noqa: E731
    x = f(model.embed)[tokens]
    ang = np.arange(n)[:, None] * THETA ** (-2.0 * np.arange(D // 2) / D)
    cos, sin = np.cos(ang)[:, None], np.sin(ang)[:, None]

    def turn(y):
        a, b = y[..., :D // 2], y[..., D // 2:]
        return np.concatenate([a * cos - b * sin, b * cos + a * sin], -1)

    for w in model.layers:
        qkv = (rms(x) @ w["qkv"].dense.T).reshape(n, HEADS + 2 * KV_HEADS, D)
        q, k, v = turn(qkv[:, :HEADS]), turn(qkv[:, HEADS:HEADS + KV_HEADS]), qkv[:, HEADS + KV_HEADS:]
        k, v = (np.repeat(t, HEADS // KV_HEADS, axis=1) for t in (k, v))
        s = np.einsum("qhd,khd->hqk", q, k) / np.sqrt(D)
        s = np.where(np.tril(np.ones((n, n), bool)), s, -np.inf)
        p = np.exp(s - s.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        a = np.einsum("hqk,khd->qhd", p, v).reshape(n, HEADS * D)
        x = x + a @ w["out"].dense.T
        g = rms(x) @ w["gate"].dense.T
        x = x + (g / (1 + np.exp(-g)) * (rms(x) @ w["up"].dense.T)) @ w["down"].dense.T
    return rms(x[-1]) @ f(model.embed).T * (4 / HIDDEN)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=24)
    ap.add_argument("--beams", type=int, default=4)
    ap.add_argument("--requests", type=int, default=2)
    ap.add_argument("--prompt", type=int, default=21)
    ap.add_argument("--check", action="store_true")
    a = ap.parse_args(argv)
    model = Model(0)
    prompts = torch.from_numpy(np.random.default_rng(1).integers(0, VOCAB, (a.requests, a.prompt)))
    out = decode(model, prompts, a.beams, a.steps)
    used, rows = int(out["used"]), len(out["lens"])
    alone = rows * -(-(a.prompt + a.steps) // PAGE)
    print(f"{rows} beams of {a.prompt + a.steps} tokens in {used} pages ({alone} without sharing), "
          f"{int(out['refused'])} refused; best scores "
          f"{[round(float(s), 3) for s in out['score'].view(a.requests, -1)[:, 0]]}")
    if a.check:
        want = np.stack([recompute(model, h) for h in out["history"].cpu().numpy()])
        err = max(np.abs(out[k].double().cpu().numpy() - want).max() for k in ("logits", "again"))
        print(f"logits against fp64 without a cache: {err:.2e} of {np.abs(want).max():.2f}")
        out["error"], out["scale"] = err, np.abs(want).max()
    return out


if __name__ == "__main__":
    main()
