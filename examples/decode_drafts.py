"""Greedy decoding that checks drafted tokens, several a step, and a cache kept short.

The decoder of decode_beams.py.  Every step lays a small tree of tokens behind the last
cached one: the newest token and two guesses at what follows it, taken from where that
token stood before.  The tree's paths (tq_tree_mask) say which node sees which; keys and
values go to the slots after the cached ones (tq_rope_append with slots), the nodes attend
to the cache and to their own paths (tq_tree_attention), and of the nodes the path
that the model itself would have taken stays (tq_pages_keep).  Prompts go in as chains
of nodes.  With --budget every head of every layer keeps that many tokens, those that
have received the most attention (tq_cache_weights, tq_cache_select, tq_pages_keep).

    python examples/decode_drafts.py [--steps 40] [--requests 2] [--budget 48] [--check]

Random weights.  --check recomputes the last logits of every request from its whole
token sequence in fp64 on the CPU, without a cache (and needs one that is whole).
"""

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from decode_beams import D, HEADS, KV_HEADS, LAYERS, PAGE, VOCAB, Model  # noqa: E402
from decode_beams import norm, recompute, tq  # noqa: E402

NODES, BRANCH, RECENT, SINKS = 7, 3, 8, 4


class Cache:
    """Pages of `requests` sequences of `capacity` tokens and a tree; `lens` slots in use,
    `at` tokens seen, and the attention that every slot has received."""

    def __init__(self, requests, capacity):
        width = -(-(capacity + NODES) // PAGE)
        self.n_pages = requests * width
        # uninitialised on purpose, as in decode_beams.py
        self.pool = torch.empty(2 * LAYERS, self.n_pages, PAGE, KV_HEADS, D, dtype=torch.float16,
                                device="cuda")
        self.pages = torch.full((requests, width), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(requests, dtype=torch.int32, device="cuda")
        self.at = torch.zeros_like(self.lens)
        self.scores = torch.zeros(LAYERS, requests, KV_HEADS, width * PAGE, device="cuda")
        self.refused = torch.zeros(1, dtype=torch.int32, device="cuda")


def step(model, cache, tokens, parents, nodes):
    """Logits [requests][NODES][VOCAB] of the first nodes[b] nodes, and what their
    attention leaves for `settle`."""
    B = len(nodes)
    mask, depth = tq.tq_tree_mask(parents)
    cache.pages, total, short = tq.tq_pages_grow(cache.pages, cache.lens, nodes, cache.n_pages, PAGE)
    cache.refused += short
    i = torch.arange(NODES, device="cuda", dtype=torch.int32)
    there = i < nodes[:, None]
    positions = torch.where(there, cache.at[:, None] + depth, -1).int().view(-1)
    slots = torch.where(there, cache.lens[:, None] + i, -1).int().view(-1)
    seqs = torch.arange(B, device="cuda", dtype=torch.int32).repeat_interleave(NODES)
    x, seen = model.embed[tokens.view(-1).long()], []
    for n, w in enumerate(model.layers):
        k, v = cache.pool[2 * n], cache.pool[2 * n + 1]
        qkv = w["qkv"](norm(x)).view(B * NODES, HEADS + 2 * KV_HEADS, D)
        q = tq.tq_rope_append(qkv, model.table, positions, cache.pages, k, v, seqs=seqs, slots=slots)
        q = q.view(B, NODES, HEADS, D)
        a, lse = tq.tq_tree_attention(q, k, v, cache.pages, cache.lens, mask=mask, nodes=nodes,
                                      return_lse=True)
        seen.append((q, lse))
        x = x + w["out"](a.view(B * NODES, HEADS * D))
        h = tq.tq_gemm_tq2_swiglu(norm(x), w["gate"].qs, w["gate"].scales, w["up"].qs, w["up"].scales)
        x = x + w["down"](h)
    logits = norm(x).float() @ model.embed.float().t() * (4 / x.shape[1])
    return logits.view(B, NODES, VOCAB), (seen, mask, nodes, total)


def settle(cache, left, paths, counts, budget):
    """Keeps the nodes paths[b][:counts[b]] of a step, and `budget` tokens (0: all)."""
    seen, mask, nodes, total = left
    lists = (cache.lens[:, None] + paths).int()
    if budget:
        taken = torch.zeros(paths.shape[0], NODES + 1, dtype=torch.bool, device="cuda")
        used = torch.arange(paths.shape[1], device="cuda") < counts[:, None]
        taken.scatter_(1, torch.where(used, paths, NODES).long(), True)
        for n, (q, lse) in enumerate(seen):  # of the nodes that stay
            lse = lse.masked_fill(~taken[:, :NODES, None], -float("inf"))
            tq.tq_cache_weights(q, cache.pool[2 * n], cache.pages, cache.lens, lse, cache.scores[n],
                                mask=mask, nodes=nodes)
        # the sums move with their tokens
        to = cache.lens[:, None] + torch.arange(paths.shape[1], device="cuda")
        index = lambda t: t.long()[None, :, None].expand(LAYERS, -1, KV_HEADS, -1)  # noqa: E731
        cache.scores.scatter_(3, index(to), cache.scores.gather(3, index(lists)))
    cache.pages, lens, short = tq.tq_pages_keep(cache.pool, cache.pages, total, lists, counts, PAGE,
                                                base=cache.lens)
    cache.refused += short
    cache.at = cache.at + (lens - cache.lens)
    cache.lens = lens
    if budget:
        chosen = [tq.tq_cache_select(s, cache.lens, budget, RECENT, SINKS) for s in cache.scores]
        cache.pages, cache.lens, short = tq.tq_pages_keep(
            cache.pool, cache.pages, cache.lens, torch.stack([c[0] for c in chosen]), chosen[0][1], PAGE)
        cache.refused += short
        room = min(budget, cache.scores.shape[-1])
        cache.scores[..., :room] = torch.stack([c[2] for c in chosen])[..., :room]


def guess(history):
    """Tokens and parents of a tree: the newest token, and up to BRANCH tokens each after two
    places where it stood before."""
    tokens, parents, starts = [history[-1]], [-1], set()
    for i in range(len(history) - 2, -1, -1):
        if history[i] == history[-1] and history[i + 1] not in starts and len(starts) < 2:
            starts.add(history[i + 1])
            for j, t in enumerate(history[i + 1:i + 1 + BRANCH]):
                parents.append(0 if j == 0 else len(tokens) - 1)
                tokens.append(t)
    return tokens, parents


def laid_out(lists, fill):
    return torch.tensor([x + [fill] * (NODES - len(x)) for x in lists], dtype=torch.int32, device="cuda")


def decode(model, prompts, steps, budget=0):
    """`steps` tokens or a few more behind each of the prompts (lists of tokens)."""
    if len(prompts) * NODES > 16:
        raise ValueError("the fused gate / up product takes 16 rows")
    # (a row's last step may go past its count by what a branch holds)
    room = max(len(p) for p in prompts) + steps + BRANCH + 1
    cache = Cache(len(prompts), room if not budget else min(room, budget + NODES))
    chain = torch.arange(NODES, device="cuda", dtype=torch.int32)
    history, calls = [list(p) for p in prompts], 0
    # all of a prompt but its last token, which begins the first tree
    for first in range(0, max(len(p) for p in prompts) - 1, NODES):
        parts = [p[first:min(first + NODES, len(p) - 1)] for p in prompts]
        nodes = torch.tensor([len(p) for p in parts], dtype=torch.int32, device="cuda")
        _, left = step(model, cache, laid_out(parts, 0), (chain - 1).expand(len(parts), -1).contiguous(),
                       nodes)
        settle(cache, left, chain.expand(len(parts), -1), nodes, budget)
    last = [None] * len(prompts)
    while any(len(h) < len(p) + steps for h, p in zip(history, prompts)):
        trees = [guess(h) if len(h) < len(p) + steps else ([], []) for h, p in zip(history, prompts)]
        nodes = torch.tensor([len(t) for t, _ in trees], dtype=torch.int32, device="cuda")
        logits, left = step(model, cache, laid_out([t for t, _ in trees], 0),
                            laid_out([p for _, p in trees], -1), nodes)
        best, paths = logits.argmax(-1).tolist(), []
        for b, (tokens, parents) in enumerate(trees):
            path = [0] if tokens else []
            for i in range(1, len(tokens)):
                if parents[i] == path[-1] and tokens[i] == best[b][path[-1]]:
                    path.append(i)
            history[b] += [best[b][i] for i in path]
            paths.append(path)
            if path:
                last[b] = logits[b, path[-1]]
        settle(cache, left, laid_out(paths, 0),
               torch.tensor([len(p) for p in paths], dtype=torch.int32, device="cuda"), budget)
        calls += 1
    return dict(history=history, logits=torch.stack(last), cache=cache, calls=calls)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--requests", type=int, default=2)
    ap.add_argument("--prompt", type=int, default=21)
    ap.add_argument("--budget", type=int, default=0)
    ap.add_argument("--check", action="store_true")
    a = ap.parse_args(argv)
    if a.check and a.budget:
        ap.error("--check needs a whole cache")
    model = Model(0)
    rng = np.random.default_rng(1)
    prompts = [rng.integers(0, VOCAB, max(1, a.prompt - 2 * i)).tolist() for i in range(a.requests)]
    out = decode(model, prompts, a.steps, a.budget)
    new = [len(h) - len(p) for h, p in zip(out["history"], prompts)]
    print(f"{new} tokens in {out['calls']} steps, {out['cache'].lens.tolist()} cached, "
          f"{int(out['cache'].refused)} refused")
    out["prompts"] = prompts
    if a.check:
        want = np.stack([recompute(model, np.array(h[:-1])) for h in out["history"]])
        err = np.abs(out["logits"].double().cpu().numpy() - want).max()
        print(f"logits against fp64 without a cache: {err:.2e} of {np.abs(want).max():.2f}")
        out["error"], out["scale"] = err, np.abs(want).max()
    return out


if __name__ == "__main__":
    main()
