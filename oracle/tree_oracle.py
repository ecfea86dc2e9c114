"""Plain fp64 definitions of the operators on several new tokens per sequence and on
caches that are kept short (numpy; test infrastructure): the paths of drafted trees,
attention of their nodes, the weight each cached token receives, the choice of tokens
to keep, and moving them together.  Shares no code with the library.
"""

from __future__ import annotations

import numpy as np

from .decode_oracle import _held, cached_rows_ref


def tree_paths_ref(parents):
    """bool [B][T][T]: j is i or a node above it; a parent that is no node before i is none."""
    B, T = parents.shape
    seen = np.zeros((B, T, T), bool)
    for b in range(B):
        for i in range(T):
            j = i
            while 0 <= j:
                seen[b, i, j] = True
                p = int(parents[b, j])
                j = p if 0 <= p < j else -1
    return seen


def mask_words_ref(seen):
    """The int64 words [B][T][ceil(T / 64)] of bool [B][T][T]."""
    B, T, _ = seen.shape
    words = -(-T // 64)
    out = np.zeros((B, T, words), np.uint64)
    for j in range(T):
        out[:, :, j // 64] |= np.where(seen[:, :, j], np.uint64(1) << np.uint64(j % 64), np.uint64(0))
    return out.view(np.int64)


def tree_tokens_ref(n, m, sees, width_tokens, window):
    """bool [m][tokens]: which tokens each of m nodes sees; n cached tokens before them."""
    n = min(max(n, 0), width_tokens)
    total = min(n + m, width_tokens)
    out = np.zeros((m, total), bool)
    for i in range(m):
        mine = [j for j in range(m) if sees[i, j]]
        lo = max(0, n + len(mine) - window) if window else 0
        out[i, min(lo, n):n] = True
        for j in mine:
            if n + j < total:
                out[i, n + j] = True
    return out


def _scores(Q, k_pages, page_table, lens, nodes, sees, scale, window, b):
    """(scores [m][Hq][tokens], -inf where not seen; seen; magnitudes; present) of sequence b."""
    _, T, Hq, D = Q.shape
    size, Hkv = k_pages.shape[1:3]
    G = Hq // Hkv
    m = min(max(int(nodes[b]), 0), T)
    seen = tree_tokens_ref(int(lens[b]), m, sees[b], page_table.shape[1] * size, window)
    tokens = range(seen.shape[1])
    k, there = cached_rows_ref(k_pages, page_table[b], tokens)
    seen &= there[None]
    k = np.where((seen.any(0))[:, None, None], k, 0.0)
    q = Q[b, :m].reshape(m, Hkv, G, D)
    shape = (m, Hq, seen.shape[1])
    s = np.einsum("ihgd,thd->ihgt", q, k).reshape(shape) * scale
    mag = np.einsum("ihgd,thd->ihgt", np.abs(q), np.abs(k)).reshape(shape) * abs(scale)
    return np.where(seen[:, None], s, -np.inf), seen, np.where(seen[:, None], mag, 0.0)


def tree_attention_ref(Q, k_pages, v_pages, page_table, lens, nodes, sees, scale, window=0):
    """(out [B][T][Hq][D], lse [B][T][Hq], score and value magnitudes for error bounds
    as paged_attention_ref's); sees bool [B][T][T]."""
    B, T, Hq, D = Q.shape
    Hkv = k_pages.shape[2]
    out, lse = np.zeros(Q.shape), np.full((B, T, Hq), -np.inf)
    smag, vmag = np.zeros((B, T, Hq)), np.zeros(Q.shape)
    for b in range(B):
        s, seen, mag = _scores(Q, k_pages, page_table, lens, nodes, sees, scale, window, b)
        m, _, total = s.shape
        if m == 0 or total == 0:
            continue
        v, _ = cached_rows_ref(v_pages, page_table[b], range(total))
        v = np.where(seen.any(0)[:, None, None], v, 0.0)
        top = s.max(-1, keepdims=True)
        w = np.exp(s - np.where(np.isfinite(top), top, 0.0))
        sums = w.sum(-1, keepdims=True)
        with np.errstate(divide="ignore"):
            lse[b, :m] = (np.where(np.isfinite(top), top, 0.0) + np.log(sums))[..., 0]
        w = (w / np.where(sums > 0, sums, 1.0)).reshape(m, Hkv, Hq // Hkv, total)
        out[b, :m] = np.einsum("ihgt,thd->ihgd", w, v).reshape(m, Hq, D)
        vmag[b, :m] = np.einsum("ihgt,thd->ihgd", w, np.abs(v)).reshape(m, Hq, D)
        smag[b, :m] = mag.max(-1)
    return out, lse, smag, vmag


def cache_weights_ref(Q, k_pages, page_table, lens, nodes, sees, lse, scores, decay, scale, window=0):
    """(scores [B][Hkv][S] after the call, the weights' own part, largest score magnitude
    [B])."""
    B, T, Hq, _ = Q.shape
    Hkv, S = k_pages.shape[2], scores.shape[2]
    size = k_pages.shape[1]
    out, add, smag = scores.astype(np.float64).copy(), np.zeros(scores.shape), np.zeros(B)
    for b in range(B):
        s, seen, mag = _scores(Q, k_pages, page_table, lens, nodes, sees, scale, window, b)
        m, _, total = s.shape
        l = lse[b, :m, :, None].astype(np.float64)
        w = np.where(np.isfinite(l), np.exp(s - np.where(np.isfinite(l), l, 0.0)), 0.0)
        w = w.reshape(m, Hkv, Hq // Hkv, total).sum((0, 2))
        n = min(max(int(lens[b]), 0), page_table.shape[1] * size)
        a, c = min(n, S), min(total, S)
        add[b, :, :c] = w[:, :c]
        out[b, :, :a] = out[b, :, :a] * decay + w[:, :a]
        out[b, :, a:c] = w[:, a:c]
        smag[b] = mag.max() if mag.size else 0.0
    return out, add, smag


def cache_select_ref(scores, lens, budget, recent, sinks):
    """(keep int32 [B][H][budget], counts, sums) of tq_cache_select."""
    B, H, S = scores.shape
    keep = np.full((B, H, budget), -1, np.int32)
    sums = np.zeros((B, H, budget), np.float32)
    counts = np.zeros(B, np.int32)
    for b in range(B):
        n = min(max(int(lens[b]), 0), S)
        counts[b] = min(n, budget)
        for h in range(H):
            if n <= budget:
                got = list(range(n))
            else:
                got = set(range(sinks)) | set(range(n - recent, n))
                rest = [t for t in range(n) if t not in got]
                key = [-np.inf if np.isnan(scores[b, h, t]) else float(scores[b, h, t]) for t in rest]
                order = sorted(range(len(rest)), key=lambda i: (-key[i], rest[i]))
                got = sorted(got | {rest[i] for i in order[:budget - len(got)]})
            keep[b, h, :len(got)] = got
            sums[b, h, :len(got)] = scores[b, h, got]
    return keep, counts, sums


def pages_keep_ref(page_table, lens, keep, counts, base, n_pages, size):
    """(page table, lengths, short, moves) of tq_pages_keep; moves: (group, head, source
    page, slot, destination page, slot).  keep [groups][rows][heads][n]."""
    page_table = np.asarray(page_table)
    rows, width = page_table.shape
    groups, _, heads, n = keep.shape
    names = lambda p: 0 <= p < n_pages  # noqa: E731
    length = [min(max(int(x), 0), width * size) for x in lens]
    refs = np.zeros(n_pages, int)
    for r in range(rows):
        for e in range(_held(lens, r, width, size)):
            if names(page_table[r, e]):
                refs[page_table[r, e]] += 1
    free = [p for p in range(n_pages) if refs[p] == 0]
    table, out, short, moves = np.full_like(page_table, -1), np.zeros(rows, np.int32), 0, []
    asked = 0
    for r in range(rows):
        first = min(max(int(base[r]), 0), length[r]) if base is not None else 0
        total = min(first + min(max(int(counts[r]), 0), n), length[r])
        new_held = -(-total // size)

        def source(g, h, i):
            t = i if i < first else int(keep[g, r, h, i - first])
            return t if i <= t < length[r] else -1

        def acts(g, h, i):
            t = source(g, h, i)
            return t >= 0 and t != i

        fresh = []
        for e in range(new_held):
            p = page_table[r, e]
            if names(p) and refs[p] > 1 and any(
                    acts(g, h, i) for g in range(groups) for h in range(heads)
                    for i in range(max(first, e * size), min(total, (e + 1) * size))):
                fresh.append(e)
        asked += len(fresh)
        if fresh and asked > len(free):
            short += 1
            out[r] = length[r]
            held = _held(lens, r, width, size)
            table[r, :held] = page_table[r, :held]
            continue
        out[r] = total
        table[r, :new_held] = page_table[r, :new_held]
        for k, e in enumerate(fresh):
            table[r, e] = free[asked - len(fresh) + k]
        for g in range(groups):
            for h in range(heads):
                for i in range(total):
                    t = source(g, h, i) if acts(g, h, i) else i
                    if t == i and i // size not in fresh:
                        continue
                    sp, dp = page_table[r, t // size], table[r, i // size]
                    if names(sp) and names(dp):
                        moves.append((g, h, sp, t % size, dp, i % size))
    return table, out, short, moves
