"""Plain fp64 definitions of the decode-side operators (numpy; test infrastructure).

Rotary positions, attention of one new token over a paged cache, and the page
bookkeeping, each written from its definition with loops over tokens, rows and
pages.  Shares no code with the library.
"""

from __future__ import annotations

import numpy as np


def rope_frequencies_ref(rot, theta, scaling="none", factor=1.0, trained=4096.0, fast=32.0,
                         slow=1.0):
    """f_i, i < rot / 2, as include/tq.h defines them for each scaling."""
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "base":
        theta = theta * factor ** (rot / (rot - 2))
    f = theta ** (-2.0 * i / rot)
    if scaling == "linear":
        f = f / factor
    elif scaling == "parts":
        keep = np.clip((trained * f / (2 * np.pi) - slow) / (fast - slow), 0.0, 1.0)
        f = f * keep + f / factor * (1 - keep)
    return f


def rope_ref(X, positions, freq, interleaved=False, inverse=False, gain=1.0, n_pos=None):
    """X [T][H][D] with each pair of the first 2 len(freq) numbers turned by
    positions[t] freq[i]; rows of positions outside [0, n_pos) are zero."""
    X = np.asarray(X, dtype=np.float64)
    half = len(freq)
    Y = X.copy()
    for t, p in enumerate(np.asarray(positions).tolist()):
        if p < 0 or (n_pos is not None and p >= n_pos):
            Y[t] = 0
            continue
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            ang = p * freq[i] * (-1 if inverse else 1)
            Y[t, :, a] = gain * (X[t, :, a] * np.cos(ang) - X[t, :, b] * np.sin(ang))
            Y[t, :, b] = gain * (X[t, :, b] * np.cos(ang) + X[t, :, a] * np.sin(ang))
    return Y


def cached_rows_ref(pages, page_table_row, tokens):
    """[len(tokens)][Hkv][D] and which of them are present: token t is slot
    t % page_size of page page_table_row[t // page_size]; a page that does not
    exist holds nothing."""
    n_pages, size = pages.shape[:2]
    out = np.zeros((len(tokens),) + pages.shape[2:])
    there = np.zeros(len(tokens), dtype=bool)
    for j, t in enumerate(tokens):
        page = int(page_table_row[t // size])
        if 0 <= page < n_pages:
            out[j] = pages[page, t % size]
            there[j] = True
    return out, there


def paged_attention_ref(Q, k_pages, v_pages, page_table, lens, scale, window=0):
    """(out [B][Hq][D], lse [B][Hq], score and value magnitudes for error bounds).

    The last two say, for each (b, h), the largest sum_d |q_d k_d| scale over the
    tokens, and for each (b, h, d) sum_t w_t |v_td|."""
    B, Hq, D = Q.shape
    n_pages, size, Hkv, _ = k_pages.shape
    G = Hq // Hkv
    out, lse = np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf)
    smag, vmag = np.zeros((B, Hq)), np.zeros((B, Hq, D))
    for b in range(B):
        n = min(max(int(lens[b]), 0), page_table.shape[1] * size)
        full = max(int(lens[b]), 0)
        lo = max(0, full - window) if window else 0
        tokens = list(range(lo, n))
        if not tokens:
            continue
        k, there = cached_rows_ref(k_pages, page_table[b], tokens)
        v, _ = cached_rows_ref(v_pages, page_table[b], tokens)
        k, v = k[there], v[there]
        if not len(k):
            continue
        for h in range(Hq):
            kh, vh, q = k[:, h // G], v[:, h // G], Q[b, h].astype(np.float64)
            s = (kh @ q) * scale
            top = s.max()
            if top == -np.inf:
                continue
            w = np.exp(s - top)
            lse[b, h] = top + np.log(w.sum())
            w = w / w.sum()
            out[b, h] = w @ vh
            smag[b, h] = (np.abs(kh) @ np.abs(q)).max() * abs(scale)
            vmag[b, h] = w @ np.abs(vh)
    return out, lse, smag, vmag


def _held(lens, row, width, size):
    return -(-min(max(int(lens[row]), 0), width * size) // size)


def pages_fork_ref(page_table, lens, parent, n_pages, size):
    """(page table, lengths, refs, short, copies [(src, dst)]) of tq_pages_fork."""
    page_table = np.asarray(page_table)
    rows_in, width = page_table.shape
    rows = len(parent)
    table, new_lens = np.full((rows, width), -1, np.int32), np.zeros(rows, np.int32)
    wants, seen, used = [], set(), set()
    for r in range(rows):
        p = int(parent[r])
        if not 0 <= p < rows_in:
            continue
        n = _held(lens, p, width, size)
        new_lens[r] = min(max(int(lens[p]), 0), width * size)
        table[r, :n] = page_table[p, :n]
        own = n
        if new_lens[r] % size and p in seen and 0 <= table[r, n - 1] < n_pages:
            wants.append((r, n - 1, int(table[r, n - 1])))
            own = n - 1
        seen.add(p)
        used.update(int(x) for x in table[r, :own] if 0 <= x < n_pages)
    free = [p for p in range(n_pages) if p not in used]
    copies, short = [], 0
    for r, at, src in wants:
        if free:
            dst = free.pop(0)
            table[r, at] = dst
            copies.append((src, dst))
        else:
            table[r, at] = -1
            new_lens[r] = new_lens[r] // size * size
            short += 1
    refs = np.zeros(n_pages, np.int32)
    for x in table.ravel():
        if 0 <= x < n_pages:
            refs[x] += 1
    return table, new_lens, refs, short, copies


def pages_grow_ref(page_table, lens, add, n_pages, size):
    """(page table, lengths, refused rows) of tq_pages_grow."""
    page_table = np.asarray(page_table)
    rows, width = page_table.shape
    table, new_lens = np.full((rows, width), -1, np.int32), np.zeros(rows, np.int32)
    used = set()
    held = [_held(lens, r, width, size) for r in range(rows)]
    for r in range(rows):
        table[r, :held[r]] = page_table[r, :held[r]]
        new_lens[r] = min(max(int(lens[r]), 0), width * size)
        used.update(int(x) for x in table[r, :held[r]] if 0 <= x < n_pages)
    free = [p for p in range(n_pages) if p not in used]
    wanted, refused = 0, 0
    for r in range(rows):
        want = int(new_lens[r]) + max(int(add[r]), 0)
        need = -(-want // size) - held[r]
        if want > width * size:
            refused += 1
            continue
        wanted += need
        if need and wanted > len(free):
            refused += 1
            continue
        table[r, held[r]:held[r] + need] = free[wanted - need:wanted]
        new_lens[r] = want
    return table, new_lens, refused


def pages_compact_ref(page_table, lens, n_pages, size):
    """(page table, pages in use, moves [(src, dst)]) of tq_pages_compact."""
    page_table = np.asarray(page_table)
    rows, width = page_table.shape
    table = np.full((rows, width), -1, np.int32)
    used = set()
    for r in range(rows):
        n = _held(lens, r, width, size)
        table[r, :n] = page_table[r, :n]
        used.update(int(x) for x in table[r, :n] if 0 <= x < n_pages)
    n = len(used)
    moves = list(zip(sorted(p for p in used if p >= n), (p for p in range(n) if p not in used)))
    to = dict(moves)
    for r in range(rows):
        for j in range(_held(lens, r, width, size)):
            table[r, j] = to.get(int(table[r, j]), table[r, j])
    return table, n, moves
