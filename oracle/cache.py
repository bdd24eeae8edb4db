"""The paged K/V cache from its definitions, in numpy float64 and Python integers.

A cache is a pair of pools [layers][pages][page_size][Hkv][d] (or one layer's,
without the first axis), a page table [B][max_pages] and lengths [B]; token p
of sequence b is at page table[b][p // page_size], slot p % page_size.
"""
from __future__ import annotations

import math

import numpy as np

PAD = -2


def ancestors(parents, t):
    """Node t and the nodes it was drafted after (none for a padding node)."""
    out = []
    while t >= 0 and parents[t] != PAD:
        out.append(t)
        t = parents[t]
    return out


def visible(n, context, parents=None):
    """Boolean [n][context + n]: which cached tokens each of n nodes sees."""
    see = np.zeros((n, context + n), dtype=bool)
    for t in range(n):
        nodes = range(t + 1) if parents is None else ancestors(parents, t)
        if len(nodes):
            see[t, :context] = True
            for a in nodes:
                see[t, context + a] = True
    return see


def gather(pool, table_row, length):
    """Tokens [length][Hkv][d] of a sequence from one layer's pool."""
    page = pool.shape[1]
    return np.stack([pool[table_row[p // page], p % page] for p in range(length)]) if length else \
        np.zeros((0,) + pool.shape[2:], pool.dtype)


def tree_attention(q, k, v, see, scale):
    """One sequence: q [n][H][d], k and v [S][Hkv][d], see [n][S].  Returns O [n][H][d],
    LSE [H][n] and A [n][H][d] = sum of softmax weight times |v|, the scale of O's errors."""
    n, H, d = q.shape
    G = H // k.shape[1]
    O, A, lse = np.zeros((n, H, d)), np.zeros((n, H, d)), np.full((H, n), -math.inf)
    for t in range(n):
        cols = np.nonzero(see[t])[0]
        if not len(cols):
            continue
        for h in range(H):
            s = scale * (k[cols, h // G] @ q[t, h])
            m = s.max()
            e = np.exp(s - m)
            vv = v[cols, h // G]
            O[t, h] = (e[:, None] * vv).sum(0) / e.sum()
            A[t, h] = (e[:, None] * np.abs(vv)).sum(0) / e.sum()
            lse[h, t] = m + math.log(e.sum())
    return O, lse, A


def append(k_new, cu, pool, table, lens):
    """New tokens written to a copy of one layer's pool."""
    pool, page = pool.copy(), pool.shape[1]
    for b in range(len(lens)):
        n = cu[b + 1] - cu[b]
        for i in range(n):
            p = lens[b] - n + i
            pool[table[b][p // page], p % page] = k_new[cu[b] + i]
    return pool


def accept(nodes, cu, pool, table, lens):
    """Accepted nodes (a list per sequence) moved together in a copy of [layers] pools."""
    pool, page, out = pool.copy(), pool.shape[2], []
    for b, acc in enumerate(nodes):
        base = lens[b] - (cu[b + 1] - cu[b])
        old = [pool[:, table[b][(base + a) // page], (base + a) % page].copy() for a in acc]
        for i, x in enumerate(old):
            pool[:, table[b][(base + i) // page], (base + i) % page] = x
        out.append(base + len(acc))
    return pool, out


def fork(parent, rows, lens, ref):
    """rows: a list of pages per sequence.  New rows, lengths and counts."""
    ref = list(ref)
    new = [list(rows[p]) if p >= 0 else [] for p in parent]
    for r in new:
        for p in r:
            ref[p] += 1
    for r in rows:
        for p in r:
            ref[p] -= 1
    return new, [lens[p] if p >= 0 else 0 for p in parent], ref


def reserve(grow, rows, lens, ref, page, max_pages):
    """New rows, lengths, counts, copies [(from, to, tokens)] and pages asked for; the inputs and
    None where the free pages do not suffice or a row would not fit (such a row asks for none)."""
    free = [p for p, r in enumerate(ref) if r == 0]
    new, ln, rf, copies, asked = [list(r) for r in rows], list(lens), list(ref), [], 0
    short = False

    def take():
        nonlocal asked, short
        asked += 1
        if asked > len(free):
            short = True
            return -1
        return free[asked - 1]

    for b, r in enumerate(new):
        if ln[b] + grow[b] > max_pages * page:
            short = True
            continue
        if grow[b] > 0 and ln[b] % page and ref[r[-1]] > 1:
            p = take()
            copies.append((r[-1], p, ln[b] % page))
            rf[r[-1]] -= 1
            r[-1] = p
            rf[p] = 1
        ln[b] += grow[b]
        while len(r) * page < ln[b]:
            r.append(take())
            rf[r[-1]] = 1
    if short:
        return [list(r) for r in rows], list(lens), list(ref), None, asked
    return new, ln, rf, copies, asked


def compact(rows, ref):
    """New rows, counts, moves [(from, to)] and the number of held pages."""
    n_live = sum(1 for r in ref if r != 0)
    holes = [p for p in range(n_live) if ref[p] == 0]
    movers = [p for p in range(n_live, len(ref)) if ref[p] != 0]
    to = dict(zip(movers, holes))
    out = [0] * len(ref)
    for p, r in enumerate(ref):
        if r:
            out[to.get(p, p)] = r
    return [[to.get(p, p) for p in r] for r in rows], out, list(zip(movers, holes)), n_live
