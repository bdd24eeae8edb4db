"""Seeded inputs and comparisons of the paged-cache tests.

Tolerances, derived once: the kernel rounds P to bf16 (at most half a step,
2^-8 relative) before it multiplies V, so O is off by at most 2^-8 A with A =
sum of softmax weight times |v|, and its output rounding adds 2^-8 |O|.
What is left is fp32: the scores (128 products of N(0,1) values, at most
128 * 2^-24 * sum|qk| * scale < 1e-4), exp2 and sums of some thousand terms
(2^-24 each): below 2^-10 A for O, and below 1e-3 for LSE.
"""
from __future__ import annotations

import numpy as np
import torch

from oracle import cache as oc
from oracle.attention import to64

LSE_TOL = 1e-3


def o_excess(got, ref, a):
    """How far |O - O_ref| is past its bound (<= 0: within)."""
    return np.abs(got - ref) - ((2.0 ** -8 + 2.0 ** -10) * a + 2.0 ** -8 * np.abs(ref) + 1e-30)


def ints(x, device="cuda"):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=device)


def tree_parents(rng, n, kind):
    """A tree of n nodes: 'chain', 'star' (all roots), 'random', 'padded' (random with padding
    nodes in the middle and at the end), 'beams' (a root and branches)."""
    if kind == "chain":
        return [t - 1 for t in range(n)]
    if kind == "star":
        return [-1] * n
    if kind == "beams":
        return [-1 if t == 0 else max(0, t - 3) for t in range(n)]
    p = [-1] + [int(rng.integers(-1, t)) for t in range(1, n)]
    if kind == "padded":
        for t in range(n):
            if t >= n - n // 4 or rng.random() < 0.2:
                p[t] = oc.PAD
    return p


class Batch:
    """A packed batch over a paged cache whose unused places hold `fill`."""

    def __init__(self, seed, lens, nodes, H, Hkv, d, page, kind=None, fill=float("nan"), device="cuda",
                 extra_pages=3):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.rng, self.page, self.H, self.Hkv, self.d = rng, page, H, Hkv, d
        self.lens, self.nodes = list(lens), list(nodes)
        B = len(lens)
        used = [-(-x // page) for x in lens]
        n_pages = sum(used) + extra_pages
        order = rng.permutation(n_pages)
        self.max_pages = max(used) + 2
        table = np.full((B, self.max_pages), -7, np.int64)
        at = 0
        for b, u in enumerate(used):
            table[b, :u] = order[at:at + u]
            at += u
        self.free = sorted(order[at:].tolist())
        self.table_np = table
        self.cu_np = np.concatenate([[0], np.cumsum(nodes)]).astype(int)
        T = int(self.cu_np[-1])
        pools = []
        for _ in range(2):
            p = torch.full((n_pages, page, Hkv, d), fill, dtype=torch.bfloat16)
            for b, x in enumerate(lens):
                for j in range(used[b]):
                    m = min(page, x - j * page)
                    p[table[b, j], :m] = torch.randn(m, Hkv, d, generator=g).to(torch.bfloat16)
            pools.append(p)
        q = torch.randn(T, H, d, generator=g).to(torch.bfloat16)
        self.k, self.v, self.q = (x.to(device) for x in (*pools, q))
        self.table, self.lens_t, self.cu = (ints(x, device) for x in (table, lens, self.cu_np))
        self.parents_np = self.parents = None
        if kind is not None:
            self.parents_np = [tree_parents(rng, n, kind) if n else [] for n in nodes]
            self.parents = ints(sum(self.parents_np, []) or np.zeros(0), device)
        self.scale = d ** -0.5

    def check(self, o, lse, rows=None, seqs=None):
        """O and LSE against the oracle (all packed rows; `rows`: at most that many a sequence;
        `seqs`: of these sequences only)."""
        k, v, q = self.k.cpu(), self.v.cpu(), to64(self.q)
        go, gl = to64(o), lse.cpu().numpy().astype(np.float64)
        for b, n in enumerate(self.nodes):
            if n == 0 or (seqs is not None and b not in seqs):
                continue
            see = oc.visible(n, self.lens[b] - n, None if self.parents is None else self.parents_np[b])
            used = -(-self.lens[b] // self.page)
            kk, vv = (to64(x[torch.tensor(self.table_np[b, :used])].reshape(-1, self.Hkv, self.d)[:self.lens[b]])
                      for x in (k, v))
            pick = np.arange(n) if rows is None or rows >= n else \
                np.unique(np.concatenate([[0, n - 1], self.rng.choice(n, rows, replace=False)]))
            at = self.cu_np[b] + pick
            ro, rl, a = oc.tree_attention(q[at], kk, vv, see[pick], self.scale)
            assert np.array_equal(np.isneginf(gl[:, at]), np.isneginf(rl)), f"-inf LSE differ in {b}"
            dead = np.isneginf(rl)
            assert np.all(go[at][dead.T] == 0), "rows that see no key must have O = 0"
            worst = o_excess(go[at], ro, a).max()
            assert worst <= 0, f"sequence {b}: O off by {worst} more than its bound"
            if (~dead).any():
                el = np.abs(gl[:, at][~dead] - rl[~dead]).max()
                assert el <= LSE_TOL, f"sequence {b}: LSE off by {el}"
