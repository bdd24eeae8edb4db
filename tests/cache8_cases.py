"""Seeded inputs and comparisons of the tests of the cache held in e4m3 codes.

Tolerance of the attention, derived before its first run.  K, V and their
scales enter the products exactly; what is rounded is P, to f16 (at most half
a step, 2^-11 of a weight), and the output, to bf16 (2^-8 of it).  Weights below
2^-21 of the largest weight times V's scale are subnormal in f16 and off by
2^-32 of that largest at most, times a code of at most 448.  The rest is
fp32: the scores (128 products; sum |q k| scale stays below 32 for N(0,1)
queries and keys of sizes up to 2, so at most 128 * 2^-24 * 32 < 2^-11), their
exponents of at most some 2^7 (2^-17 each), exp2 and sums (2^-20): below 2^-10
of A, the sum of softmax weight times |v|, in all.  LSE: the scores' 2^-11 again,
below 1e-3 with the rest.
"""
from __future__ import annotations

import numpy as np
import torch

from cache_cases import LSE_TOL, Batch, ints  # noqa: F401
from oracle import cache as oc
from oracle import cache8 as o8
from oracle.attention import to64

F8 = torch.float8_e4m3fn
NAN = 0x7f


def codes64(t):
    """Codes as float64 values."""
    return t.cpu().view(torch.uint8).view(F8).to(torch.float32).numpy().astype(np.float64)


def same_codes(got, want):
    """Codes against float64 values, NaN equal to NaN and -0 to 0."""
    return np.array_equal(codes64(got), want, equal_nan=True)


def quantized(rng, pool, device):
    """Codes and scales of a bf16 pool [pages][page][Hkv][d] whose blocks get sizes between 1/8
    and 2; NaN values become NaN codes, and blocks of nothing else get a NaN as their scale."""
    pages, page, Hkv, d = pool.shape
    x = pool.float().view(pages, page // o8.BLOCK, o8.BLOCK, Hkv, d)
    x = x * torch.from_numpy(2.0 ** rng.uniform(-3, 1, (pages, page // o8.BLOCK, 1, Hkv, 1))).float()
    top = x.abs().nan_to_num(0.0).amax((2, 4))
    s = torch.from_numpy(o8.scale_for(top.numpy().astype(np.float64))).float()
    c = (x / s[:, :, None, :, None]).clamp(-448, 448).to(F8).view(pages, page, Hkv, d)
    s = torch.where(x.isnan().all(4).all(2), float("nan"), s)
    return c.to(device), s.transpose(1, 2).contiguous().to(device)


class Batch8(Batch):
    """Batch over a cache of codes; unused places hold NaN."""

    def __init__(self, seed, lens, nodes, H, Hkv, d, page, kind=None, device="cuda", extra_pages=3):
        super().__init__(seed, lens, nodes, H, Hkv, d, page, kind, device="cpu", extra_pages=extra_pages)
        rng = np.random.default_rng(seed + 1000)
        self.k, self.k_scale = quantized(rng, self.k, device)
        self.v, self.v_scale = quantized(rng, self.v, device)
        self.q = self.q.to(device)
        self.table, self.lens_t, self.cu = (x.to(device) for x in (self.table, self.lens_t, self.cu))
        if self.parents is not None:
            self.parents = self.parents.to(device)

    def check(self, o, lse, rows=None, seqs=None, tol=1.0):
        """O and LSE against the oracle (all packed rows; `rows`: at most that many a sequence;
        `seqs`: of these sequences only)."""
        sk, sv = (x.cpu().numpy().astype(np.float64) for x in (self.k_scale, self.v_scale))
        q, go, gl = to64(self.q), to64(o), lse.cpu().numpy().astype(np.float64)
        kc, vc = self.k.cpu(), self.v.cpu()
        for b, n in enumerate(self.nodes):
            if n == 0 or (seqs is not None and b not in seqs):
                continue
            see = oc.visible(n, self.lens[b] - n, None if self.parents is None else self.parents_np[b])
            own = self.table_np[b, :-(-self.lens[b] // self.page)]
            kk, vv = (o8.values(codes64(x.view(torch.uint8)[torch.tensor(own)].view(F8)), s[own])
                      .reshape(-1, self.Hkv, self.d)[:self.lens[b]] for x, s in ((kc, sk), (vc, sv)))
            per_key = np.repeat(o8.as_read(sv[own]).transpose(0, 2, 1).reshape(-1, self.Hkv), o8.BLOCK, axis=0)[:self.lens[b]]
            pick = np.arange(n) if rows is None or rows >= n else \
                np.unique(np.concatenate([[0, n - 1], self.rng.choice(n, rows, replace=False)]))
            at = self.cu_np[b] + pick
            ro, rl, a = oc.tree_attention(q[at], kk, vv, see[pick], self.scale)
            assert np.array_equal(np.isneginf(gl[:, at]), np.isneginf(rl)), f"-inf LSE differ in {b}"
            dead = np.isneginf(rl)
            assert np.all(go[at][dead.T] == 0), "rows that see no key must have O = 0"
            small = self.lens[b] * 2.0 ** -32 * 448 * per_key.max(0)              # [Hkv], weights are 1 at most
            small = np.repeat(small, self.H // self.Hkv)[None, :, None]
            bound = (2.0 ** -11 + 2.0 ** -10) * a + 2.0 ** -8 * np.abs(ro) + small + 1e-30
            worst = (np.abs(go[at] - ro) - tol * bound).max()
            assert worst <= 0, f"sequence {b}: O off by {worst} more than its bound"
            if (~dead).any():
                el = np.abs(gl[:, at][~dead] - rl[~dead]).max()
                assert el <= LSE_TOL, f"sequence {b}: LSE off by {el}"
