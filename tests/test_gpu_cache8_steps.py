"""Drafting and verifying on a cache of e4m3 codes, layer by layer and step by step: every attention against
the fp64 oracle over what the cache holds then, and what it holds against the tokens that were kept."""
import numpy as np
import pytest
import torch

import masked_attention_bound_gb300 as fm
from cache8_cases import F8, LSE_TOL, codes64, ints
from oracle import cache as oc
from oracle import cache8 as o8
from oracle.attention import to64
from test_gpu_cache8_pages import _freqs, pair_size

pytestmark = pytest.mark.gpu
PARENTS = [[-1, 0, 0, 1, 1, 2, 3, 6, 5], [-1, 0, 1, 1, 0, 4, 5, 6, 2]]
PATHS = [[[0, 2, 5], [0, 1, 2, 8]], [[0, 1, 3, 6, 7], [0, 4, 5]]]


@pytest.mark.parametrize("H,Hkv,d,page", [(4, 2, 64, 16), (8, 2, 128, 32), (40, 2, 128, 16)])
def test_every_step(H, Hkv, d, page):
    rng = np.random.default_rng(60)
    g = torch.Generator().manual_seed(61)
    words, layers, pages = 40, 2, 40
    # words of sizes from 1/8 to 8, so that scales of blocks grow and differ
    size = torch.exp2(torch.randint(-3, 4, (words,), generator=g).float())[:, None, None]
    emb = [(torch.randn(layers, words, n, d, generator=g) * s).to(torch.bfloat16).cuda()
           for n, s in ((H, 1.0), (Hkv, size), (Hkv, size))]
    freqs, scale = _freqs(d // 4), 0.25 * d ** -0.5
    pools = [torch.zeros(layers, pages, page, Hkv, d, device="cuda").to(F8) for _ in range(2)]
    scales = [fm.cache_scales(p) for p in pools]
    kw = dict(k_scale=scales[0], v_scale=scales[1])
    table = torch.full((2, 12), -1, dtype=torch.int32, device="cuda")
    lens, ref = ints([0, 0]), torch.zeros(pages, dtype=torch.int32, device="cuda")
    kept = [[], []]

    def held(which, layer, s, n):
        """Sequence s's first n tokens: values and the scale of each token and head."""
        own = table[s, :-(-n // page)].tolist()
        sc = scales[which][layer].cpu().numpy().astype(np.float64)[own]
        x = o8.values(codes64(pools[which][layer].view(torch.uint8)[own].view(F8)), sc).reshape(-1, Hkv, d)[:n]
        return x, np.repeat(o8.as_read(sc).transpose(0, 2, 1).reshape(-1, Hkv), o8.BLOCK, axis=0)[:n]

    def step(tokens, parents):
        nonlocal lens
        n = [len(t) for t in tokens]
        fm.pages_reserve(ints(n), *pools, table, lens, ref, **kw)
        cu_np = np.concatenate([[0], np.cumsum(n)])
        cu, flat = ints(cu_np), torch.tensor(sum(tokens, [])).cuda()
        depth = [[0 if p < 0 else None for p in pp] for pp in parents]
        for dd, pp in zip(depth, parents):
            for i, p in enumerate(pp):
                if p >= 0:
                    dd[i] = dd[p] + 1
        pos = np.concatenate([len(kept[s]) + np.array(depth[s]) for s in range(2)]).astype(int)
        for i in range(layers):
            q, k, v = (e[i][flat] for e in emb)
            lay = dict(k_scale=scales[0][i], v_scale=scales[1][i])
            rq = fm.cache_append_rotary(q, k, v, cu, freqs, pools[0][i], pools[1][i], table, lens, positions=ints(pos), **lay)
            o, lse = fm.tree_forward(rq, pools[0][i], pools[1][i], table, lens, cu, scale, parents=ints(sum(parents, [])),
                                     max_nodes=max(n), **lay)
            go, gl, qq = to64(o), lse.cpu().numpy().astype(np.float64), to64(rq)
            for s in range(2):
                total = int(lens[s])
                kk, vv = held(0, i, s, total)[0], held(1, i, s, total)[0]
                at = slice(cu_np[s], cu_np[s + 1])
                ro, rl, a = oc.tree_attention(qq[at], kk, vv, oc.visible(n[s], total - n[s], parents[s]), scale)
                # P to f16 (2^-11 of a weight), the output (2^-8 of it), fp32 sums (2^-10)
                assert (np.abs(go[at] - ro) <= (2.0 ** -11 + 2.0 ** -10) * a + 2.0 ** -8 * np.abs(ro) + 1e-6).all(), (i, s)
                assert np.abs(gl[:, at] - rl).max() <= LSE_TOL
        return cu

    def check_kept():
        for s in range(2):
            n = len(kept[s])
            assert int(lens[s]) == n
            for i in range(layers):
                k, v = (to64(e[i][torch.tensor(kept[s]).cuda()]) for e in emb[1:])
                rk = o8.rotate(k, np.arange(n), to64(freqs), False)
                for which, want, sz in ((0, rk, pair_size(k, d // 4, False)), (1, v, np.zeros(v.shape))):
                    x, sc = held(which, i, s, n)
                    # half a step of a code, 2^-4 of the value, and below the scale's normal codes 2^-10 of
                    # the scale for each time it grew: scales are powers of two, so these sum to 2^-9
                    bound = 2.0 ** -4 * np.abs(want) * (1 + 2.0 ** -10) + 2.0 ** -9 * sc[..., None] + 2.0 ** -22 * sz
                    assert (np.abs(x - want) <= bound).all(), (s, i, which)

    prompts = [rng.integers(0, words, m).tolist() for m in (21, 5)]
    step(prompts, [[i - 1 for i in range(len(p))] for p in prompts])
    kept = [list(p) for p in prompts]
    check_kept()
    for turn in range(6):
        nodes = [rng.integers(0, words, 9).tolist() for _ in range(2)]
        cu = step(nodes, PARENTS)
        paths = PATHS[turn % 2]
        most = max(len(p) for p in paths)
        lens = fm.cache_accept(ints([p + [0] * (most - len(p)) for p in paths]), ints([len(p) for p in paths]), cu,
                               *pools, table, lens, ref=ref, **kw)
        for s, p in enumerate(paths):
            kept[s] += [nodes[s][x] for x in p]
        check_kept()
