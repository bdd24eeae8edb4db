"""Cases, plain forms and exact results of the operators of a paged K/V cache
held in 8 bits, and of appending with the position rotation.

Operators: attention of drafted trees, causal runs and single tokens over a
paged cache of e4m3 codes with a scale for each block of 16 tokens and head;
appending new tokens, their keys (and queries) rotated by position on the way,
to a cache of bf16 or of e4m3 codes; moving the accepted nodes of a tree
together in a cache of e4m3 codes, between blocks of different scales.

``own`` selects what ``run`` executes: the plain forms in elementary torch
operations, or this package's calls.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

BLOCK = 16                    # tokens that share a scale
LEAST, MOST = -60, 60         # exponents of the scales
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one token of one short sequence: the latency of a call
        dict(name="attend one token", op="attend", B=1, ctx=256, nodes=1, branch=0, H=2, Hkv=2,
             d=64, page=16),
        # a decoding step of a full batch with ragged contexts, 4 query heads per K/V head
        dict(name="attend decode batch", op="attend", B=128, ctx=8192, nodes=1, branch=0, H=32,
             Hkv=8, d=128, page=64),
        # verification of drafted trees, padded to 64 nodes each, ragged contexts, small pages
        dict(name="attend trees", op="attend", B=16, ctx=16384, nodes=64, branch=4, H=32, Hkv=8,
             d=128, page=16),
        # one very long sequence with a drafted tree: the work has to be split along the keys
        dict(name="attend long context", op="attend", B=1, ctx=131072, nodes=32, branch=3, H=8,
             Hkv=2, d=128, page=128),
        # the next piece of a few prompts that are read in pieces of 480 tokens
        dict(name="attend prompt pieces", op="attend", B=4, ctx=2000, nodes=480, branch=0, H=32,
             Hkv=8, d=128, page=32),
        # a decoding step's query, K and V of one sequence, half of each head rotated, neighbours
        # as pairs, a cache of bf16
        dict(name="append one token", op="append", B=1, ctx=1000, nodes=1, H=2, Hkv=2, d=64,
             page=16, bits=16, rot=32, inter=True, branch=0),
        # a packed batch of prompts of 16K tokens in all (U[512, 4096] each), a cache of bf16
        dict(name="append prompts", op="append", B=7, ctx=4096, nodes=4096, H=16, Hkv=16, d=128,
             page=16, bits=16, rot=128, inter=False, branch=0),
        # a decoding step's queries, K and V of one layer, a cache of 8 bits
        dict(name="append decode batch 8 bits", op="append", B=128, ctx=4096, nodes=1, H=32, Hkv=8,
             d=128, page=64, bits=8, rot=128, inter=False, branch=0),
        # the same packed batch of prompts, 4 query heads per K/V head, a cache of 8 bits
        dict(name="append prompts 8 bits", op="append", B=7, ctx=4096, nodes=4096, H=32, Hkv=8,
             d=128, page=16, bits=8, rot=128, inter=False, branch=0),
        # drafted trees: a node's position is its depth's, not its place in the cache
        dict(name="append trees 8 bits", op="append", B=16, ctx=1024, nodes=64, H=32, Hkv=8, d=128,
             page=16, bits=8, rot=64, inter=False, branch=4),
        # after the verification of one tree, a small model
        dict(name="accept one tree", op="accept", B=1, ctx=1000, nodes=32, take=6, L=4, Hkv=2,
             d=64, page=16),
        # after the verification of a batch, all layers of a model at once
        dict(name="accept batch", op="accept", B=64, ctx=1024, nodes=64, take=8, L=16, Hkv=8,
             d=128, page=16),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "append", "accept"])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    c = dict(op=op, Hkv=Hkv, d=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]))
    if op == "attend":
        H = Hkv * rng.choice([1, 2, 3, 4, 5, 7, 8])
        B = _logint(rng, 1, 128)
        # the K/V of the cache stays below that of the largest listed case
        most = (1 << 32) // (B * Hkv * c["d"] * 4)
        c.update(B=B, ctx=_logint(rng, 1, min(131072, most)), H=H)
        branch = rng.choice([0, 0, 2, 3, 8])
        nodes = 1 if branch == 0 and rng.random() < 0.5 else _logint(rng, 2, 64 if branch else 480)
        # as many score products as the largest listed case has, at most
        nodes = max(1, min(nodes, (1 << 29) // (B * H * (c["ctx"] + nodes))))
        c.update(nodes=nodes, branch=branch)
    elif op == "append":
        branch = rng.choice([0, 0, 3])
        nodes = rng.choice([1, _logint(rng, 2, 64 if branch else 4096)])
        B = _logint(rng, 1, max(1, min(256, 16384 // nodes)))
        c.update(B=B, ctx=_logint(rng, nodes, max(nodes, min(8192, 131072 // B))), nodes=nodes,
                 H=Hkv * rng.choice([1, 2, 3, 4]), bits=rng.choice([8, 8, 16]), branch=branch,
                 rot=rng.choice([c["d"], c["d"], c["d"] // 2, 16]), inter=rng.random() < 0.3)
    else:
        nodes = _logint(rng, 2, 64)
        c.update(B=_logint(rng, 1, 64), ctx=_logint(rng, 1, 1024), nodes=nodes,
                 take=rng.randint(1, min(8, nodes)), L=16)
        # layers: the pools' bytes stay below those of the largest listed pools
        tokens = c["B"] * (c["ctx"] + c["page"] + nodes)
        c["L"] = _logint(rng, 1, max(1, min(16, int((1 << 30) / (tokens * Hkv * c["d"] * 2)))))
    return c


# ------------------------------------------------------------------ inputs
def _dev():
    return torch.device("cuda", torch.cuda.current_device())


def _int(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=_dev())


def _gen(seed):
    g = torch.Generator(device=_dev())
    g.manual_seed(seed)
    return g


def _randn(seed, *shape):
    return torch.randn(*shape, generator=_gen(seed), device=_dev(), dtype=torch.bfloat16)


def _pool8(seed, pages, page, Hkv, d):
    """Codes and scales of tokens whose size differs from block to block by some e^(N(0,1) / 2), as a
    few pages at a time."""
    g, nb = _gen(seed), page // BLOCK
    codes = torch.empty(pages, page, Hkv, d, dtype=F8, device=_dev())
    scales = torch.empty(pages, Hkv, nb, dtype=torch.float32, device=_dev())
    step = max(1, (1 << 26) // (page * Hkv * d))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        size = torch.exp(0.5 * torch.randn(n, nb, 1, Hkv, 1, generator=g, device=_dev()))
        x = torch.randn(n, nb, BLOCK, Hkv, d, generator=g, device=_dev()) * size
        s = _scale_of(x.abs().amax((2, 4)))                              # [n, nb, Hkv]
        codes[p:p + n] = _code(x / s[:, :, None, :, None]).view(n, page, Hkv, d)
        scales[p:p + n] = s.transpose(1, 2)
    return codes, scales


def _lens(rng, B, ctx):
    """Ragged lengths spread evenly between half of ctx and ctx, in random order."""
    return rng.permutation(np.linspace((ctx + 1) // 2, ctx, B + 1).round().astype(np.int64)[1:])


def _tables(rng, lens, page, width, n_pages):
    """Page tables whose pages are spread over the pool at random; 0 past the end."""
    order = rng.permutation(n_pages)
    t = np.zeros((len(lens), width), np.int64)
    at = 0
    for b, u in enumerate(-(-lens // page)):
        t[b, :u] = order[at:at + u]
        at += u
    return t


def _tree(rng, n, real, branch):
    """Parents of a drafted tree of `real` nodes in order of depth, padded to n."""
    p = np.full(n, -2, np.int64)
    p[0] = -1
    for t in range(1, real):
        p[t] = max(0, (t - 1) // branch - int(rng.integers(0, 2)))
    return p


def prepare(case, seed):
    c = dict(case)
    rng = np.random.default_rng(seed)
    op, B, page, Hkv, d = c["op"], c["B"], c["page"], c["Hkv"], c["d"]
    s = dict(op=op, page=page)
    if op == "attend":
        n = c["nodes"]
        lens = _lens(rng, B, c["ctx"]) + n
        width = -(-(c["ctx"] + n) // page)
        n_pages = int((-(-lens // page)).sum()) + 3
        s.update(q=_randn(seed * 8 + 1, B * n, c["H"], d), lens=_int(lens), cu=_int(np.arange(B + 1) * n),
                 table=_int(_tables(rng, lens, page, width, n_pages)), nodes=n, longest=c["ctx"] + n,
                 scale=d ** -0.5, parents=None)
        s["k"], s["k_scale"] = _pool8(seed * 8 + 2, n_pages, page, Hkv, d)
        s["v"], s["v_scale"] = _pool8(seed * 8 + 3, n_pages, page, Hkv, d)
        if c["branch"]:
            real = rng.integers((n + 1) // 2, n + 1, size=B)
            s["parents"] = _int(np.concatenate([_tree(rng, n, int(r), c["branch"]) for r in real]))
    elif op == "append":
        n = c["nodes"]
        new = rng.permutation(np.linspace((n + 7) // 8, n, B + 1).round().astype(np.int64)[1:])
        lens = np.maximum(_lens(rng, B, c["ctx"]), new)
        width = -(-c["ctx"] // page)
        n_pages = B * width + 3
        cu = np.concatenate([[0], np.cumsum(new)])
        T = int(cu[-1])
        s.update(q=_randn(seed * 8 + 1, T, c["H"], d), new_k=_randn(seed * 8 + 2, T, Hkv, d),
                 new_v=_randn(seed * 8 + 3, T, Hkv, d), lens=_int(lens), cu=_int(cu), bits=c["bits"],
                 table=_int(_tables(rng, lens, page, width, n_pages)), inter=c["inter"], positions=None,
                 freqs=torch.tensor(10000.0 ** (-2.0 * np.arange(c["rot"] // 2) / c["rot"]),
                                    dtype=torch.float32, device=_dev()))
        if c["bits"] == 8:
            s["k"], s["k_scale"] = _pool8(seed * 8 + 4, n_pages, page, Hkv, d)
            s["v"], s["v_scale"] = _pool8(seed * 8 + 5, n_pages, page, Hkv, d)
        else:
            s["k"], s["v"] = (torch.zeros(n_pages, page, Hkv, d, dtype=torch.bfloat16, device=_dev())
                              for _ in range(2))
            s["k_scale"] = s["v_scale"] = None
        if c["branch"]:
            at = []
            for b in range(B):
                p, depth = _tree(rng, int(new[b]), int(new[b]), c["branch"]), []
                for t in range(len(p)):
                    depth.append(0 if p[t] < 0 else depth[p[t]] + 1)
                at += [int(lens[b] - new[b]) + x for x in depth]
            s["positions"] = _int(at)
    else:
        n, L = c["nodes"], c["L"]
        lens = _lens(rng, B, c["ctx"]) + n
        width = -(-(c["ctx"] + n) // page)
        n_pages = int((-(-lens // page)).sum()) + 3
        table = _tables(rng, lens, page, width, n_pages)
        take = rng.integers(1, c["take"] + 1, size=B)
        acc = np.zeros((B, c["take"]), np.int64)
        for b in range(B):
            # the accepted path: node 0, then nodes of growing index.  A moved
            # node lies past the accepted ones, so that a pass can be repeated
            # on the same pools.
            m = min(int(take[b]), n - int(take[b]) + 1)
            take[b] = m
            acc[b, 1:m] = np.sort(rng.choice(np.arange(m, n), size=m - 1, replace=False)) if m > 1 else 0
        for i, name in enumerate("kv"):
            x, y = _pool8(seed * 8 + 1 + i, L * n_pages, page, Hkv, d)
            s[name], s[name + "_scale"] = x.view(L, n_pages, page, Hkv, d), y.view(L, n_pages, Hkv, -1)
        s.update(table=_int(table), lens=_int(lens), cu=_int(np.arange(B + 1) * n), accept=_int(acc),
                 n_accept=_int(take), lens_out=_int(np.zeros(B)))
    return s


# ------------------------------------------------------------------ run
def run(s):
    op = s["op"]
    if own:
        import masked_attention_bound_gb300 as fm
        if op == "attend":
            return fm.tree_forward(s["q"], s["k"], s["v"], s["table"], s["lens"], s["cu"], s["scale"],
                                   parents=s["parents"], max_nodes=s["nodes"], k_scale=s["k_scale"],
                                   v_scale=s["v_scale"])
        if op == "append":
            q = fm.cache_append_rotary(s["q"], s["new_k"], s["new_v"], s["cu"], s["freqs"], s["k"], s["v"],
                                       s["table"], s["lens"], positions=s["positions"], interleaved=s["inter"],
                                       k_scale=s["k_scale"], v_scale=s["v_scale"])
            return q, s["k"], s["v"], s["k_scale"], s["v_scale"]
        fm.cache_accept(s["accept"], s["n_accept"], s["cu"], s["k"], s["v"], s["table"], s["lens"],
                        lens_out=s["lens_out"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return s["k"], s["v"], s["k_scale"], s["v_scale"], s["lens_out"]
    return {"attend": _plain_attend, "append": _plain_append, "accept": _plain_accept}[op](s)


def _scale_of(amax):
    """The least power of two that brings amax to 448 or less, within 2^LEAST and 2^MOST."""
    m, e = torch.frexp(amax)                                  # amax = m 2^e, m in [1/2, 1)
    e = torch.where(amax > 0, e - 9 + (m > 0.875), LEAST)
    return torch.ldexp(torch.ones_like(amax), e.clamp(LEAST, MOST))


def _code(x):
    """e4m3, to nearest, the largest ones for what is larger (NaN stays one)."""
    return x.clamp(-448, 448).to(F8)


def _take8(pool, *at):
    """Codes pool[at]."""
    return pool.view(torch.uint8)[at].view(F8)


def _put8(pool, codes, *at):
    pool.view(torch.uint8)[at] = codes.view(torch.uint8)


def _slots(table, pos, page):
    """(page, slot) of token positions pos [B, n] of each sequence."""
    return torch.gather(table.long(), 1, pos // page), pos % page


def _plain_attend(s):
    q, page, n, span = s["q"], s["page"], s["nodes"], s["longest"]
    T, H, d = q.shape
    B, Hkv = T // n, s["k"].shape[2]
    G = H // Hkv
    pos = torch.arange(span, device=q.device).expand(B, span)
    pg, sl = _slots(s["table"], pos, page)
    # values of the codes, [B, span, Hkv, d]
    k = _take8(s["k"], pg, sl).float() * s["k_scale"].transpose(1, 2)[pg, sl // BLOCK][..., None]
    v = _take8(s["v"], pg, sl).float() * s["v_scale"].transpose(1, 2)[pg, sl // BLOCK][..., None]
    j = pos - (s["lens"].long() - n)[:, None]                        # the key's node, < 0: context
    node = torch.arange(n, device=q.device)
    if s["parents"] is None:
        sees = (node[:, None] >= node[None, :]).expand(B, n, n)
    else:
        # ancestors: powers of the matrix that links each node to its parent and itself
        par = s["parents"].view(B, n).long()
        link = (par[:, :, None] == node).double() + torch.eye(n, device=q.device, dtype=torch.float64)
        sees = (torch.linalg.matrix_power(link, n) > 0) & (par != -2)[:, :, None]
    vis = torch.gather(sees, 2, j.clamp(0, n - 1)[:, None, :].expand(B, n, span))
    live = torch.ones(B, n, dtype=torch.bool, device=q.device) if s["parents"] is None else par != -2
    vis = torch.where(j[:, None, :] < 0, live[:, :, None], vis & (j < n)[:, None, :])
    qg = q.float().view(B, n, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, d)
    x = torch.matmul(qg, k.permute(0, 2, 3, 1)).view(B, Hkv, G, n, span) * s["scale"]
    x = torch.where(vis[:, None, None], x, -math.inf)
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    tot = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(B, Hkv, G * n, span), v.permute(0, 2, 1, 3)).view(B, Hkv, G, n, d)
    o = o / torch.where(tot > 0, tot, 1.0)
    lse = (m + torch.log(tot)).squeeze(-1)                           # log 0 = -inf
    o = o.permute(0, 3, 1, 2, 4).reshape(T, H, d).to(q.dtype)
    return o, lse.permute(1, 2, 0, 3).reshape(H, T)


def _rotated(x, cos, sin, inter):
    """x [T, heads, d] in fp32 with its first 2 n elements rotated, cos and sin [T, n]."""
    x, n = x.float(), cos.shape[1]
    a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if inter else (x[..., :n], x[..., n:2 * n])
    c, s = cos[:, None], sin[:, None]
    y = a * c - b * s, b * c + a * s
    y = torch.stack(y, -1).flatten(-2) if inter else torch.cat(y, -1)
    return torch.cat([y, x[..., 2 * n:]], -1)


def _append8(x, pool, scales, pg, sl):
    """Values x [T, Hkv, d] to pages pg, slots sl [T] of a pool of codes."""
    nb, dev = scales.shape[2], x.device
    blocks, of = torch.unique(pg * nb + sl // BLOCK, return_inverse=True)
    n, Hkv, d = blocks.numel(), x.shape[1], x.shape[2]
    top = torch.where(x.isfinite(), x.abs(), 0).amax(-1)                     # [T, Hkv]
    amax = torch.zeros(n, Hkv, device=dev).scatter_reduce_(0, of[:, None].expand_as(top), top, "amax")
    first = torch.full((n,), BLOCK, device=dev).scatter_reduce_(0, of, sl % BLOCK, "amin")
    bp, bb = blocks // nb, blocks % nb
    old = scales[bp, :, bb]
    need = _scale_of(amax)
    new = torch.where((first > 0)[:, None], torch.maximum(old, need), need)  # slot 0 begins a block
    scales[bp, :, bb] = new
    # where the scale of a block has grown its tokens keep their values
    rows = bb[:, None] * BLOCK + torch.arange(BLOCK, device=dev)             # [n, 16]
    there = _take8(pool, bp[:, None], rows)                                  # [n, 16, Hkv, d]
    grown = ((first > 0)[:, None] & (new > old))[:, None, :, None]
    moved = _code(there.float() * (old / new)[:, None, :, None])
    _put8(pool, torch.where(grown, moved.view(torch.uint8), there.view(torch.uint8)), bp[:, None], rows)
    _put8(pool, _code(x / new[of][..., None]), pg, sl)


def _plain_append(s):
    cu, lens, page = s["cu"].long(), s["lens"].long(), s["page"]
    i = torch.arange(s["new_k"].shape[0], device=cu.device)
    b = torch.searchsorted(cu[1:], i, right=True)
    place = lens[b] - cu[b + 1] + i
    pg, sl = s["table"].long()[b, place // page], place % page
    pos = place if s["positions"] is None else s["positions"].long()
    angle = pos[:, None].double() * s["freqs"].double()       # far positions: more than 32 bits hold
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    q = _rotated(s["q"], cos, sin, s["inter"]).to(s["q"].dtype)
    k = _rotated(s["new_k"], cos, sin, s["inter"])
    if s["bits"] == 8:
        _append8(k, s["k"], s["k_scale"], pg, sl)
        _append8(s["new_v"].float(), s["v"], s["v_scale"], pg, sl)
    else:
        s["k"][pg, sl] = k.to(s["k"].dtype)
        s["v"][pg, sl] = s["new_v"]
    return q, s["k"], s["v"], s["k_scale"], s["v_scale"]


def _accept8(pool, scales, src, dst):
    """Tokens (page, slot) src to dst, both [N], in all layers of a pool of codes."""
    (sp, ss), (dp, ds), nb = src, dst, scales.shape[3]
    L, dev = pool.shape[0], pool.device
    sizes = scales[:, sp, :, ss // BLOCK].movedim(0, 1)                      # [L, N, Hkv]
    values = _take8(pool, slice(None), sp, ss).float() * sizes[..., None]
    blocks, of = torch.unique(dp * nb + ds // BLOCK, return_inverse=True)
    bp, bb = blocks // nb, blocks % nb
    old = scales[:, bp, :, bb].movedim(0, 1)                                 # [L, n, Hkv]
    new = old.scatter_reduce(1, of[None, :, None].expand_as(sizes), sizes, "amax")
    rows = bb[:, None] * BLOCK + torch.arange(BLOCK, device=dev)
    there = _take8(pool, slice(None), bp[:, None], rows)                     # [L, n, 16, Hkv, d]
    _put8(pool, _code(there.float() * (old / new)[:, :, None, :, None]), slice(None), bp[:, None], rows)
    _put8(pool, _code(values / new[:, of][..., None]), slice(None), dp, ds)
    scales[:, bp, :, bb] = new.movedim(1, 0)


def _plain_accept(s):
    cu, acc = s["cu"].long(), s["accept"].long()
    base = s["lens"].long() - (cu[1:] - cu[:-1])
    step = torch.arange(acc.shape[1], device=acc.device)
    use = step < s["n_accept"][:, None]
    src = _slots(s["table"], base[:, None] + torch.where(use, acc, 0), s["page"])
    dst = _slots(s["table"], base[:, None] + step, s["page"])
    src, dst = tuple(x[use] for x in src), tuple(x[use] for x in dst)
    _accept8(s["k"], s["k_scale"], src, dst)
    _accept8(s["v"], s["v_scale"], src, dst)
    s["lens_out"].copy_(base + s["n_accept"])
    return s["k"], s["v"], s["k_scale"], s["v_scale"], s["lens_out"]


# ------------------------------------------------------------------ work
def work(case):
    c = case
    op, B, Hkv, d, page = c["op"], c["B"], c["Hkv"], c["d"], c["page"]
    token = Hkv * 2 * (d + 4 / BLOCK)           # K and V of one token of one layer: codes and its share of a scale
    if op == "attend":
        n, H = c["nodes"], c["H"]
        rows = B * n * (0.75 if c["branch"] else 1.0)
        keys = 0.75 * c["ctx"] + n
        return dict(bytes=B * keys * token + B * n * H * (4 * d + 4) + 4 * B * keys / page,
                    flops=4.0 * rows * H * d * (0.75 * c["ctx"] + n / 2))
    if op == "append":
        new = np.linspace((c["nodes"] + 7) // 8, c["nodes"], B + 1).round()[1:].sum()
        cached = token if c["bits"] == 8 else Hkv * d * 4
        return dict(bytes=float(new * (4 * c["H"] * d + 4 * Hkv * d + cached)),
                    flops=float(3 * new * (c["H"] + Hkv) * c["rot"]))
    return dict(bytes=2.0 * B * (c["take"] - 1) / 2 * c["L"] * token + 4.0 * B * (c["take"] + 3), flops=0.0)


# ------------------------------------------------------------------ exact results
def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": _exact_attend, "append": _exact_append, "accept": _exact_accept}[case["op"]](s)


def _host(t):
    return t.cpu().numpy().astype(np.int64)


def _exact_attend(s):
    """softmax over each row's visible keys, in float64, one sequence and K/V head at a time."""
    q, n, page = s["q"], s["nodes"], s["page"]
    T, H, d = q.shape
    Hkv = s["k"].shape[2]
    G = H // Hkv
    lens, table = _host(s["lens"]), s["table"].long()
    par = None if s["parents"] is None else _host(s["parents"])
    o = torch.zeros(T, H, d, dtype=torch.float64, device=q.device)
    lse = torch.full((H, T), -math.inf, dtype=torch.float64, device=q.device)
    for b in range(T // n):
        size = int(lens[b])
        pages = table[b, :-(-size // page)]
        see = np.zeros((n, size), bool)
        for t in range(n):
            if par is not None and par[b * n + t] == -2:
                continue
            see[t, :size - n] = True
            a = t
            while a >= 0:                       # itself and its ancestors
                see[t, size - n + a] = True
                a = a - 1 if par is None else int(par[b * n + a])
        rows = np.nonzero(see.any(1))[0]
        see = torch.from_numpy(see[rows]).to(q.device)
        rows = torch.from_numpy(rows).to(q.device) + b * n
        for h in range(Hkv):
            k, v = (x.view(torch.uint8)[pages, :, h].view(F8).double().view(-1, BLOCK, d)
                    * y[pages, h].double().view(-1, 1, 1) for x, y in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])))
            k, v = k.view(-1, d)[:size], v.view(-1, d)[:size]
            x = torch.einsum("tgc,sc->tgs", q[rows, h * G:(h + 1) * G].double(), k) * s["scale"]
            x = x.masked_fill(~see[:, None], -math.inf)
            lse[h * G:(h + 1) * G, rows] = torch.logsumexp(x, -1).T
            o[rows, h * G:(h + 1) * G] = torch.einsum("tgs,sc->tgc", torch.softmax(x, -1), v)
    return o, lse


def _nearest8(x):
    """The e4m3 value nearest to x (float64), the even one of two, as a float64."""
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6)))
    step = np.exp2(e - 3)
    return np.clip(np.round(x / step) * step, -448, 448)


def _exact_scale(amax):
    s = np.full(amax.shape, 2.0 ** LEAST)
    for e in range(LEAST, MOST):
        s = np.where(amax > 448 * 2.0 ** e, 2.0 ** (e + 1), s)
    return s


def _turned(x, pos, freqs, inter):
    """x [T, heads, d] rotated, as complex numbers in 128 bits."""
    x, n = x.double().cpu().numpy().copy(), len(freqs)
    at = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if inter else (slice(0, n), slice(n, 2 * n))
    z = (x[..., at[0]] + 1j * x[..., at[1]]) * np.exp(1j * (pos[:, None] * freqs))[:, None]
    x[..., at[0]], x[..., at[1]] = z.real, z.imag
    return x


def _exact_append(s):
    cu, lens, table, page = _host(s["cu"]), _host(s["lens"]), _host(s["table"]), s["page"]
    place = np.concatenate([np.arange(lens[b] - (cu[b + 1] - cu[b]), lens[b]) for b in range(len(lens))])
    pos = place if s["positions"] is None else _host(s["positions"])
    freqs = s["freqs"].double().cpu().numpy()
    q = _turned(s["q"], pos, freqs, s["inter"])
    k, v = _turned(s["new_k"], pos, freqs, s["inter"]), s["new_v"].double().cpu().numpy()
    out = [torch.from_numpy(q)]
    for x, pool, scales in ((k, s["k"], s["k_scale"]), (v, s["v"], s["v_scale"])):
        for b in range(len(lens)):
            at = int(lens[b] - (cu[b + 1] - cu[b]))
            i = int(cu[b])
            while i < cu[b + 1]:                # up to the end of the block at a time
                m = int(min(BLOCK - at % BLOCK, cu[b + 1] - i))
                pg, sl = int(table[b, at // page]), at % page
                if scales is None:
                    pool[pg, sl:sl + m] = torch.from_numpy(x[i:i + m]).to(pool)
                else:
                    j, first = sl // BLOCK, sl % BLOCK
                    there = pool[pg, j * BLOCK:(j + 1) * BLOCK]
                    old = scales[pg, :, j].double().cpu().numpy()
                    new = _exact_scale(np.abs(x[i:i + m]).max((0, 2)))
                    if first:
                        new = np.maximum(new, old)
                        y = _nearest8(there.double().cpu().numpy() * (old / new)[:, None])
                    else:
                        y = there.double().cpu().numpy()
                    y[first:first + m] = _nearest8(x[i:i + m] / new[:, None])
                    there.copy_(torch.from_numpy(y).to(F8))
                    scales[pg, :, j] = torch.from_numpy(new)
                i, at = i + m, at + m
        out.append(pool)
    return (*out, s["k_scale"], s["v_scale"])


def _exact_accept(s):
    cu, lens, table, page = _host(s["cu"]), _host(s["lens"]), _host(s["table"]), s["page"]
    acc, take, out = _host(s["accept"]), _host(s["n_accept"]), []
    for b in range(len(lens)):
        base = int(lens[b] - (cu[b + 1] - cu[b]))
        first, last = base // BLOCK, (int(lens[b]) - 1) // BLOCK
        # the blocks of the tree, token by token, [L, tokens, Hkv, d] and [L, blocks, Hkv]
        at = np.arange(first, last + 1) * BLOCK
        pg, sl = torch.from_numpy(table[b, at // page]), at % page
        for pool, scales in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])):
            codes = [pool[:, p, x:x + BLOCK].double().cpu().numpy() for p, x in zip(pg, sl)]
            sizes = [scales[:, p, :, x // BLOCK].double().cpu().numpy() for p, x in zip(pg, sl)]
            new = [x.copy() for x in sizes]
            moves = [(base + int(acc[b, i]) - first * BLOCK, base + i - first * BLOCK) for i in range(int(take[b]))]
            for x, y in moves:
                new[y // BLOCK] = np.maximum(new[y // BLOCK], sizes[x // BLOCK])
            for j in sorted({y // BLOCK for _, y in moves}):
                y = _nearest8(codes[j] * (sizes[j] / new[j])[:, None, :, None])
                for x, to in moves:
                    if to // BLOCK == j:
                        ratio = sizes[x // BLOCK] / new[j]
                        y[:, to % BLOCK] = _nearest8(codes[x // BLOCK][:, x % BLOCK] * ratio[..., None])
                pool[:, pg[j], sl[j]:sl[j] + BLOCK] = torch.from_numpy(y).to(pool.device).to(F8)
                scales[:, pg[j], :, sl[j] // BLOCK] = torch.from_numpy(new[j]).to(scales)
        out.append(base + int(take[b]))
    return s["k"], s["v"], s["k_scale"], s["v_scale"], _int(out)
