"""Cases, plain forms and exact results of the paged-cache operators.

Operators: attention of a tree of drafted tokens (a single token or a causal
run of tokens being trees without branches) over a paged K/V cache; appending
new tokens' K/V to the cache; moving the accepted nodes of a tree together
after verification; forking, freeing and growing the sequences of a cache
(with copies of shared last pages); compacting the pages of a pool.

``own`` selects what ``run`` executes: the plain forms in elementary torch
operations, or this package's calls.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

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
        # a decoding step's K/V of one layer
        dict(name="append decode batch", op="append", B=128, ctx=8192, nodes=1, Hkv=8, d=128,
             page=64),
        # a packed batch of prompts of 16K tokens in all (U[512, 4096] each, as in the varlen workload)
        dict(name="append prompts", op="append", B=7, ctx=4096, nodes=4096, Hkv=16, d=128, page=16),
        # after the verification of one tree, a small model
        dict(name="accept one tree", op="accept", B=1, ctx=1000, nodes=32, take=6, L=4, Hkv=2,
             d=64, page=16),
        # after the verification of a batch, all layers of a model at once
        dict(name="accept batch", op="accept", B=64, ctx=1024, nodes=64, take=8, L=16, Hkv=8,
             d=128, page=16),
        # a step of a small beam search: rows reordered, last pages copied
        dict(name="branch beams", op="branch", B=8, ctx=500, grow=1, L=4, Hkv=2, d=64, page=16),
        # a large batch of beams and samples, some sequences ending, all layers
        dict(name="branch batch", op="branch", B=256, ctx=500, grow=4, L=8, Hkv=8, d=128, page=16),
        # a small pool
        dict(name="compact small pool", op="compact", B=4, ctx=1000, holes=0.3, L=4, Hkv=2, d=64,
             page=16),
        # a pool half of whose pages are free after many requests ended
        dict(name="compact pool", op="compact", B=64, ctx=1000, holes=0.5, L=8, Hkv=8, d=128,
             page=32),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "accept", "branch", "compact"])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    c = dict(op=op, Hkv=Hkv, d=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]))
    if op == "attend":
        H = Hkv * rng.choice([1, 2, 3, 4, 5, 7, 8])
        B = _logint(rng, 1, 128)
        # the K/V of the cache stays below that of the largest listed case
        most = (1 << 32) // (B * Hkv * c["d"] * 4)
        c.update(B=B, ctx=_logint(rng, 1, min(131072, most)), H=H)
        branch = rng.choice([0, 0, 2, 3, 8])
        nodes = 1 if branch == 0 and rng.random() < 0.5 else _logint(rng, 2, 64)
        # as many score products as the largest listed case has, at most
        nodes = max(1, min(nodes, (1 << 29) // (B * H * c["ctx"])))
        c.update(nodes=nodes, branch=branch)
    elif op == "append":
        nodes = rng.choice([1, _logint(rng, 2, 4096)])
        B = _logint(rng, 1, max(1, min(256, 16384 // nodes)))
        c.update(B=B, ctx=_logint(rng, nodes, max(nodes, min(8192, 131072 // B))), nodes=nodes)
    elif op == "accept":
        nodes = _logint(rng, 2, 64)
        c.update(B=_logint(rng, 1, 64), ctx=_logint(rng, 1, 1024), nodes=nodes,
                 take=rng.randint(1, min(8, nodes)), L=16)
    elif op == "branch":
        c.update(B=_logint(rng, 2, 256), ctx=_logint(rng, 1, 500), grow=rng.choice([1, 1, 4, 17]), L=8)
    else:
        c.update(B=_logint(rng, 1, 64), ctx=_logint(rng, 16, 1000), holes=rng.choice([0.1, 0.3, 0.5]),
                 L=8)
    if "L" in c:
        # layers: the pools' bytes stay below those of the largest listed pools
        tokens = c["B"] * (c["ctx"] + c["page"] + c.get("nodes", 0) + c.get("grow", 0)) / (1 - c.get("holes", 0))
        c["L"] = _logint(rng, 1, max(1, min(c["L"], int((1 << 31) / (tokens * Hkv * c["d"] * 4)))))
    return c


# ------------------------------------------------------------------ inputs
def _dev():
    return torch.device("cuda", torch.cuda.current_device())


def _int(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=_dev())


def _randn(seed, *shape):
    g = torch.Generator(device=_dev())
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device=_dev(), dtype=torch.bfloat16)


def _lens(rng, B, ctx):
    """Ragged lengths spread evenly between half of ctx and ctx, in random order."""
    return rng.permutation(np.linspace((ctx + 1) // 2, ctx, B + 1).round().astype(np.int64)[1:])


def _tables(rng, lens, page, width, n_pages):
    """Page tables whose pages are spread over the pool at random; -1 past the end."""
    used = -(-lens // page)
    order = rng.permutation(n_pages)
    t = np.full((len(lens), width), -1, np.int64)
    at = 0
    for b, u in enumerate(used):
        t[b, :u] = order[at:at + u]
        at += u
    return t, order[at:]


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
        table, _ = _tables(rng, lens, page, width, n_pages)
        table[table < 0] = 0
        s.update(q=_randn(seed * 4 + 1, B * n, c["H"], d), k=_randn(seed * 4 + 2, n_pages, page, Hkv, d),
                 v=_randn(seed * 4 + 3, n_pages, page, Hkv, d), table=_int(table), lens=_int(lens),
                 cu=_int(np.arange(B + 1) * n), nodes=n, longest=c["ctx"] + n, scale=d ** -0.5)
        s["parents"] = None
        if c["branch"]:
            real = rng.integers((n + 1) // 2, n + 1, size=B)
            s["parents"] = _int(np.concatenate([_tree(rng, n, int(r), c["branch"]) for r in real]))
    elif op == "append":
        n = c["nodes"]
        new = rng.permutation(np.linspace((n + 7) // 8, n, B + 1).round().astype(np.int64)[1:])
        lens = np.maximum(_lens(rng, B, c["ctx"]), new)
        width = -(-c["ctx"] // page)
        n_pages = B * width + 3
        table, _ = _tables(rng, lens, page, width, n_pages)
        cu = np.concatenate([[0], np.cumsum(new)])
        s.update(new_k=_randn(seed * 4 + 1, int(cu[-1]), Hkv, d), new_v=_randn(seed * 4 + 2, int(cu[-1]), Hkv, d),
                 k=torch.zeros(n_pages, page, Hkv, d, dtype=torch.bfloat16, device=_dev()),
                 v=torch.zeros(n_pages, page, Hkv, d, dtype=torch.bfloat16, device=_dev()),
                 table=_int(table), lens=_int(lens), cu=_int(cu))
    elif op == "accept":
        n, L = c["nodes"], c["L"]
        lens = _lens(rng, B, c["ctx"]) + n
        width = -(-(c["ctx"] + n) // page)
        n_pages = int((-(-lens // page)).sum()) + 3
        table, _ = _tables(rng, lens, page, width, n_pages)
        take = rng.integers(1, c["take"] + 1, size=B)
        acc = np.zeros((B, c["take"]), np.int64)
        for b in range(B):
            # the accepted path: node 0, then nodes of growing index.  A moved
            # node lies past the accepted ones, so that a pass can be repeated
            # on the same pools.
            m = min(int(take[b]), n - int(take[b]) + 1)
            take[b] = m
            acc[b, 1:m] = np.sort(rng.choice(np.arange(m, n), size=m - 1, replace=False)) if m > 1 else 0
        s.update(k=_randn(seed * 4 + 1, L, n_pages, page, Hkv, d), v=_randn(seed * 4 + 2, L, n_pages, page, Hkv, d),
                 table=_int(table), lens=_int(lens), cu=_int(np.arange(B + 1) * n), accept=_int(acc),
                 n_accept=_int(take), lens_out=_int(np.zeros(B)))
    elif op == "branch":
        L = c["L"]
        lens = _lens(rng, B, c["ctx"])
        width = -(-(c["ctx"] + c["grow"]) // page) + 1
        own_pages = int((-(-lens // page)).sum())
        n_pages = own_pages + B * (2 + c["grow"] // page) + 5
        table, _ = _tables(rng, lens, page, width, n_pages)
        ref = np.zeros(n_pages, np.int64)
        ref[table[table >= 0]] = 1
        # groups of four beams choose among themselves; one row in sixteen ends
        parent = np.minimum((np.arange(B) // 4) * 4 + rng.integers(0, 4, size=B), B - 1)
        parent[rng.random(B) < 1 / 16] = -1
        s.update(k=_randn(seed * 4 + 1, L, n_pages, page, Hkv, d), v=_randn(seed * 4 + 2, L, n_pages, page, Hkv, d),
                 table=_int(table), lens=_int(lens), ref=_int(ref), parent=_int(parent),
                 grow=_int(np.where(parent >= 0, c["grow"], 0)))
        for name in ("table_fork", "table_out"):
            s[name] = torch.full_like(s["table"], -1)
        for name in ("lens_fork", "lens_out"):
            s[name] = torch.zeros_like(s["lens"])
        for name in ("ref_fork", "ref_out"):
            s[name] = torch.zeros_like(s["ref"])
    else:
        L = c["L"]
        lens = _lens(rng, B, c["ctx"])
        width = -(-c["ctx"] // page)
        live = int((-(-lens // page)).sum())
        n_pages = int(live / (1 - c["holes"])) + 1
        table, _ = _tables(rng, lens, page, width, n_pages)
        ref = np.zeros(n_pages, np.int64)
        ref[table[table >= 0]] = 1
        s.update(k=_randn(seed * 4 + 1, L, n_pages, page, Hkv, d), v=_randn(seed * 4 + 2, L, n_pages, page, Hkv, d),
                 table=_int(table), lens=_int(lens), ref=_int(ref))
        s.update(table_out=torch.full_like(s["table"], -1), ref_out=torch.zeros_like(s["ref"]))
    return s


# ------------------------------------------------------------------ run
def run(s):
    op = s["op"]
    if own:
        import masked_attention_bound_gb300 as fm
        if op == "attend":
            return fm.tree_forward(s["q"], s["k"], s["v"], s["table"], s["lens"], s["cu"], s["scale"],
                                   parents=s["parents"], max_nodes=s["nodes"])
        if op == "append":
            fm.cache_append(s["new_k"], s["new_v"], s["cu"], s["k"], s["v"], s["table"], s["lens"])
            return s["k"], s["v"]
        if op == "accept":
            fm.cache_accept(s["accept"], s["n_accept"], s["cu"], s["k"], s["v"], s["table"], s["lens"],
                            lens_out=s["lens_out"])
            return s["k"], s["v"], s["lens_out"]
        if op == "branch":
            fm.pages_fork(s["parent"], s["page"], s["table"], s["lens"], s["ref"], s["table_fork"],
                          s["lens_fork"], s["ref_fork"])
            info = fm.pages_reserve(s["grow"], s["k"], s["v"], s["table_fork"], s["lens_fork"],
                                    s["ref_fork"], s["table_out"], s["lens_out"], s["ref_out"])
            return s["k"], s["v"], s["table_out"], s["lens_out"], s["ref_out"], info
        n_live = fm.pages_compact(s["k"], s["v"], s["table"], s["lens"], s["ref"], s["table_out"],
                                  s["ref_out"])
        return s["k"], s["v"], s["table_out"], s["ref_out"], n_live
    return {"attend": _plain_attend, "append": _plain_append, "accept": _plain_accept,
            "branch": _plain_branch, "compact": _plain_compact}[op](s)


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
    k, v = s["k"][pg, sl].float(), s["v"][pg, sl].float()           # [B, span, Hkv, d]
    j = pos - (s["lens"].long() - n)[:, None]                        # the key's node, < 0: context
    node = torch.arange(n, device=q.device)
    if s["parents"] is None:
        sees = node[None, :, None] >= node[None, None, :]
        sees = sees.expand(B, n, n)
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


def _plain_append(s):
    cu, lens = s["cu"].long(), s["lens"].long()
    T = s["new_k"].shape[0]
    i = torch.arange(T, device=cu.device)
    b = torch.searchsorted(cu[1:], i, right=True)
    pos = lens[b] - cu[b + 1] + i
    pg = s["table"].long()[b, pos // s["page"]]
    s["k"][pg, pos % s["page"]] = s["new_k"]
    s["v"][pg, pos % s["page"]] = s["new_v"]
    return s["k"], s["v"]


def _plain_accept(s):
    cu, acc = s["cu"].long(), s["accept"].long()
    base = s["lens"].long() - (cu[1:] - cu[:-1])
    step = torch.arange(acc.shape[1], device=acc.device)
    use = step < s["n_accept"][:, None]
    # places past the accepted ones repeat the first one, which stays where it is
    src = base[:, None] + torch.where(use, acc, 0)
    dst = base[:, None] + torch.where(use, step, 0)
    sp, ss = _slots(s["table"], src, s["page"])
    dp, ds = _slots(s["table"], dst, s["page"])
    s["k"][:, dp, ds] = s["k"][:, sp, ss]
    s["v"][:, dp, ds] = s["v"][:, sp, ss]
    s["lens_out"].copy_(base + s["n_accept"])
    return s["k"], s["v"], s["lens_out"]


def _plain_branch(s):
    page, parent = s["page"], s["parent"].long()
    table, lens, ref = s["table"].long(), s["lens"].long(), s["ref"].long()
    B, width = table.shape
    j = torch.arange(width, device=table.device)
    # fork
    keep = parent >= 0
    row = parent.clamp(min=0)
    old_used = j < ((lens + page - 1) // page)[:, None]
    lens1 = torch.where(keep, lens[row], 0)
    have = (lens1 + page - 1) // page
    used = j < have[:, None]
    table1 = torch.where(used, table[row], -1)
    ref1 = ref.scatter_add(0, table1.clamp(min=0).view(-1), used.long().view(-1))
    ref1 = ref1.scatter_add(0, table.clamp(min=0).view(-1), -old_used.long().view(-1))
    # reserve
    grow = s["grow"].long()
    lens2 = lens1 + grow
    last = torch.gather(table1, 1, (have - 1).clamp(min=0)[:, None]).squeeze(1)
    copy = (grow > 0) & (lens1 % page != 0) & (ref1[last.clamp(min=0)] > 1)
    need = (lens2 + page - 1) // page - have
    ends = torch.cumsum(need + copy.long(), 0)
    first = ends - need - copy.long()
    order = torch.argsort((ref1 != 0).int(), stable=True)
    n_free = (ref1 == 0).sum()
    ok = (ends[-1] <= n_free) & (lens2.amax() <= width * page)
    take = j - have[:, None] + (first + copy.long())[:, None]
    fresh = (j >= have[:, None]) & (j < (have + need)[:, None])
    swap = copy[:, None] & (j == (have - 1)[:, None])
    pick = torch.where(swap, first[:, None], take)
    new = (fresh | swap) & ok
    got = order[pick.clamp(0, order.numel() - 1)]
    table2 = torch.where(new, got, table1)
    ref2 = ref1.scatter_add(0, torch.where(new, got, 0).view(-1), new.long().view(-1))
    ref2 = ref2.scatter_add(0, last.clamp(min=0), -(copy & ok).long())
    # the tokens so far of the shared last pages
    b = torch.nonzero(copy & ok).squeeze(1)
    src, dst = last[b], torch.gather(table2, 1, (have - 1).clamp(min=0)[:, None]).squeeze(1)[b]
    fill = (torch.arange(page, device=table.device) < (lens1 % page)[b, None])[None, :, :, None, None]
    s["k"][:, dst] = torch.where(fill, s["k"][:, src], s["k"][:, dst])
    s["v"][:, dst] = torch.where(fill, s["v"][:, src], s["v"][:, dst])
    lens2 = torch.where(ok, lens2, lens1)
    s["table_out"].copy_(torch.where(j < ((lens2 + page - 1) // page)[:, None], table2, s["table_out"]))
    s["lens_out"].copy_(lens2)
    s["ref_out"].copy_(ref2)
    info = torch.stack([(ref2 == 0).sum(), ends[-1]]).int()
    return s["k"], s["v"], s["table_out"], s["lens_out"], s["ref_out"], info


def _plain_compact(s):
    ref, table = s["ref"].long(), s["table"].long()
    live = ref != 0
    n_live = live.sum()
    at = torch.arange(ref.numel(), device=ref.device)
    # the k-th live page past the live count goes to the k-th free one below it
    src = torch.nonzero(live & (at >= n_live)).squeeze(1)
    dst = torch.nonzero(~live & (at < n_live)).squeeze(1)
    to = at.scatter(0, src, dst)
    s["k"][:, dst] = s["k"][:, src]
    s["v"][:, dst] = s["v"][:, src]
    used = torch.arange(table.shape[1], device=ref.device) < ((s["lens"].long() + s["page"] - 1) // s["page"])[:, None]
    s["table_out"].copy_(torch.where(used, to[table.clamp(min=0)], s["table_out"]))
    s["ref_out"].copy_(torch.where(at < n_live, ref.scatter(0, dst, ref[src]), 0))
    return s["k"], s["v"], s["table_out"], s["ref_out"], n_live.int().view(1)


# ------------------------------------------------------------------ work
def work(case):
    c = case
    op, B, Hkv, d, page = c["op"], c["B"], c["Hkv"], c["d"], c["page"]
    token = Hkv * d * 2 * 2                     # K and V of one token of one layer, bf16
    if op == "attend":
        n, H = c["nodes"], c["H"]
        rows = B * n * (0.75 if c["branch"] else 1.0)
        keys = 0.75 * c["ctx"] + n
        return dict(bytes=B * keys * token + B * n * H * (4 * d + 4) + 4 * B * keys / page,
                    flops=4.0 * rows * H * d * (0.75 * c["ctx"] + n / 2))
    if op == "append":
        return dict(bytes=2.0 * B * 0.5625 * c["nodes"] * token, flops=0.0)
    if op == "accept":
        return dict(bytes=2.0 * B * (c["take"] - 1) / 2 * c["L"] * token + 4.0 * B * (c["take"] + 3), flops=0.0)
    tables = 4.0 * B * 0.75 * c["ctx"] / page
    if op == "branch":
        copies = B * 0.54 * (1 - 1 / page)      # rows whose last page another row shares
        pages = B * 0.75 * c["ctx"] / page + B
        return dict(bytes=2.0 * copies * page / 2 * c["L"] * token + 2 * tables + 8 * pages + 16 * B, flops=0.0)
    moved = B * 0.75 * c["ctx"] * c["holes"]
    return dict(bytes=2.0 * moved * c["L"] * token + 2 * tables + 8.0 * B * 0.75 * c["ctx"] / page / (1 - c["holes"]),
                flops=0.0)


# ------------------------------------------------------------------ exact results
def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": _exact_attend, "append": _exact_append, "accept": _exact_accept,
            "branch": _exact_branch, "compact": _exact_compact}[case["op"]](s)


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
            k = s["k"][pages, :, h].reshape(-1, d)[:size].double()
            v = s["v"][pages, :, h].reshape(-1, d)[:size].double()
            x = torch.einsum("tgc,sc->tgs", q[rows, h * G:(h + 1) * G].double(), k) * s["scale"]
            x = x.masked_fill(~see[:, None], -math.inf)
            lse[h * G:(h + 1) * G, rows] = torch.logsumexp(x, -1).T
            o[rows, h * G:(h + 1) * G] = torch.einsum("tgs,sc->tgc", torch.softmax(x, -1), v)
    return o, lse


def _exact_append(s):
    cu, lens, table, page = _host(s["cu"]), _host(s["lens"]), _host(s["table"]), s["page"]
    for b in range(len(lens)):
        at = int(lens[b] - (cu[b + 1] - cu[b]))
        i = int(cu[b])
        while i < cu[b + 1]:                    # up to the end of the page at a time
            m = int(min(page - at % page, cu[b + 1] - i))
            pg, sl = int(table[b, at // page]), at % page
            s["k"][pg, sl:sl + m] = s["new_k"][i:i + m]
            s["v"][pg, sl:sl + m] = s["new_v"][i:i + m]
            i, at = i + m, at + m
    return s["k"], s["v"]


def _exact_accept(s):
    cu, lens, table, page = _host(s["cu"]), _host(s["lens"]), _host(s["table"]), s["page"]
    acc, take, out = _host(s["accept"]), _host(s["n_accept"]), []
    for b in range(len(lens)):
        base = int(lens[b] - (cu[b + 1] - cu[b]))
        for i in range(int(take[b])):
            x, y = base + int(acc[b, i]), base + i
            for t in (s["k"], s["v"]):
                t[:, table[b, y // page], y % page] = t[:, table[b, x // page], x % page].clone()
        out.append(base + int(take[b]))
    return s["k"], s["v"], _int(out)


def _exact_branch(s):
    page = s["page"]
    table, lens, ref = _host(s["table"]), _host(s["lens"]), _host(s["ref"]).tolist()
    parent, grow = _host(s["parent"]), _host(s["grow"])
    rows = [table[p, :-(-int(lens[p]) // page)].tolist() if p >= 0 else [] for p in parent]
    size = [int(lens[p]) if p >= 0 else 0 for p in parent]
    for r in rows:
        for p in r:
            ref[p] += 1
    for b in range(len(lens)):
        for p in table[b, :-(-int(lens[b]) // page)]:
            ref[p] -= 1
    free = [p for p, r in enumerate(ref) if r == 0]
    was, asked = list(ref), 0
    for b, r in enumerate(rows):
        if grow[b] > 0 and size[b] % page and was[r[-1]] > 1:
            p, fill = free[asked], size[b] % page
            for t in (s["k"], s["v"]):
                t[:, p, :fill] = t[:, r[-1], :fill].clone()
            ref[r[-1]] -= 1
            ref[p] += 1
            r[-1] = p
            asked += 1
        size[b] += int(grow[b])
        while len(r) * page < size[b]:
            r.append(free[asked])
            ref[r[-1]] += 1
            asked += 1
    out = np.full(table.shape, -1)
    for b, r in enumerate(rows):
        out[b, :len(r)] = r
    return s["k"], s["v"], _int(out), _int(size), _int(ref), _int([ref.count(0), asked])


def _exact_compact(s):
    page = s["page"]
    table, lens, ref = _host(s["table"]), _host(s["lens"]), _host(s["ref"]).tolist()
    n_live = sum(r != 0 for r in ref)
    holes, to = [p for p in range(n_live) if ref[p] == 0], {}
    for p in range(n_live, len(ref)):
        if ref[p]:
            to[p] = holes[len(to)]
            ref[to[p]], ref[p] = ref[p], 0
            for t in (s["k"], s["v"]):
                t[:, to[p]] = t[:, p]
    out = np.full(table.shape, -1)
    for b in range(len(lens)):
        u = -(-int(lens[b]) // page)
        out[b, :u] = [to.get(int(p), int(p)) for p in table[b, :u]]
    return s["k"], s["v"], _int(out), _int(ref), _int([n_live])
