"""Appending, accepting, forking, reserving and compacting on the GPU, bit for bit
against the oracle."""
import numpy as np
import pytest
import torch

import masked_attention_bound_gb300 as fm
from cache_cases import LSE_TOL, Batch, ints, o_excess
from masked_attention_bound_gb300 import _abi
from oracle import cache as oc

pytestmark = pytest.mark.gpu


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _bits(t):
    return t.view(torch.int16).cpu().numpy()


def _pools(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return [torch.randint(-32768, 32767, shape, generator=g, dtype=torch.int16).cuda().view(torch.bfloat16)
            for _ in range(2)]


# ------------------------------------------------------------------ append, accept
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("Hkv,d,nodes", [(1, 64, [1, 1, 1]), (2, 128, [3, 0, 200, 1]), (3, 64, [17, 16, 15]),
                                         (16, 128, [1, 130]), (8, 128, [700])])
def test_append(page, Hkv, d, nodes):
    lens = [n + 5 * i for i, n in enumerate(nodes)]
    b = Batch(1, lens, nodes, Hkv, Hkv, d, page)
    T = sum(nodes)
    wide = _pools(2, T + 3, Hkv + 2, d + 8)
    k, v = (x[:, 1:1 + Hkv, :d] for x in wide)          # rows past cu[B] are not read
    want = [oc.append(_bits(x.contiguous()), b.cu_np, _bits(p), b.table_np, lens) for x, p in ((k, b.k), (v, b.v))]
    st = _status()
    fm.cache_append(k, v, b.cu, b.k, b.v, b.table, b.lens_t, status=st)
    assert fm.device_status(st) == 0
    assert np.array_equal(_bits(b.k), want[0]) and np.array_equal(_bits(b.v), want[1])


@pytest.mark.parametrize("B", [31, 33, 1025, 2500])
@pytest.mark.parametrize("Hkv,d", [(1, 64), (8, 128)])
def test_append_to_many_sequences(B, Hkv, d):
    """The search for a token's sequence: none, one or some new tokens each, in runs."""
    nodes = [(0, 1, 0, 0, 3, 1, 1)[(i * i) % 7] for i in range(B)]
    lens = [n + i % 20 for i, n in enumerate(nodes)]
    b = Batch(13, lens, nodes, Hkv, Hkv, d, 16)
    k, v = _pools(14, sum(nodes), Hkv, d)
    want = [oc.append(_bits(x), b.cu_np, _bits(p), b.table_np, lens) for x, p in ((k, b.k), (v, b.v))]
    st = _status()
    fm.cache_append(k, v, b.cu, b.k, b.v, b.table, b.lens_t, status=st)
    assert fm.device_status(st) == 0
    assert np.array_equal(_bits(b.k), want[0]) and np.array_equal(_bits(b.v), want[1])


def test_append_skips_what_is_out_of_range():
    b = Batch(3, [20, 20, 20], [2, 2, 2], 2, 2, 64, 16)
    k, v = _pools(4, 6, 2, 64)
    lens = b.lens_t.clone()
    lens[0] = 1
    b.table[2, 1] = b.k.shape[0]
    want = _bits(b.k).copy()
    for i in range(2):
        want[b.table_np[1, 1], 2 + i] = _bits(k)[2 + i]
    st = _status()
    fm.cache_append(k, v, b.cu, b.k, b.v, b.table, lens, status=st)
    assert fm.device_status(st) == _abi.FM_ERR_CACHE
    assert np.array_equal(_bits(b.k), want)


@pytest.mark.parametrize("Hkv,d,page,L", [(1, 64, 16, 1), (2, 128, 32, 3), (9, 128, 16, 2), (17, 64, 64, 1)])
def test_accept(Hkv, d, page, L):
    nodes, lens = [1, 5, 40, 0, 64], [1, 30, 140, 7, 64]
    b = Batch(5, lens, nodes, Hkv, Hkv, d, page)
    k, v = _pools(6, L, b.k.shape[0], page, Hkv, d)
    acc = [[0], [0, 1, 3, 4], sorted(b.rng.choice(40, 17, replace=False).tolist()), [], list(range(1, 64, 2))]
    arr = np.full((5, 40), 99)
    for i, a in enumerate(acc):
        arr[i, :len(a)] = a
    want = [oc.accept(acc, b.cu_np, _bits(p), b.table_np, lens) for p in (k, v)]
    st, ref = _status(), torch.full((b.k.shape[0],), 3, dtype=torch.int32, device="cuda")
    out = fm.cache_accept(ints(arr), ints([len(a) for a in acc]), b.cu, k, v, b.table, b.lens_t, ref=ref, status=st)
    assert fm.device_status(st) == 0 and out.tolist() == want[0][1]
    counts = [3] * b.k.shape[0]
    for i, x in enumerate(want[0][1]):
        for p in b.table_np[i, -(-x // page):-(-lens[i] // page)]:
            counts[p] = 2
    assert ref.tolist() == counts
    assert np.array_equal(_bits(k), want[0][0]) and np.array_equal(_bits(v), want[1][0])


@pytest.mark.parametrize("acc,count", [([3, 2], 2), ([1, 1], 2), ([0, 5], 2), ([-1, 2], 2), ([0, 1], 6), ([0, 1], -1)])
def test_accept_leaves_sequences_with_bad_lists(acc, count):
    b = Batch(7, [20, 25], [5, 5], 2, 2, 64, 16)
    k, v = _pools(8, 2, b.k.shape[0], 16, 2, 64)
    arr = np.zeros((2, 3))
    arr[0, :2], arr[1, :2] = acc, [2, 4]
    want, lens = oc.accept([[], [2, 4]], b.cu_np, _bits(k), b.table_np, [20, 25])
    st = _status()
    out = fm.cache_accept(ints(arr), ints([count, 2]), b.cu, k, v, b.table, b.lens_t, status=st)
    assert fm.device_status(st) == _abi.FM_ERR_CACHE
    assert out.tolist() == [20, lens[1]] and np.array_equal(_bits(k), want)


# ------------------------------------------------------------------ pages
class Pool:
    """Rows, counts and contents of a pool, on the GPU and as the oracle has them."""

    def __init__(self, seed, B, n_pages, page=16, L=2, Hkv=2, d=64, max_pages=12):
        self.rng = np.random.default_rng(seed)
        self.page, self.max_pages, self.B = page, max_pages, B
        self.rows, self.lens, self.ref = [[] for _ in range(B)], [0] * B, [0] * n_pages
        self.k, self.v = _pools(seed, L, n_pages, page, Hkv, d)
        self.kn, self.vn = _bits(self.k).copy(), _bits(self.v).copy()
        self.table = torch.full((B, max_pages), -7, dtype=torch.int32, device="cuda")
        self.lens_t, self.ref_t = ints(self.lens), ints(self.ref)

    def same(self):
        assert self.lens_t.tolist() == self.lens
        assert self.ref_t.tolist() == self.ref
        t = self.table.tolist()
        for b, r in enumerate(self.rows):
            assert t[b][:len(r)] == r, b
        assert np.array_equal(_bits(self.k), self.kn) and np.array_equal(_bits(self.v), self.vn)

    def fork(self, parent):
        self.rows, self.lens, self.ref = oc.fork(parent, self.rows, self.lens, self.ref)
        table = torch.full_like(self.table, -7)
        self.table, self.lens_t, self.ref_t = fm.pages_fork(ints(parent), self.page, self.table, self.lens_t,
                                                            self.ref_t, table_out=table)

    def reserve(self, grow, inplace=True):
        rows, lens, ref, copies, asked = oc.reserve(grow, self.rows, self.lens, self.ref, self.page, self.max_pages)
        for src, dst, n in copies or []:
            for p in (self.kn, self.vn):
                p[:, dst, :n] = p[:, src, :n]
        self.rows, self.lens, self.ref = rows, lens, ref
        st, out = _status(), {}
        if not inplace:
            old = (self.table.clone(), self.lens_t.clone(), self.ref_t.clone())
            out = dict(table_out=torch.full_like(self.table, -9), lens_out=torch.full_like(self.lens_t, -9),
                       ref_out=torch.full_like(self.ref_t, -9))
        info = fm.pages_reserve(ints(grow), self.k, self.v, self.table, self.lens_t, self.ref_t, status=st, **out)
        if not inplace:
            for x, y in zip(old, (self.table, self.lens_t, self.ref_t)):
                assert torch.equal(x, y)
            self.table, self.lens_t, self.ref_t = out.values()
        return info.tolist(), asked, copies is not None, fm.device_status(st)

    def compact(self, inplace=True):
        self.rows, self.ref, moves, live = oc.compact(self.rows, self.ref)
        for src, dst in moves:
            for p in (self.kn, self.vn):
                p[:, dst] = p[:, src]
        out = {} if inplace else dict(table_out=torch.full_like(self.table, -9), ref_out=torch.full_like(self.ref_t, -9))
        st = _status()
        n = fm.pages_compact(self.k, self.v, self.table, self.lens_t, self.ref_t, status=st, **out)
        if not inplace:
            self.table, self.ref_t = out.values()
        assert fm.device_status(st) == 0 and n.tolist() == [live]


@pytest.mark.parametrize("inplace", [True, False])
@pytest.mark.parametrize("seed,B,n_pages,page,L,Hkv,d", [(1, 6, 100, 16, 2, 2, 64), (2, 1, 7, 128, 1, 1, 128),
                                                         (3, 70, 1500, 16, 1, 3, 64), (4, 9, 333, 64, 3, 1, 64)])
def test_a_life_of_a_pool(inplace, seed, B, n_pages, page, L, Hkv, d):
    p = Pool(seed, B, n_pages, page, L, Hkv, d)
    short = 0
    for step in range(14):
        if step:
            p.fork([int(p.rng.integers(-1, B)) for _ in range(B)] if p.rng.random() < 0.7 else list(range(B)))
            p.same()
        grow = [int(p.rng.integers(0, 2 * page)) if p.rng.random() < 0.8 else 0 for _ in range(B)]
        info, asked, done, code = p.reserve(grow, inplace)
        p.same()
        assert info == [p.ref.count(0), asked]
        if done:
            assert code == 0
        else:
            short += 1
            assert code in (_abi.FM_ERR_PAGES, _abi.FM_ERR_CACHE)
        if p.rng.random() < 0.4:
            p.compact(inplace)
            p.same()
    assert short < 14


def test_reserve_with_exactly_the_free_pages_and_with_one_too_few():
    p = Pool(5, 3, 10)
    info, _, done, code = p.reserve([16 * 4, 16 * 4, 16 * 2])
    assert done and code == 0 and info == [0, 10]
    p.same()
    info, _, done, code = p.reserve([1, 0, 0])
    assert not done and code == _abi.FM_ERR_PAGES and info == [0, 1]
    p.same()
    p.fork([0, -1, 2])
    info, _, done, code = p.reserve([1, 0, 0])
    assert done and code == 0 and info == [3, 1]
    p.same()


def test_reserve_refuses_a_row_past_its_table_and_negative_growth():
    p = Pool(6, 2, 40)
    for grow in ([16 * 12 + 1, 1], [2 ** 31 - 1, 1], [-1, 1]):
        st = _status()
        info = fm.pages_reserve(ints(grow), p.k, p.v, p.table, p.lens_t, p.ref_t, status=st)
        assert fm.device_status(st) == _abi.FM_ERR_CACHE and info.tolist()[0] == 40
        p.same()


def test_many_pages_and_rows():
    """More pages than the plan's blocks take in one pass, more rows than a block has threads."""
    B, n = 9000, 100_000
    rng = np.random.default_rng(7)
    ref = (rng.random(n) < 0.5).astype(int)
    held = np.nonzero(ref)[0]
    rows = [[int(held[i])] if i < len(held) and i % 3 else [] for i in range(B)]
    ref[:] = 0
    for r in rows:
        for x in r:
            ref[x] = 1
    lens = [5 if r else 0 for r in rows]
    table = np.full((B, 3), -7)
    for b, r in enumerate(rows):
        table[b, :len(r)] = r
    grow = rng.integers(0, 32, B).tolist()
    k, v = _pools(8, 1, n, 16, 1, 64)
    t, ln, rf = ints(table), ints(lens), ints(ref)
    want = oc.reserve(grow, rows, lens, ref.tolist(), 16, 3)
    info = fm.pages_reserve(ints(grow), k, v, t, ln, rf)
    assert want[3] is not None and info.tolist() == [want[2].count(0), want[4]]
    assert ln.tolist() == want[1] and rf.tolist() == want[2]
    for b, r in enumerate(want[0]):
        assert t[b, :len(r)].tolist() == r if b % 50 == 0 else True
    flat = t.cpu().numpy()
    assert all(flat[b, :len(r)].tolist() == r for b, r in enumerate(want[0]))
    rows2, ref2, moves, live = oc.compact(want[0], want[2])
    kn = _bits(k).copy()
    for src, dst in moves:
        kn[:, dst] = kn[:, src]
    assert fm.pages_compact(k, v, t, ln, rf).tolist() == [live]
    assert rf.tolist() == ref2 and np.array_equal(_bits(k), kn)
    flat = t.cpu().numpy()
    assert all(flat[b, :len(r)].tolist() == r for b, r in enumerate(rows2))


@pytest.mark.parametrize("B,n_pages", [(1, 4), (40, 4096), (64, 700), (65, 700), (300, 9000)])
def test_fork_with_counts_of_its_own(B, n_pages):
    p = Pool(12, B, n_pages, L=1, Hkv=1, max_pages=4)
    p.reserve([int(x) for x in p.rng.integers(0, 50, B)])
    before = p.ref_t.clone()
    parent = [int(x) for x in p.rng.integers(-1, B, B)]
    want = oc.fork(parent, p.rows, p.lens, p.ref)
    out = torch.full_like(p.ref_t, -9)
    t, ln, rf = fm.pages_fork(ints(parent), 16, p.table, p.lens_t, p.ref_t, ref_out=out)
    assert rf.data_ptr() == out.data_ptr() and out.tolist() == want[2]
    assert ln.tolist() == want[1] and torch.equal(p.ref_t, before)
    assert all(t[b, :len(r)].tolist() == r for b, r in enumerate(want[0]))


def test_fork_reports_bad_rows():
    p = Pool(9, 3, 20)
    p.reserve([20, 20, 20])
    p.lens_t[1] = -1
    st = _status()
    t, ln, rf = fm.pages_fork(ints([0, 7, 1]), 16, p.table, p.lens_t, p.ref_t, status=st)
    assert fm.device_status(st) == _abi.FM_ERR_CACHE
    assert ln.tolist() == [20, 0, 0] and t[0, :2].tolist() == p.rows[0]


def test_compact_with_table_entries_out_of_range():
    p = Pool(10, 2, 20)
    p.reserve([40, 40])
    p.fork([-1, 1])
    p.table[1, 0] = 99
    st = _status()
    fm.pages_compact(p.k, p.v, p.table, p.lens_t, p.ref_t, status=st)
    assert fm.device_status(st) == _abi.FM_ERR_CACHE and p.table[1, 0].item() == 99


def test_captured_page_steps_replay():
    """A scheduler's step (fork, reserve, compact) captured once and replayed on new rows."""
    p = Pool(11, 8, 300, L=1)
    p.reserve([20] * 8)
    parent, grow = ints(list(range(8))), ints([0] * 8)
    tables = [p.table.clone(), torch.full_like(p.table, -7)]
    lens = [p.lens_t.clone(), torch.zeros_like(p.lens_t)]
    ws = fm.pages_workspace(p.k, p.v, p.table)
    info, n_live = ints([0, 0]), ints([0])

    def step():
        fm.pages_fork(parent, 16, tables[0], lens[0], p.ref_t, tables[1], lens[1])
        fm.pages_reserve(grow, p.k, p.v, tables[1], lens[1], p.ref_t, info=info, ws=ws)
        fm.pages_compact(p.k, p.v, tables[1], lens[1], p.ref_t, n_live=n_live, ws=ws)
        tables[0].copy_(tables[1])
        lens[0].copy_(lens[1])

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    p.rows, p.ref, moves, _ = oc.compact(p.rows, p.ref)
    for _ in range(6):
        par = [int(p.rng.integers(-1, 8)) for _ in range(8)]
        gr = [int(p.rng.integers(0, 15)) if x >= 0 else 0 for x in par]
        parent.copy_(ints(par))
        grow.copy_(ints(gr))
        graph.replay()
        torch.cuda.synchronize()
        p.rows, p.lens, p.ref = oc.fork(par, p.rows, p.lens, p.ref)
        p.rows, p.lens, p.ref, copies, _ = oc.reserve(gr, p.rows, p.lens, p.ref, 16, 12)
        assert copies is not None
        for src, dst, n in copies:
            p.kn[:, dst, :n] = p.kn[:, src, :n]
            p.vn[:, dst, :n] = p.vn[:, src, :n]
        p.rows, p.ref, moves, live = oc.compact(p.rows, p.ref)
        for src, dst in moves:
            p.kn[:, dst] = p.kn[:, src]
            p.vn[:, dst] = p.vn[:, src]
        assert n_live.tolist() == [live]
        p.table, p.lens_t = tables[0], lens[0]
        p.same()


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("H,Hkv,d,page", [(4, 2, 64, 16), (8, 2, 128, 32)])
def test_drafting_and_verifying_equals_decoding_token_by_token(H, Hkv, d, page):
    """The operators as a serving program runs them.  Two layers, a prompt, then steps of: room
    for a tree, its K/V appended, attention, acceptance of one path.  The cache then holds the
    context in order, and attention of the next token equals the oracle on the plain sequence."""
    rng = np.random.default_rng(12)
    g = torch.Generator().manual_seed(12)
    B, L, P, width = 3, 2, 200, 30
    rand = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)  # noqa: E731
    k = torch.full((L, P, page, Hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    v = torch.full_like(k, float("nan"))
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    lens, ref, st = ints([0] * B), ints([0] * P), _status()
    plain = [[([], []) for _ in range(B)] for _ in range(L)]     # K, V of every kept token
    prompt = [37, 1, 80]

    def feed(count, parents):
        cu = np.concatenate([[0], np.cumsum(count)])
        fm.pages_reserve(ints(count), k, v, table, lens, ref, status=st)
        new = [[rand(int(cu[-1]), Hkv, d) for _ in range(2)] for _ in range(L)]
        outs = []
        for layer in range(L):
            fm.cache_append(new[layer][0].cuda(), new[layer][1].cuda(), ints(cu), k[layer], v[layer], table, lens,
                            status=st)
            q = rand(int(cu[-1]), H, d).cuda()
            outs.append((q, *fm.tree_forward(q, k[layer], v[layer], table, lens, ints(cu), d ** -0.5,
                                             parents=parents, max_nodes=max(count), status=st)))
        return cu, new, outs

    def keep(cu, new, nodes):
        for layer in range(L):
            for b in range(B):
                for t in nodes[b]:
                    for i in range(2):
                        plain[layer][b][i].append(new[layer][i][cu[b] + t].float().numpy())

    cu, new, _ = feed(prompt, None)
    keep(cu, new, [range(n) for n in prompt])
    for _ in range(4):
        count = [int(rng.integers(4, 9)) for _ in range(B)]
        par = [[-1] + [int(rng.integers(0, t)) for t in range(1, n)] for n in count]
        cu, new, outs = feed(count, ints(sum(par, [])))
        for layer, (q, o, lse) in enumerate(outs):
            for b in range(B):
                kk, vv = (np.stack(x + [y.float().numpy() for y in new[layer][i][cu[b]:cu[b + 1]]]).astype(np.float64)
                          for i, x in enumerate(plain[layer][b]))
                see = oc.visible(count[b], len(kk) - count[b], par[b])
                rows = slice(cu[b], cu[b + 1])
                ro, rl, a = oc.tree_attention(q[rows].double().cpu().numpy(), kk, vv, see, d ** -0.5)
                assert o_excess(o[rows].double().cpu().numpy(), ro, a).max() <= 0
                assert np.abs(lse[:, rows].cpu().numpy() - rl).max() <= LSE_TOL
        path = [sorted(oc.ancestors(par[b], int(rng.integers(0, count[b])))) for b in range(B)]
        arr = np.zeros((B, 9))
        for b, x in enumerate(path):
            arr[b, :len(x)] = x
        lens = fm.cache_accept(ints(arr), ints([len(x) for x in path]), ints(cu), k, v, table, lens, ref=ref,
                               status=st)
        keep(cu, new, path)
        # the pages past the accepted tokens are free again
        want = [0] * P
        for b, x in enumerate(lens.tolist()):
            for p in table[b, :-(-x // page)].tolist():
                want[p] = 1
        assert ref.tolist() == want
    assert fm.device_status(st) == 0
    for b in range(B):
        n = int(lens[b])
        rows = table[b].cpu().numpy()
        for layer in range(L):
            for i, pool in enumerate((k, v)):
                got = oc.gather(pool[layer].float().cpu().numpy(), rows, n)
                assert np.array_equal(got, np.stack(plain[layer][b][i]))


@pytest.mark.parametrize("value", [-1, 1 << 23, "pages"])
@pytest.mark.parametrize("at", [2, 3, 4])
def test_accept_leaves_a_sequence_with_a_bad_page_to_release(at, value):
    """A page past the new length that is out of range: nothing of the sequence is moved or released."""
    b = Batch(14, [20 + 50, 25], [50, 5], 2, 2, 64, 16)
    k, v = _pools(15, 3, b.k.shape[0], 16, 2, 64)
    ref = torch.full((b.k.shape[0],), 3, dtype=torch.int32, device="cuda")
    b.table[0, at] = b.k.shape[0] if value == "pages" else value
    arr = np.zeros((2, 3))
    arr[0], arr[1, :2] = [1, 4, 8], [2, 4]       # row 0: tokens 21, 24 and 28, all in good pages
    want, lens = oc.accept([[], [2, 4]], b.cu_np, _bits(k), b.table_np, [70, 25])
    st = _status()
    out = fm.cache_accept(ints(arr), ints([3, 2]), b.cu, k, v, b.table, b.lens_t, ref=ref, status=st)
    assert fm.device_status(st) == _abi.FM_ERR_CACHE
    assert out.tolist() == [70, lens[1]] and np.array_equal(_bits(k), want)
    assert ref.tolist() == [3] * b.k.shape[0]


def test_tables_of_more_rows_than_32_bits_are_refused():
    table = torch.empty((1 << 32) + 2, 1, dtype=torch.int32, device="cuda")
    k, v = _pools(16, 4, 16, 1, 64)
    two, ref = ints([0, 0]), ints([1, 0, 0, 0])
    with pytest.raises(ValueError):
        fm.pages_fork(two, 16, table, two, ref, table_out=torch.empty_like(table), lens_out=ints([0, 0]))
    with pytest.raises(ValueError):
        fm.pages_reserve(two, k, v, table, two, ref)
    with pytest.raises(ValueError):
        fm.cache_append(k[0, :2], v[0, :2], ints([0, 1, 2]), k, v, table, ints([1, 1]))
    with pytest.raises(ValueError):
        fm.make_cache(k, v, table)
