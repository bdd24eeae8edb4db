"""Attention over the paged cache (fm_tree_fwd) against the fp64 oracle."""
import pytest
import torch

import masked_attention_bound_gb300 as fm
from cache_cases import Batch, ints, o_excess
from masked_attention_bound_gb300 import _abi

pytestmark = pytest.mark.gpu


def run(b, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = torch.full_like(b.q, float("nan"))
    lse = torch.full((b.H, b.q.shape[0]), float("nan"), dtype=torch.float32, device="cuda")
    kw.setdefault("max_nodes", max(b.nodes))
    fm.tree_forward(b.q, b.k, b.v, b.table, b.lens_t, b.cu, b.scale, parents=b.parents, o=o, lse=lse,
                    status=status, **kw)
    torch.cuda.synchronize()
    code = fm.device_status(status)
    return o, lse, code


# one token a sequence: lengths around page and tile ends, empty context
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(2, 2), (8, 1), (7, 1), (12, 4), (40, 2), (3, 1)])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_single_tokens(d, H, Hkv, page):
    lens = [1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 300, 1000]
    b = Batch(1, lens, [1] * len(lens), H, Hkv, d, page)
    o, lse, code = run(b)
    assert code == 0
    b.check(o, lse)


@pytest.mark.parametrize("kind", [None, "chain", "star", "random", "padded", "beams"])
@pytest.mark.parametrize("H,Hkv,d,page", [(2, 2, 64, 16), (8, 2, 128, 16), (6, 2, 128, 64), (5, 1, 64, 128),
                                          (16, 2, 128, 32)])
def test_trees(kind, H, Hkv, d, page):
    nodes = [1, 2, 5, 16, 17, 33, 64, 0, 3]
    lens = [1, 130, 5, 300, 128 + 17, 33, 190, 100, 259]
    b = Batch(2, lens, nodes, H, Hkv, d, page, kind)
    o, lse, code = run(b)
    assert code == 0
    b.check(o, lse)


@pytest.mark.parametrize("kind", [None, "random"])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (4, 1), (9, 3)])
def test_many_nodes(kind, H, Hkv):
    b = Batch(3, [256, 700, 513], [256, 200, 129], H, Hkv, 128, 16, kind)
    o, lse, code = run(b)
    assert code == 0
    b.check(o, lse)


@pytest.mark.parametrize("d", [64, 128])
def test_causal_run_longer_than_a_tree(d):
    b = Batch(4, [1500, 1000], [700, 1000], 4, 2, d, 64)
    o, lse, code = run(b)
    assert code == 0
    b.check(o, lse, rows=60)


@pytest.mark.parametrize("nodes", [1, 40])
def test_long_context_is_split_and_joined(nodes):
    b = Batch(5, [131072 - 7, 40000], [nodes] * 2, 8, 2, 128, 128, "random")
    o, lse, code = run(b)
    assert code == 0
    b.check(o, lse, rows=5)


def test_a_batch_with_empty_sequences_and_rows_behind_the_last():
    b = Batch(6, [0, 40, 0, 9, 0], [0, 3, 0, 1, 0], 4, 2, 64, 16)
    q = torch.randn(9, 4, 64, device="cuda").to(torch.bfloat16)
    q[:4] = b.q
    o = torch.full_like(q, 7.0)
    lse = torch.full((4, 9), 7.0, device="cuda")
    fm.tree_forward(q, b.k, b.v, b.table, b.lens_t, b.cu, b.scale, max_nodes=3, o=o, lse=lse)
    torch.cuda.synchronize()
    assert (o[4:] == 7).all() and (lse[:, 4:] == 7).all()
    b.check(o[:4], lse[:, :4])


def test_no_sequence_has_nodes():
    b = Batch(7, [5, 9], [1, 1], 2, 2, 64, 16)
    o = torch.full_like(b.q, 7.0)
    lse = torch.full((2, 2), 7.0, device="cuda")
    fm.tree_forward(b.q, b.k, b.v, b.table, b.lens_t, ints([0, 0, 0]), b.scale, o=o, lse=lse)
    torch.cuda.synchronize()
    assert (o == 7).all() and (lse == 7).all()


@pytest.mark.parametrize("nodes,H,Hkv", [(12, 2, 2), (30, 8, 2)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_values_not_finite_in_places_that_a_row_does_not_see(nodes, H, Hkv, bad):
    """NaN and infinities of a drafted node reach exactly the rows that see it; unused places of
    the pages hold NaN throughout (Batch's fill)."""
    b = Batch(8, [nodes + 100, nodes], [nodes, nodes], H, Hkv, 128, 16, "beams")
    clean, clean_lse, _ = run(b)
    node, ctx = 2, 100
    for seq, base in ((0, ctx), (1, 0)):
        p = base + node
        b.v[b.table_np[seq, p // 16], p % 16, :, 5] = bad
        b.v[b.table_np[seq, p // 16], p % 16, 0, 77] = bad
    p = ctx + nodes - 1                      # the last node's K: only its own rows
    b.k[b.table_np[0, p // 16], p % 16] = float("nan")
    o, lse, code = run(b)
    assert code == 0
    G = H // Hkv
    for seq in range(2):
        for t in range(nodes):
            a = t
            while a > node:
                a = b.parents_np[seq][a]
            row = b.cu_np[seq] + t
            if seq == 0 and t == nodes - 1:
                assert o[row].isnan().all() and lse[:, row].isnan().all()
                continue
            want = clean[row].clone()
            if a == node:
                want[:, 5] = bad
                want[:G, 77] = bad
            assert torch.equal(o[row].nan_to_num(nan=123.0), want.nan_to_num(nan=123.0)), (seq, t)
            assert torch.equal(lse[:, row], clean_lse[:, row])


def test_opposite_infinities_meet():
    b = Batch(9, [4], [4], 1, 1, 64, 16, "chain")
    b.v[b.table_np[0, 0], 1, 0, 3] = float("inf")
    b.v[b.table_np[0, 0], 2, 0, 3] = float("-inf")
    o, _, _ = run(b)
    x = o[:, 0, 3].float().cpu()
    assert x[0].isfinite() and x[1] == float("inf") and x[2].isnan() and x[3].isnan()


@pytest.mark.parametrize("nodes", [1, 20])
def test_values_not_finite_in_the_context_reach_every_row(nodes):
    b = Batch(10, [300], [nodes], 4, 1, 128, 32)
    b.v[b.table_np[0, 1], 4, 0, 9] = float("nan")
    o, lse, _ = run(b)
    assert o[:, :, 9].isnan().all() and not o[:, :, 10].isnan().any() and lse.isfinite().all()


def test_large_scores_and_queries_not_finite():
    b = Batch(11, [200, 50], [2, 1], 2, 1, 64, 16)
    clean, _, _ = run(b)
    b.q[1] = float("nan")
    o, lse, _ = run(b)
    assert o[1].isnan().all() and lse[:, 1].isnan().all()
    assert torch.equal(o[0], clean[0]) and torch.equal(o[2], clean[2])
    b.q.copy_(torch.randn(3, 2, 64).to(torch.bfloat16) * 300)     # scores of some thousands
    o, lse, _ = run(b)
    assert o.isfinite().all() and lse.isfinite().all()


@pytest.mark.parametrize("nodes", [1, 24])
def test_strides(nodes):
    """Heads before slots in the pools, pools inside larger tensors, q and o cut from larger ones."""
    b = Batch(12, [77, 260], [nodes] * 2, 6, 2, 128, 32)
    want, wlse, _ = run(b)
    n = b.k.shape[0]
    big = torch.full((n, 2, 4, 32, 136), float("nan"), dtype=torch.bfloat16, device="cuda")
    k, v = (big[:, i, 1:3].transpose(1, 2)[..., :128] for i in range(2))
    k.copy_(b.k)
    v.copy_(b.v)
    wide = torch.full((b.q.shape[0], 8, 3, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    q, o = wide[:, 1:7, 0], wide[:, 1:7, 2]
    q.copy_(b.q)
    lse = torch.empty_like(wlse)
    fm.tree_forward(q, k, v, b.table, b.lens_t, b.cu, b.scale, max_nodes=nodes, o=o, lse=lse)
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(lse, wlse)
    assert wide[:, :, 1].isnan().all() and wide[:, 0].isnan().all() and wide[:, 7].isnan().all()


@pytest.mark.parametrize("nodes", [1, 24])
def test_offsets_past_32_bits(nodes):
    """Pages whose elements lie more than 2^32 into the pool."""
    b = Batch(13, [300, 40], [nodes] * 2, 8, 2, 128, 64)
    want, wlse, _ = run(b)
    n = (1 << 32) // (64 * 2 * 128) + 40
    pools = [torch.empty(n, 64, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    m = b.k.shape[0]
    for big, small in zip(pools, (b.k, b.v)):
        big[n - m:] = small
    lse = torch.empty_like(wlse)
    o, lse = fm.tree_forward(b.q, *pools, b.table + (n - m), b.lens_t, b.cu, b.scale, max_nodes=nodes)
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(lse, wlse)


@pytest.mark.parametrize("nodes,kind", [(1, None), (24, "random")])
def test_bad_entries_are_reported_and_stay_in_bounds(nodes, kind):
    b = Batch(14, [100, 50, 200, 90], [nodes] * 4, 4, 2, 64, 16, kind)

    def same(o, lse, seqs):
        b.check(o, lse, seqs=seqs)      # the others' tiles are cut elsewhere: not the same bits

    for value in (nodes - 1, b.max_pages * 16 + 1, -5):
        b.lens_t[1] = value
        o, lse, code = run(b)
        assert code == _abi.FM_ERR_CACHE
        r = slice(b.cu_np[1], b.cu_np[2])
        assert (o[r] == 0).all() and (lse[:, r] == float("-inf")).all()
        same(o, lse, (0, 2, 3))
    b.lens_t[1] = 50
    for value in (-1, b.k.shape[0], 1 << 30):
        b.table[2, 1] = value
        o, lse, code = run(b)
        assert code == _abi.FM_ERR_CACHE and o.isfinite().all()
        same(o, lse, (0, 1, 3))
    b.table[2, 1] = int(b.table_np[2, 1])
    o, lse, code = run(b, max_nodes=nodes - 1) if nodes > 1 else (None, None, _abi.FM_ERR_CACHE)
    assert code == _abi.FM_ERR_CACHE and (o is None or (o == 0).all())
    if kind:
        b.parents[3] = 3
        b.parents[5] = -9
        o, lse, code = run(b)
        assert code == _abi.FM_ERR_CACHE
        same(o, lse, (1, 2, 3))
        b.parents[3], b.parents[5] = b.parents_np[0][3], b.parents_np[0][5]
    b.cu[2] = 10000
    o, lse, code = run(b)
    assert code == _abi.FM_ERR_CACHE
    same(o, lse, (0,))


@pytest.mark.parametrize("nodes", [1, 24])
def test_equal_inputs_give_equal_bits(nodes):
    b = Batch(15, [5000, 333, 12000, 77], [nodes] * 4, 8, 2, 128, 16, "random")
    first = run(b)
    for _ in range(5):
        o, lse, _ = run(b)
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])


@pytest.mark.parametrize("nodes", [1, 24])
def test_captured_and_replayed_with_growing_lengths(nodes):
    b = Batch(16, [600, 333], [nodes] * 2, 8, 2, 128, 16)
    ws = fm.tree_workspace(b.q, b.k, b.v, b.table, nodes)
    ws.fill_(255)
    o, lse = torch.empty_like(b.q), torch.empty(8, b.q.shape[0], device="cuda")
    lens = b.lens_t.clone()

    def call():
        fm.tree_forward(b.q, b.k, b.v, b.table, lens, b.cu, b.scale, max_nodes=nodes, o=o, lse=lse, ws=ws)

    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for short in (0, 100, 37, 300):
        lens.copy_(b.lens_t - short)
        o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        want, wlse = fm.tree_forward(b.q, b.k, b.v, b.table, lens, b.cu, b.scale, max_nodes=nodes)
        assert torch.equal(o, want) and torch.equal(lse, wlse)


def test_on_another_stream():
    b = Batch(17, [600, 4000], [4, 4], 8, 2, 128, 16)
    want, wlse, _ = run(b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = [fm.tree_forward(b.q, b.k, b.v, b.table, b.lens_t, b.cu, b.scale, max_nodes=4, stream=s)
            for _ in range(20)]
    junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(20)]   # on the current stream
    s.synchronize()
    for o, lse in outs:
        assert torch.equal(o, want) and torch.equal(lse, wlse)
    del junk


@pytest.mark.parametrize("nodes", [8, 64])
def test_max_nodes_only_chooses(nodes):
    """A looser bound gives the same rows, up to the rounding of another kernel's order."""
    b = Batch(18, [500, 130], [nodes, 3], 4, 2, 128, 32, "beams")
    for bound in (nodes, 100, 256, None):
        o, lse, code = run(b, max_nodes=bound)
        assert code == 0
        b.check(o, lse)


def test_excess_sees_a_wrong_row():
    """The comparison itself: a row that sees one key too many is past its bound."""
    b = Batch(19, [30], [4], 1, 1, 64, 16, "star")
    o, lse, _ = run(b)
    b.parents_np = [[-1, 0, -1, -1]]
    with pytest.raises(AssertionError):
        b.check(o, lse)
    assert o_excess(o.float().cpu().numpy(), o.float().cpu().numpy(), 0 * o.float().cpu().numpy()).max() <= 0


@pytest.mark.parametrize("nodes,d", [(1, 128), (1, 64), (16, 128), (16, 64), (50, 128)])
def test_a_wait_that_runs_out_is_reported_then_the_next_call_is_clean(nodes, d):
    """A hook withholds one release in each block (see fm_test_hooks): its wait runs out after 20 ms, and
    the call ends by itself with the status set; one for each kernel."""
    b = Batch(20, [2100] * 8, [nodes] * 8, 32, 8, d, 16, "random")
    ws = fm.tree_workspace(b.q, b.k, b.v, b.table, nodes)
    ws.zero_()
    assert fm.lib().fm_test_hooks(20_000_000, 8) == _abi.FM_OK
    try:
        _, _, code = run(b, max_nodes=nodes, ws=ws)
    finally:
        assert fm.lib().fm_test_hooks(0, 0) == _abi.FM_OK
    assert code == _abi.FM_ERR_TIMEOUT, _abi.status_string(code)
    o, lse, code = run(b, max_nodes=nodes, ws=ws)
    assert code == 0
    b.check(o, lse, rows=10)


@pytest.mark.parametrize("nodes", [1, 24, 70])
def test_two_calls_at_once(nodes):
    """Two streams, a workspace each (the default), the kernels in flight together."""
    b = Batch(21, [6000, 900, 3000], [nodes] * 3, 8, 2, 128, 16, "random")
    want = run(b)[:2]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for i in range(30):
        outs.append(fm.tree_forward(b.q, b.k, b.v, b.table, b.lens_t, b.cu, b.scale, parents=b.parents,
                                    max_nodes=nodes, stream=streams[i % 2]))
    torch.cuda.synchronize()
    for got in outs:
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_two_graphs_share_a_workspace():
    b = Batch(22, [3000, 700], [20, 20], 8, 2, 128, 16, "random")
    ws = fm.tree_workspace(b.q, b.k, b.v, b.table, 20)
    want = run(b)[:2]
    graphs, outs = [], []
    lens = [b.lens_t, b.lens_t.clone()]
    for i in range(2):
        outs.append((torch.empty_like(b.q), torch.empty_like(want[1])))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fm.tree_forward(b.q, b.k, b.v, b.table, lens[i], b.cu, b.scale, parents=b.parents, max_nodes=20,
                            o=outs[i][0], lse=outs[i][1], ws=ws)
        graphs.append(g)
    lens[1].sub_(100)
    second = fm.tree_forward(b.q, b.k, b.v, b.table, lens[1], b.cu, b.scale, parents=b.parents, max_nodes=20)
    for _ in range(20):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for got, ref in zip(outs, (want, second)):
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


@pytest.mark.parametrize("nodes,longest", [(1, 60), (1, 1500), (5, 400), (30, 700)])
def test_many_sequences(nodes, longest):
    """More sequences than a warp has lanes, of mixed lengths, some without nodes."""
    n = [nodes if i % 7 else 0 for i in range(333)]
    lens = [max(m, 1 + (i * 7919) % longest) for i, m in enumerate(n)]
    b = Batch(23, lens, n, 4, 2, 64, 16, None if nodes == 1 else "random")
    o, lse, code = run(b)
    assert code == 0
    b.check(o, lse, rows=3)


@pytest.mark.parametrize("nodes,kind", [(1, None), (24, "random")])
def test_offsets_at_the_ends_of_32_bits_are_reported_and_stay_in_bounds(nodes, kind):
    b = Batch(24, [100, 50, 200, 90], [nodes] * 4, 4, 2, 64, 16, kind)
    top, low = 2 ** 31 - 1, -2 ** 31
    for cu in ([0, top, low, top, low], [top, low, 0, top, 4 * nodes], [low, low, top, top, top],
               [0, nodes, top, low, 4 * nodes]):
        b.cu.copy_(ints(cu))
        around = torch.full((b.q.shape[0] + 64, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        fm.tree_forward(b.q, b.k, b.v, b.table, b.lens_t, b.cu, b.scale, parents=b.parents, max_nodes=nodes,
                        o=around[32:-32], status=status)
        torch.cuda.synchronize()
        assert fm.device_status(status) == _abi.FM_ERR_CACHE
        assert (around[:32] == 7).all() and (around[-32:] == 7).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv,nodes", [(128, 1, 1), (256, 2, 3), (300, 1, 2), (512, 1, 1), (129, 1, 5)])
def test_groups_of_many_heads(H, Hkv, nodes, d):
    """A node's heads fill row tiles, or pass over their ends."""
    b = Batch(25, [700, nodes, 130], [nodes] * 3, H, Hkv, d, 32, "random")
    o, lse, code = run(b)
    assert code == 0
    b.check(o, lse)


def test_in_inference_mode_and_with_allocated_outputs():
    b = Batch(26, [700, 40], [9, 3], 8, 2, 128, 16, "random")
    want = run(b)[:2]
    with torch.inference_mode():
        o, lse = fm.tree_forward(b.q, b.k, b.v, b.table, b.lens_t, b.cu, b.scale, parents=b.parents, max_nodes=9)
    assert not o.requires_grad and o.device == b.q.device
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("H,Hkv", [(8, 2), (10, 2), (8, 8)])
@pytest.mark.parametrize("bad", [float("nan"), float("-inf")])
def test_values_not_finite_beside_a_long_context(H, Hkv, bad):
    """As above, with a table that holds more tokens and units of more than 128 rows or of few."""
    nodes, ctx, node = 40, 900, 33
    b = Batch(27, [nodes + ctx], [nodes], H, Hkv, 128, 16, "beams")
    clean, clean_lse, _ = run(b)
    p = ctx + node
    b.v[b.table_np[0, p // 16], p % 16, :, 64] = bad
    o, lse, code = run(b)
    assert code == 0 and torch.equal(lse, clean_lse)
    for t in range(nodes):
        a = t
        while a > node:
            a = b.parents_np[0][a]
        want = clean[t].clone()
        if a == node:
            want[:, 64] = bad
        assert torch.equal(o[t].nan_to_num(nan=123.0), want.nan_to_num(nan=123.0)), t


@pytest.mark.parametrize("kind", [None, "padded", "random"])
@pytest.mark.parametrize("H,Hkv", [(8, 2), (6, 2), (5, 1)])
def test_trees_beside_a_long_context(kind, H, Hkv):
    nodes = [1, 64, 33, 0, 50, 64]
    lens = [1, 64, 700, 100, 1500, 900]
    b = Batch(28, lens, nodes, H, Hkv, 128, 16, kind)
    o, lse, code = run(b)
    assert code == 0
    b.check(o, lse)


@pytest.mark.parametrize("kind", [None, "chain", "padded", "random"])
@pytest.mark.parametrize("H,Hkv,d,lens", [(8, 1, 128, [260, 16, 100]), (14, 2, 64, [16, 31, 290]),
                                          (5, 1, 128, [1500, 700, 16]), (64, 2, 64, [200, 16, 20])])
def test_few_nodes_of_many_heads(kind, H, Hkv, d, lens):
    """Up to 16 nodes whose rows are several units of 16, NaN in a place that not all see."""
    b = Batch(29, lens, [16, 7, 12], H, Hkv, d, 16, kind)
    o, lse, code = run(b)
    assert code == 0
    b.check(o, lse)
    node, base = 5, lens[0] - 16
    p = base + node
    b.v[b.table_np[0, p // 16], p % 16, :, 3] = float("nan")
    o2, lse2, code = run(b)
    assert code == 0 and torch.equal(lse2, lse)
    for t in range(16):
        see = t >= node if kind is None else False
        a = t
        while kind is not None and a >= 0 and b.parents_np[0][a] != -2:
            see |= a == node
            a = b.parents_np[0][a]
        want = o[t].clone()
        if see:
            want[:, 3] = float("nan")
        assert torch.equal(o2[t].nan_to_num(nan=123.0), want.nan_to_num(nan=123.0)), t


# kernels: 16 rows; several units of 16 rows; 128 rows; 256 rows (with a sequence of up to 128, whose
# key tiles two slots take in turn)
KERNELS = [(64, [1, 1], 8, 2, 300, 16), (128, [1, 1], 5, 1, 300, 16), (128, [12, 3], 2, 2, 300, 16),
           (64, [12, 5], 8, 2, 100, 16), (128, [12, 16], 12, 2, 100, 32), (64, [20, 7], 8, 2, 300, 16),
           (128, [20, 32], 8, 2, 300, 64), (128, [20, 60], 8, 2, 900, 16), (128, [200, 33], 4, 1, 700, 16)]


@pytest.mark.parametrize("kind", [None, "random"])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf")])
@pytest.mark.parametrize("d,nodes,H,Hkv,ctx,page", KERNELS)
def test_infinities_in_the_context_reach_every_row(d, nodes, H, Hkv, ctx, page, bad, kind):
    """Whatever the weight's last bits, the infinity's sign stays; a context of one key too."""
    b = Batch(30, [1 + nodes[0], ctx + nodes[1]], nodes, H, Hkv, d, page, kind)
    clean, clean_lse, _ = run(b)
    cols = [1, min(ctx, d - 1)]           # a key each, spread over the context; the last column stays finite
    for seq, m in enumerate(cols):
        for c in range(m):
            p = c * ((1, ctx)[seq] // m)
            b.v[b.table_np[seq, p // page], p % page, :, c] = bad
    o, lse, code = run(b)
    assert code == 0 and torch.equal(lse, clean_lse)
    for seq, m in enumerate(cols):
        rows = slice(b.cu_np[seq], b.cu_np[seq + 1])
        assert (o[rows, :, :m] == bad).all(), (seq, int((o[rows, :, :m] != bad).sum()))
        assert torch.equal(o[rows, :, m:], clean[rows, :, m:])


@pytest.mark.parametrize("bad", [float("inf"), float("-inf")])
@pytest.mark.parametrize("d,nodes,H,Hkv,ctx,page", KERNELS)
def test_infinities_under_small_weights(d, nodes, H, Hkv, ctx, page, bad):
    """Weights down to 2^-125 of the largest one (the smallest normal number is 2^-126)."""
    b = Batch(31, [ctx + n for n in nodes], nodes, H, Hkv, d, page)
    b.scale = 1.0
    b.q.zero_()
    b.q[:, :, 0] = 1.0
    b.k.zero_()
    for seq in range(2):
        for c, x in enumerate((0.0, -1.0, -20.25, -40.5, -76.0, -80.0, -83.0, -85.5, -86.5)):
            p = 3 + c
            b.k[b.table_np[seq, p // page], p % page, :, 0] = x
            b.v[b.table_np[seq, p // page], p % page, :, c] = bad
    o, lse, code = run(b)
    assert code == 0 and lse.isfinite().all()
    assert (o[:, :, :9] == bad).all(), [(o[:, :, c] != bad).any().item() for c in range(9)]
    assert o[:, :, 9:].isfinite().all()


@pytest.mark.parametrize("d,nodes,H,Hkv,ctx,page", KERNELS)
def test_nan_under_a_weight_of_zero_reaches_every_row(d, nodes, H, Hkv, ctx, page):
    """Context keys whose weight underflows to 0 (scores 200 below the others') are visible all the same."""
    ctx = max(ctx, 256)
    b = Batch(32, [ctx + n for n in nodes], nodes, H, Hkv, d, page)
    b.scale = 1.0
    b.q.zero_()
    b.q[:, :, 0] = 1.0
    b.k.zero_()
    for seq in range(2):
        for p in range(128, 256):
            b.k[b.table_np[seq, p // page], p % page, :, 0] = -200.0
        b.v[b.table_np[seq, 130 // page], 130 % page, :, 9] = float("nan")
    o, lse, code = run(b)
    assert code == 0 and lse.isfinite().all()
    assert o[:, :, 9].isnan().all() and o[:, :, 10:].isfinite().all()


@pytest.mark.parametrize("d,G", [(128, 4), (64, 4), (128, 1)])
def test_a_workspace_for_the_largest_step_serves_smaller_ones(d, G):
    """One workspace, sized once for 60 nodes, through every kernel that fewer nodes take."""
    b = Batch(33, [900, 700], [60, 60], 2 * G, 2, d, 16)
    ws = fm.tree_workspace(b.q, b.k, b.v, b.table, 60)
    for nodes in (60, 40, 33, 32, 31, 17, 16, 5, 4, 1):
        c = Batch(33, [900, 700], [nodes, nodes], 2 * G, 2, d, 16)
        ws.fill_(255)
        o, lse, code = run(c, ws=ws)
        assert code == 0
        c.check(o, lse, rows=3)
