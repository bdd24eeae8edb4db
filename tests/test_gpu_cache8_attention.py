"""Attention over the paged cache of e4m3 codes (fm_tree_fwd_fp8) against the fp64 oracle."""
import numpy as np
import pytest
import torch

import masked_attention_bound_gb300 as fm
from cache8_cases import F8, NAN, Batch8, ints
from masked_attention_bound_gb300 import _abi

pytestmark = pytest.mark.gpu


def run(b, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = torch.full_like(b.q, float("nan"))
    lse = torch.full((b.H, b.q.shape[0]), float("nan"), dtype=torch.float32, device="cuda")
    kw.setdefault("max_nodes", max(b.nodes))
    fm.tree_forward(b.q, b.k, b.v, b.table, b.lens_t, b.cu, b.scale, parents=b.parents, o=o, lse=lse,
                    status=status, k_scale=b.k_scale, v_scale=b.v_scale, **kw)
    torch.cuda.synchronize()
    return o, lse, fm.device_status(status)


# one token a sequence: lengths around page and tile ends, empty context
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(2, 2), (8, 1), (7, 1), (12, 4), (40, 2), (3, 1)])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_single_tokens(d, H, Hkv, page):
    lens = [1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 300, 1000]
    b = Batch8(1, lens, [1] * len(lens), H, Hkv, d, page)
    o, lse, code = run(b)
    assert code == 0
    b.check(o, lse)


@pytest.mark.parametrize("kind", [None, "chain", "star", "random", "padded", "beams"])
@pytest.mark.parametrize("H,Hkv,d,page", [(2, 2, 64, 16), (8, 2, 128, 16), (6, 2, 128, 64), (5, 1, 64, 128),
                                          (16, 2, 128, 32)])
def test_trees(kind, H, Hkv, d, page):
    nodes = [1, 2, 5, 16, 17, 33, 64, 0, 3]
    lens = [1, 130, 5, 300, 128 + 17, 33, 190, 100, 259]
    b = Batch8(2, lens, nodes, H, Hkv, d, page, kind)
    o, lse, code = run(b)
    assert code == 0
    b.check(o, lse)


@pytest.mark.parametrize("kind", [None, "random"])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (4, 1), (9, 3)])
def test_many_nodes(kind, H, Hkv):
    b = Batch8(3, [256, 700, 513], [256, 200, 129], H, Hkv, 128, 16, kind)
    o, lse, code = run(b)
    assert code == 0
    b.check(o, lse)


@pytest.mark.parametrize("d", [64, 128])
def test_causal_run_longer_than_a_tree(d):
    b = Batch8(4, [1500, 1000], [700, 1000], 4, 2, d, 64)
    o, lse, code = run(b)
    assert code == 0
    b.check(o, lse, rows=60)


@pytest.mark.parametrize("kind", [None, "random", "padded"])
@pytest.mark.parametrize("H,Hkv,d,nodes,ctx", [(3, 1, 64, [28, 5], 4000), (4, 4, 128, [200, 17], 600),
                                               (8, 1, 128, [3, 16], 1250), (1, 1, 64, [17, 256], 2000)])
def test_little_work_of_more_than_16_rows(kind, H, Hkv, d, nodes, ctx):
    b = Batch8(29, [ctx + n for n in nodes], nodes, H, Hkv, d, 32, kind)
    o, lse, code = run(b)
    assert code == 0
    b.check(o, lse)


@pytest.mark.parametrize("nodes", [1, 40])
def test_long_context_is_split_and_joined(nodes):
    b = Batch8(5, [131072 - 7, 40000], [nodes] * 2, 8, 2, 128, 128, "random")
    o, lse, code = run(b)
    assert code == 0
    b.check(o, lse, rows=5)


@pytest.mark.parametrize("nodes,longest", [(1, 60), (1, 1500), (5, 400), (30, 700)])
def test_many_sequences(nodes, longest):
    rng = np.random.default_rng(19)
    lens = [int(x) for x in rng.integers(nodes, longest + nodes, size=300)]
    b = Batch8(19, lens, [nodes] * 300, 4, 1, 64, 16)
    o, lse, code = run(b)
    assert code == 0
    b.check(o, lse, rows=3, seqs=range(0, 300, 7))


def test_a_batch_with_empty_sequences_and_rows_behind_the_last():
    b = Batch8(6, [0, 40, 0, 9, 0], [0, 3, 0, 1, 0], 4, 2, 64, 16)
    q = torch.randn(9, 4, 64, device="cuda").to(torch.bfloat16)
    q[:4] = b.q
    o = torch.full_like(q, 7.0)
    lse = torch.full((4, 9), 7.0, device="cuda")
    fm.tree_forward(q, b.k, b.v, b.table, b.lens_t, b.cu, b.scale, max_nodes=3, o=o, lse=lse, k_scale=b.k_scale,
                    v_scale=b.v_scale)
    torch.cuda.synchronize()
    assert (o[4:] == 7).all() and (lse[:, 4:] == 7).all()
    b.check(o[:4], lse[:, :4])


# a kernel each: few rows, up to 16, more; more on the kernel for 16; pairs of tiles, whole and split
KERNELS = [(64, 1, 2, 1, 100, 16), (128, 1, 4, 1, 300, 64), (128, 3, 8, 2, 300, 16), (64, 12, 2, 2, 200, 32),
           (128, 30, 8, 2, 140, 16), (64, 70, 4, 2, 100, 16), (128, 64, 8, 2, 900, 128),
           (64, 40, 4, 1, 700, 64), (128, 64, 8, 2, 300, 64), (128, 50, 8, 2, 9000, 32)]


@pytest.mark.parametrize("d,nodes,H,Hkv,ctx,page", KERNELS)
def test_nan_codes_of_drafted_nodes_reach_the_rows_that_see_them(d, nodes, H, Hkv, ctx, page):
    b = Batch8(8, [nodes + ctx, nodes], [nodes, nodes], H, Hkv, d, page, "beams")
    clean, clean_lse, _ = run(b)
    node = min(2, nodes - 1)
    v = b.v.view(torch.uint8)
    for seq, base in ((0, ctx), (1, 0)):
        p = base + node
        v[b.table_np[seq, p // page], p % page, :, 5] = NAN
        v[b.table_np[seq, p // page], p % page, 0, 60] = NAN | 0x80
    last = nodes > 3
    p = ctx + nodes - 1                      # the last node's K: only its own rows
    if last:
        b.k.view(torch.uint8)[b.table_np[0, p // page], p % page] = NAN
    o, lse, code = run(b)
    assert code == 0
    G = H // Hkv
    for seq in range(2):
        for t in range(nodes):
            a = t
            while a > node:
                a = b.parents_np[seq][a]
            row = b.cu_np[seq] + t
            if last and seq == 0 and t == nodes - 1:
                assert o[row].isnan().all() and lse[:, row].isnan().all()
                continue
            want = clean[row].clone()
            if a == node:
                want[:, 5] = float("nan")
                want[:G, 60] = float("nan")
            assert torch.equal(o[row].nan_to_num(nan=123.0), want.nan_to_num(nan=123.0)), (seq, t)
            assert torch.equal(lse[:, row], clean_lse[:, row])


@pytest.mark.parametrize("d,nodes,H,Hkv,ctx,page", KERNELS)
def test_nan_codes_in_the_context_reach_every_row(d, nodes, H, Hkv, ctx, page):
    b = Batch8(10, [ctx + nodes], [nodes], H, Hkv, d, page)
    b.v.view(torch.uint8)[b.table_np[0, 40 // page], 40 % page, 0, 9] = NAN
    o, lse, code = run(b)
    assert code == 0 and lse.isfinite().all()
    assert o[:, :H // Hkv, 9].isnan().all()
    o[:, :H // Hkv, 9] = 0
    assert o.isfinite().all()


@pytest.mark.parametrize("d,nodes,H,Hkv,ctx,page", KERNELS)
def test_scales_far_apart(d, nodes, H, Hkv, ctx, page):
    """Blocks whose V is larger or smaller than others' by powers up to 2^40, one of zeros with the
    least scale, and keys that make one of the small ones' tokens dominate."""
    b = Batch8(11, [ctx + nodes, ctx + nodes + 7], [nodes, nodes], H, Hkv, d, page)
    e = torch.from_numpy(np.random.default_rng(12).integers(-40, 3, b.v_scale.shape)).cuda()
    b.v_scale *= torch.exp2(e.float())
    z = b.table_np[0, 16 // page], 16 % page // 16
    b.v.view(torch.uint8)[z[0], z[1] * 16:z[1] * 16 + 16] = 0
    b.v_scale[z[0], :, z[1]] = 2.0 ** -60
    o, lse, code = run(b)
    assert code == 0
    b.check(o, lse, rows=8)


@pytest.mark.parametrize("d,nodes,H,Hkv,ctx,page", KERNELS)
def test_scales_out_of_range_are_read_as_the_nearest(d, nodes, H, Hkv, ctx, page):
    b = Batch8(13, [ctx + nodes], [nodes], H, Hkv, d, page)
    first = b.table_np[0, 0]
    results = []
    for least in (2.0 ** -60, 0.0, -1.0, 2.0 ** -100, float("nan")):
        b.v_scale[first, :, 0] = least
        b.k_scale[first, :, 0] = least
        results.append(run(b)[:2])
    for o, lse in results[1:]:
        assert torch.equal(o, results[0][0]) and torch.equal(lse, results[0][1])


@pytest.mark.parametrize("d,nodes,H,Hkv,ctx,page", KERNELS)
def test_queries_of_all_sizes(d, nodes, H, Hkv, ctx, page):
    """Rows scaled by 2^-100 to 2^100 (with keys that undo it), rows of zeros, elements far below
    their row's largest."""
    b = Batch8(14, [ctx + nodes], [nodes], H, Hkv, d, page)
    T = b.q.shape[0]
    b.q[:, :, 3] *= 2.0 ** -30
    b.q[T // 2, 0] = 0
    o, lse, code = run(b)
    assert code == 0
    b.check(o, lse, rows=8)
    b.q *= 2.0 ** -50
    b.k_scale *= 2.0 ** 50
    o2, lse2, _ = run(b)
    b.check(o2, lse2, rows=8)


def test_large_scores_and_queries_not_finite():
    b = Batch8(15, [200], [3], 2, 1, 64, 16)
    b.q[0, 0] *= 1e4
    b.q[1, 1, 5] = float("inf")
    b.q[2, 0, 5] = float("nan")
    o, lse, code = run(b)
    assert code == 0
    assert o[1, 1].isnan().all() and o[2, 0].isnan().all()
    assert o[0].isfinite().all() and o[1, 0].isfinite().all() and o[2, 1].isfinite().all()


@pytest.mark.parametrize("nodes", [1, 24])
def test_strides(nodes):
    b = Batch8(16, [150, 77], [nodes, nodes], 4, 2, 64, 32, "random" if nodes > 1 else None)
    want = run(b)
    pages, page, Hkv, d = b.k.shape

    def wide(x):
        y = torch.full((pages, Hkv + 1, page + 2, d + 16), NAN, dtype=torch.uint8, device="cuda")
        y = y.permute(0, 2, 1, 3)[:, 1:page + 1, :Hkv, 16:]          # heads before tokens
        y.copy_(x.view(torch.uint8))
        return y.view(F8)

    b.k, b.v = wide(b.k), wide(b.v)
    q = torch.full((b.q.shape[0] + 1, 6, 72), float("nan"), dtype=torch.bfloat16, device="cuda")[1:, 1:5, 8:]
    q.copy_(b.q)
    b.q = q
    got = run(b)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("nodes", [1, 24])
def test_offsets_past_32_bits(nodes):
    """Pools whose last pages lie more than 2^32 bytes from the first."""
    b = Batch8(17, [100], [nodes], 2, 1, 128, 16)
    want = run(b)
    n, stride = b.k.shape[0], 1 << 30
    used = b.table_np[0, :-(-b.lens[0] // 16)]
    big = [torch.zeros((n - 1) * stride + 16 * 128, dtype=torch.uint8, device="cuda")
           .as_strided((n, 16, 1, 128), (stride, 128, 128, 1)) for _ in range(2)]
    assert used.max() * stride > 1 << 32
    for to, x in zip(big, (b.k, b.v)):
        to.copy_(x.view(torch.uint8))
    b.k, b.v = (x.view(F8) for x in big)
    got = run(b)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("nodes,kind", [(1, None), (24, "random"), (70, "random")])
def test_bad_entries_are_reported_and_stay_in_bounds(nodes, kind):
    b = Batch8(18, [nodes + 50] * 6, [nodes] * 6, 4, 2, 64, 16, kind)
    want, want_lse, _ = run(b)
    b.lens_t[0] = -3
    b.lens_t[1] = nodes - 1
    b.lens_t[2] = b.max_pages * 16 + 1
    b.table[3, 1] = b.k.shape[0]
    b.table[4, 0] = -1
    o, lse, code = run(b)
    assert code == _abi.FM_ERR_CACHE
    assert (o[:3 * nodes] == 0).all() and lse[:, :3 * nodes].isneginf().all()
    assert o.isfinite().all()
    assert torch.equal(o[5 * nodes:], want[5 * nodes:]) and torch.equal(lse[:, 5 * nodes:], want_lse[:, 5 * nodes:])
    # keys on a page out of range read as 0
    zero = b.table_np[4, 0]
    b.table[4, 0] = int(zero)
    b.k.view(torch.uint8)[zero] = 0
    b.v.view(torch.uint8)[zero] = 0
    o2, lse2, _ = run(b)
    at = slice(4 * nodes, 5 * nodes)
    assert (o2[at].float() - o[at].float()).abs().max() < 0.02 and (lse2[:, at] - lse[:, at]).abs().max() < 1e-4


@pytest.mark.parametrize("nodes", [1, 24, 64])
def test_equal_inputs_give_equal_bits(nodes):
    b = Batch8(20, [20000, 5000, 100], [nodes] * 3, 8, 2, 128, 64)
    first = run(b)
    for _ in range(3):
        again = run(b)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


@pytest.mark.parametrize("nodes", [1, 24])
def test_captured_and_replayed_with_growing_lengths(nodes):
    b = Batch8(21, [400, 300], [nodes] * 2, 8, 2, 128, 16)
    full = b.lens_t.clone()
    o, lse = torch.empty_like(b.q), torch.empty(8, b.q.shape[0], device="cuda")
    ws = fm.tree_workspace(b.q, b.k, b.v, b.table, nodes)

    def call():
        fm.tree_forward(b.q, b.k, b.v, b.table, b.lens_t, b.cu, b.scale, max_nodes=nodes, o=o, lse=lse, ws=ws,
                        k_scale=b.k_scale, v_scale=b.v_scale)

    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for less in (70, 33, 0):
        b.lens_t.copy_(full - less)
        g.replay()
        torch.cuda.synchronize()
        b.lens = [x - less for x in (400, 300)]
        b.check(o, lse)


@pytest.mark.parametrize("nodes", [1, 24, 70])
def test_two_calls_at_once(nodes):
    batches = [Batch8(22 + i, [3000, 200], [nodes] * 2, 8, 2, 128, 64) for i in range(2)]
    want = [run(b) for b in batches]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for b, s in zip(batches, streams):
        got.append([fm.tree_forward(b.q, b.k, b.v, b.table, b.lens_t, b.cu, b.scale, max_nodes=nodes, stream=s,
                                    k_scale=b.k_scale, v_scale=b.v_scale) for _ in range(3)])
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for o, lse in g:
            assert torch.equal(o, w[0]) and torch.equal(lse, w[1])


@pytest.mark.parametrize("nodes,d", [(1, 128), (1, 64), (16, 128), (50, 128), (50, 64)])
def test_a_wait_that_runs_out_is_reported_then_the_next_call_is_clean(nodes, d):
    """A hook withholds one release in each block (see fm_test_hooks): its wait runs out after 20 ms, and
    the call ends by itself with the status set; one for each kernel.  (Long enough that every block
    comes back to its first stage.)"""
    b = Batch8(24, [4100] * 8, [nodes] * 8, 32, 8, d, 16, "random")
    ws = fm.tree_workspace(b.q, b.k, b.v, b.table, nodes)
    ws.zero_()
    assert fm.lib().fm_test_hooks(20_000_000, 8) == _abi.FM_OK
    try:
        code = run(b, ws=ws)[2]
    finally:
        assert fm.lib().fm_test_hooks(0, 0) == _abi.FM_OK
    assert code == _abi.FM_ERR_TIMEOUT, _abi.status_string(code)
    o, lse, code = run(b, ws=ws)
    assert code == 0
    b.check(o, lse, rows=3, seqs=[0, 5])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv,nodes", [(128, 1, 1), (256, 2, 3), (300, 1, 2), (129, 1, 5)])
def test_groups_of_many_heads(H, Hkv, nodes, d):
    b = Batch8(25, [300, 90], [nodes] * 2, H, Hkv, d, 32, "random")
    o, lse, code = run(b)
    assert code == 0
    b.check(o, lse)


def test_agrees_with_the_bf16_cache_of_the_same_values():
    """Values that both caches hold exactly give the same attention to the roundings of P."""
    b = Batch8(26, [700, 80], [20, 20], 8, 2, 128, 16, "random")
    o, lse, _ = run(b)
    values = []
    for c, s in ((b.k, b.k_scale), (b.v, b.v_scale)):
        s = s.nan_to_num(1.0).transpose(1, 2).repeat_interleave(16, 1)[..., None]
        x = (c.float() * s).to(torch.bfloat16)
        assert torch.equal(x.float().nan_to_num(), (c.float() * s).nan_to_num())
        values.append(x)
    o2, lse2 = fm.tree_forward(b.q, *values, b.table, b.lens_t, b.cu, b.scale, parents=b.parents, max_nodes=20)
    # Off by the roundings of P (2^-8 of a weight in bf16, 2^-11 in f16) and of the two outputs (2^-8
    # each), all relative to the sum of the weighted magnitudes, of which `a` is one rounded to bf16 in
    # its turn (P and output: 2^-7): (3 * 2^-8 + 2^-11) (1 + 2^-7) < 3 * 2^-8 + 2^-11 + 2^-12.
    a = fm.tree_forward(b.q, values[0], values[1].abs(), b.table, b.lens_t, b.cu, b.scale, parents=b.parents,
                        max_nodes=20)[0].float()
    assert ((o.float() - o2.float()).abs() <= (3 * 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -12) * a + 1e-6).all()
    assert (lse - lse2).abs().max() < 1e-3
