"""The paged-cache oracle against independent definitions (CPU)."""
import numpy as np
import pytest
import torch

from oracle import attention as oa
from oracle import cache as oc
from oracle import masks as om


def test_chain_equals_causal_attention():
    rng = np.random.default_rng(0)
    n, ctx, H, Hkv, d = 7, 12, 4, 2, 8
    S = ctx + n
    q, k, v = rng.normal(size=(n, H, d)), rng.normal(size=(S, Hkv, d)), rng.normal(size=(S, Hkv, d))
    o, lse, _ = oc.tree_attention(q, k, v, oc.visible(n, ctx), 0.3)
    ii, jj = np.arange(n)[:, None] + ctx, np.arange(S)[None]
    mask = torch.tensor(jj <= ii)
    for h in range(H):
        ref = torch.nn.functional.scaled_dot_product_attention(
            torch.tensor(q[:, h]), torch.tensor(k[:, h // 2]), torch.tensor(v[:, h // 2]),
            attn_mask=mask, scale=0.3).numpy()
        assert np.abs(o[:, h] - ref).max() < 1e-12
        s = 0.3 * q[:, h] @ k[:, h // 2].T
        want = [np.log(np.exp(s[t, : ctx + t + 1]).sum()) for t in range(n)]
        assert np.abs(lse[h] - want).max() < 1e-12


def test_tree_in_depth_first_order_equals_column_bounds():
    """In depth-first order the nodes that see node j are j and the ones up to the end of its
    subtree: the framework's column bounds describe the same mask."""
    parents = [-1, 0, 1, 1, 0, 4, -1, 6]
    ends = [6, 4, 3, 4, 6, 6, 8, 8]
    n = len(parents)
    see = oc.visible(n, 0, parents)
    lts, lte = np.array(ends), np.full(n, n)
    uts, ute = np.zeros(n, int), np.arange(n)
    assert np.array_equal(see, ~om.dense_mask(lts, lte, uts, ute, n))


def test_padding_sees_nothing_and_is_seen_by_none():
    see = oc.visible(4, 3, [-1, -2, 1, 0])
    assert not see[1].any() and not see[:, 4].any()
    assert np.array_equal(see[2], [1, 1, 1, 0, 0, 1, 0]) and np.array_equal(see[3], [1, 1, 1, 1, 0, 0, 1])


def test_empty_row():
    o, lse, _ = oc.tree_attention(np.ones((1, 1, 2)), np.ones((1, 1, 2)), np.ones((1, 1, 2)),
                                  oc.visible(1, 0, [-2]), 1.0)
    assert (o == 0).all() and np.isneginf(lse).all()


def test_append_and_accept_by_hand():
    pool = np.zeros((3, 2, 1, 1))
    got = oc.append(np.arange(1., 4.).reshape(3, 1, 1), [0, 1, 3], pool, [[2, -1], [0, 1]], [2, 3])
    assert got[:, :, 0, 0].tolist() == [[0, 2], [3, 0], [0, 1]]
    pool = np.arange(8.).reshape(1, 4, 2, 1, 1)
    got, lens = oc.accept([[1, 3]], [0, 4], pool, [[3, 0, 1]], [5])   # tokens 6 7 0 1 2, base 1
    assert lens == [3] and got[0, :, :, 0, 0].tolist() == [[2, 1], [2, 3], [4, 5], [6, 0]]


def test_pages_by_hand():
    rows, lens, ref = [[0, 2], [5], []], [5, 4, 0], [1, 0, 1, 0, 0, 1]
    rows1, lens1, ref1 = oc.fork([0, 0, -1], rows, lens, ref)
    assert rows1 == [[0, 2], [0, 2], []] and lens1 == [5, 5, 0] and ref1 == [2, 0, 2, 0, 0, 0]
    rows2, lens2, ref2, copies, asked = oc.reserve([1, 4, 2], rows1, lens1, ref1, 4, 3)
    assert rows2 == [[0, 1], [0, 3, 4], [5]] and lens2 == [6, 9, 2] and asked == 4
    assert ref2 == [2, 1, 0, 1, 1, 1] and copies == [(2, 1, 1), (2, 3, 1)]
    same = oc.reserve([1, 4, 5], rows1, lens1, ref1, 4, 3)
    assert same[:3] == (rows1, lens1, ref1) and same[3] is None and same[4] == 5
    rows3, ref3, moves, live = oc.compact(rows2, ref2)
    assert live == 5 and moves == [(5, 2)] and rows3 == [[0, 1], [0, 3, 4], [2]]
    assert ref3 == [2, 1, 1, 1, 1, 0]


@pytest.mark.parametrize("seed", range(4))
def test_page_counts_add_up(seed):
    """After any step, every page's count is the number of rows that hold it, and rows that
    grew share no page that they will write."""
    rng = np.random.default_rng(seed)
    page, B, P = 4, 6, 60
    rows, lens, ref = [[] for _ in range(B)], [0] * B, [0] * P
    for _ in range(12):
        rows, lens, ref = oc.fork([int(rng.integers(-1, B)) for _ in range(B)], rows, lens, ref)
        grow = [int(rng.integers(0, 6)) for _ in range(B)]
        rows, lens, ref, copies, _ = oc.reserve(grow, rows, lens, ref, page, 20)
        if rng.random() < 0.3:
            rows, ref, _, live = oc.compact(rows, ref)
            assert all(r != 0 for r in ref[:live]) and not any(ref[live:])
        count = [0] * P
        for r in rows:
            for p in r:
                count[p] += 1
        assert count == ref
        assert [len(r) for r in rows] == [-(-x // page) for x in lens]
        if copies is not None:
            for b in range(B):
                if grow[b] and lens[b]:
                    assert ref[rows[b][-1]] == 1


def test_gather():
    pool = np.arange(12.).reshape(3, 2, 1, 2)
    assert oa.to64(oc.gather(pool, [2, 0], 3))[:, 0, 0].tolist() == [8, 10, 0]
