"""Attention over the cache of e4m3 codes where its factors leave the range of fp32 or Q's parts that of a
code, against the fp64 oracle."""
import numpy as np
import pytest
import torch

from cache8_cases import Batch8
from test_gpu_cache8_attention import KERNELS, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", [None, "beams"])
@pytest.mark.parametrize("d,nodes,H,Hkv,ctx,page", KERNELS)
def test_rows_of_tiny_queries(d, nodes, H, Hkv, ctx, page, kind):
    """A score times its factors is 0 long before bf16 ends; what a row does not see stays unseen."""
    b = Batch8(40, [ctx + nodes, nodes + 3], [nodes, nodes], H, Hkv, d, page, kind)
    T = b.q.shape[0]
    e = torch.tensor([-130.0, -100.0, 0.0, -90.0, -60.0, -120.0, -75.0], dtype=torch.float64, device="cuda")
    at = (torch.arange(T, device="cuda")[:, None] * 3 + torch.arange(H, device="cuda")) % len(e)
    b.q = (b.q.double() * torch.exp2(e[at])[..., None]).to(torch.bfloat16)
    o, lse, code = run(b)
    assert code == 0
    b.check(o, lse)


@pytest.mark.parametrize("d,nodes,H,Hkv,ctx,page", KERNELS)
@pytest.mark.parametrize("scale", [1e-30, 2e-38])
def test_tiny_scales(d, nodes, H, Hkv, ctx, page, scale):
    b = Batch8(41, [ctx + nodes, nodes + 3], [nodes, nodes], H, Hkv, d, page)
    b.scale = scale
    o, lse, code = run(b)
    assert code == 0
    b.check(o, lse, rows=12)


@pytest.mark.parametrize("d,nodes,H,Hkv,ctx,page", KERNELS)
def test_large_factors_of_keys_of_zeros(d, nodes, H, Hkv, ctx, page):
    """Scores of 0 under a factor past the range of fp32."""
    b = Batch8(42, [ctx + nodes, nodes + 3], [nodes, nodes], H, Hkv, d, page)
    b.k.view(torch.uint8).zero_()
    b.k_scale.fill_(2.0 ** 60)
    b.q[::2] *= 2.0 ** 100
    o, lse, code = run(b)
    assert code == 0
    b.check(o, lse, rows=12)


@pytest.mark.parametrize("d,nodes,H,Hkv,ctx,page", KERNELS)
@pytest.mark.parametrize("e", [-100, 100])
def test_queries_of_all_sizes_with_keys_and_scale_that_undo_them(d, nodes, H, Hkv, ctx, page, e):
    b = Batch8(43, [ctx + nodes], [nodes], H, Hkv, d, page)
    b.q *= 2.0 ** e
    b.k_scale *= 2.0 ** (-e // 2)
    b.scale *= 2.0 ** (-e // 2)
    o, lse, code = run(b)
    assert code == 0
    b.check(o, lse, rows=12)


@pytest.mark.parametrize("d,nodes,H,Hkv,ctx,page", KERNELS)
@pytest.mark.parametrize("inf", [float("inf"), float("-inf")])
def test_a_row_with_an_infinite_query_is_nan(d, nodes, H, Hkv, ctx, page, inf):
    """Also where every score is -inf: there is no softmax of them.  Other rows are not touched."""
    b = Batch8(44, [ctx + nodes], [nodes], H, Hkv, d, page, "beams")
    k = b.k.view(torch.uint8)
    k[..., 5] = torch.where(k[..., 5] & 0x7f == 0x7f, k[..., 5], 0x38)
    want, want_lse, _ = run(b)
    t, h = nodes // 2, H - 1
    b.q[t, h, 5] = inf
    o, lse, code = run(b)
    assert code == 0
    assert o[t, h].isnan().all() and lse[h, t].isnan()
    o[t, h], lse[h, t] = want[t, h], want_lse[h, t]
    assert torch.equal(o, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("d,nodes,H,Hkv,ctx,page", KERNELS)
@pytest.mark.parametrize("ratio", [2.0 ** 10, -(2.0 ** 12)])
def test_one_element_of_a_row_far_above_the_others(d, nodes, H, Hkv, ctx, page, ratio):
    """The others decide the scores (K is 0 at the large one).  They are 2^-13 of it or more, which every
    kernel keeps exactly, so that the tolerance has no term for Q."""
    b = Batch8(45, [ctx + nodes, nodes + 3], [nodes, nodes], H, Hkv, d, page, "beams")
    k = b.k.view(torch.uint8)
    k[..., 9] = torch.where(k[..., 9] & 0x7f == 0x7f, k[..., 9], 0)
    least = abs(ratio) * 2.0 ** -13
    b.q = torch.copysign(b.q.abs().clamp_min(least), b.q)
    b.q[..., 9] = ratio
    o, lse, code = run(b)
    assert code == 0
    b.check(o, lse)
