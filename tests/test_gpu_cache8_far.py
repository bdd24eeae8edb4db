"""The page operations on a cache of e4m3 codes, and the append with rotation, whose pools lie past 32 bits:
layers and pages further than 2^32 bytes from the first, and the largest number of pages.  Each call
is compared with the same call on small contiguous pools."""
import numpy as np
import pytest
import torch

import masked_attention_bound_gb300 as fm
from cache8_cases import F8, Batch8, ints
from cache_cases import Batch

pytestmark = pytest.mark.gpu


def _raw(x):
    """A pool as numbers that every operation of torch takes."""
    return x.view(torch.uint8) if x.dtype is F8 else x.view(torch.int16)


def _spread(x, page_stride, layer_stride=None):
    """A copy of a contiguous pool [pages].. or [layers][pages].. with these strides (elements)."""
    raw = _raw(x)
    strides = list(raw.stride())
    strides[-4] = page_stride
    if layer_stride:
        strides[0] = layer_stride
    size = sum((n - 1) * s for n, s in zip(raw.shape, strides)) + 1
    y = torch.zeros(size, dtype=raw.dtype, device="cuda").as_strided(raw.shape, strides)
    y.copy_(raw)
    return y.view(x.dtype)


def _same(a, b):
    assert torch.equal(_raw(a), _raw(b))


@pytest.mark.parametrize("codes", [True, False])
def test_append_with_rotation_past_32_bits(codes):
    nodes, lens = [40, 3, 1], [70, 20, 16]
    b = (Batch8 if codes else Batch)(50, lens, nodes, 2, 2, 128, 16)
    g = torch.Generator().manual_seed(51)
    q, k, v = (torch.randn(44, n, 128, generator=g).to(torch.bfloat16).cuda() for n in (4, 2, 2))
    freqs = torch.tensor(10.0 ** -np.arange(32.0), dtype=torch.float32, device="cuda")
    stride = (1 << 30) if codes else (1 << 29)                 # a GB a page
    far = [_spread(x, stride) for x in (b.k, b.v)]
    assert b.table_np[0, :5].max() << 30 > 1 << 32
    scales = [[x.clone() for x in (b.k_scale, b.v_scale)] if codes else [] for _ in range(2)]
    out = []
    for pools, s in (((b.k, b.v), scales[0]), (far, scales[1])):
        kw = dict(zip(("k_scale", "v_scale"), s))
        out.append(fm.cache_append_rotary(q, k, v, b.cu, freqs, *pools, b.table, b.lens_t, **kw))
    assert torch.equal(*out)
    for x, y in zip((b.k, b.v), far):
        _same(x, y)
    for x, y in zip(*scales):
        assert torch.equal(x.nan_to_num(-1.0), y.nan_to_num(-1.0))


def _layers(x, L, codes):
    """L layers of a pool: the rows of codes shifted by layer (scales: times a power of two)."""
    if codes:
        return torch.stack([_raw(x).roll(i, -1) for i in range(L)]).contiguous().view(F8)
    return torch.stack([x * 2.0 ** (i % 3) for i in range(L)]).contiguous()


@pytest.mark.parametrize("page_stride,layer_stride", [(1 << 30, 1 << 34), (1 << 13, (1 << 32) + (1 << 16))])
def test_accept_past_32_bits(page_stride, layer_stride):
    nodes, lens, L = [33, 5], [90, 25], 4
    b = Batch8(52, lens, nodes, 2, 2, 128, 16)
    k, v, ks, vs = (_layers(x, L, x.dtype is F8) for x in (b.k, b.v, b.k_scale, b.v_scale))
    far = [_spread(x, page_stride, layer_stride) for x in (k, v)]
    far_scales = [x.clone() for x in (ks, vs)]
    acc = ints([[0, 3, 4, 17, 18, 30, 32], [1, 3, 0, 0, 0, 0, 0]])
    a = fm.cache_accept(acc, ints([7, 2]), b.cu, k, v, b.table, b.lens_t, k_scale=ks, v_scale=vs)
    c = fm.cache_accept(acc, ints([7, 2]), b.cu, *far, b.table, b.lens_t, k_scale=far_scales[0], v_scale=far_scales[1])
    assert torch.equal(a, c) and a.tolist() == [64, 22]
    _same(k, far[0])
    _same(v, far[1])
    for x, y in zip((ks, vs), far_scales):
        assert torch.equal(x.nan_to_num(-1.0), y.nan_to_num(-1.0))


@pytest.mark.parametrize("page_stride,layer_stride", [(1 << 30, 1 << 34), (1 << 13, (1 << 32) + (1 << 16))])
def test_page_copies_past_32_bits(page_stride, layer_stride):
    """Room for more tokens of two rows that share their last page, then compaction."""
    g = torch.Generator().manual_seed(53)
    L, P, page, Hkv, d = 3, 12, 16, 2, 128
    pools = [torch.randint(0, 255, (L, P, page, Hkv, d), generator=g, dtype=torch.uint8).cuda() for _ in range(2)]
    scales = [torch.rand(L, P, Hkv, 1, generator=g).cuda() for _ in range(2)]
    far = [_spread(x.view(F8), page_stride, layer_stride) for x in pools]
    results = []
    for p, s in ((pools, scales), (far, [x.clone() for x in scales])):
        table = ints([[11, 9, -1, -1], [11, 9, -1, -1]])
        lens, ref = ints([25, 25]), ints([0] * 9 + [2, 0, 2])
        kw = dict(k_scale=s[0], v_scale=s[1])
        k, v = (x.view(F8) for x in p)
        fm.pages_reserve(ints([3, 30]), k, v, table, lens, ref, **kw)
        n = fm.pages_compact(k, v, table, lens, ref, **kw)
        results.append([table, lens, ref, n, *s, *(_raw(x.view(F8))[:, table[table >= 0].long().unique()] for x in p)])
    for x, y in zip(*results):
        assert torch.equal(x, y)


def test_the_largest_number_of_pages():
    """2^23 - 1 pages of 1 KB: appending, attention, accepting and compaction at the pool's end."""
    P, page, d = (1 << 23) - 1, 16, 64
    nodes, lens = [20, 1], [60, 17]
    g = torch.Generator().manual_seed(54)
    q, k, v = (torch.randn(21, n, d, generator=g).to(torch.bfloat16).cuda() for n in (2, 1, 1))
    freqs = torch.tensor(10.0 ** -np.arange(16.0), dtype=torch.float32, device="cuda")
    small = Batch8(55, lens, nodes, 2, 1, d, page)
    n_small = small.k.shape[0]
    results = []
    for shift in (0, P - n_small):
        if shift:
            pools = [torch.zeros(P, page, 1, d, dtype=torch.uint8, device="cuda").view(F8) for _ in range(2)]
            scales = [torch.ones(P, 1, 1, device="cuda") for _ in range(2)]
            for x, y in zip(pools, (small.k, small.v)):
                _raw(x)[shift:] = _raw(y)
            for x, y in zip(scales, (small.k_scale, small.v_scale)):
                x[shift:] = y
        else:
            pools, scales = [x.clone() for x in (small.k, small.v)], [x.clone() for x in (small.k_scale, small.v_scale)]
        table = torch.where(small.table >= 0, small.table + shift, small.table)
        kw = dict(k_scale=scales[0], v_scale=scales[1])
        rq = fm.cache_append_rotary(q, k, v, small.cu, freqs, *pools, table, small.lens_t, **kw)
        o, lse = fm.tree_forward(rq, *pools, table, small.lens_t, small.cu, 0.125, max_nodes=20, **kw)
        ref = torch.zeros(pools[0].shape[0], dtype=torch.int32, device="cuda")
        used = torch.cat([table[0, :4], table[1, :2]]).long()
        ref[used] = 1
        after = fm.cache_accept(ints([[2, 5, 6, 19], [0, 0, 0, 0]]), ints([4, 1]), small.cu, *pools, table, small.lens_t,
                                ref=ref, **kw)
        live = fm.pages_compact(*pools, table, after, ref, **kw)
        assert int(live) == 5 and table[0, :3].max() < 5 and table[1, :2].max() < 5
        first = [table[0, :3].long(), table[1, :2].long()]
        results.append([rq, o, lse, after] + [x[at] for x in (*map(_raw, pools), *(s.nan_to_num(-1.0) for s in scales))
                                              for at in first])
    for x, y in zip(*results):
        assert torch.equal(x, y)
