"""Appending with the rotation by position, to caches of bf16 and of e4m3 codes, and the page
operations on a cache of codes, against the fp64 oracle."""
import numpy as np
import pytest
import torch

import masked_attention_bound_gb300 as fm
from cache8_cases import F8, NAN, Batch8, codes64, ints, same_codes
from cache_cases import Batch
from masked_attention_bound_gb300 import _abi
from oracle import cache as oc
from oracle import cache8 as o8
from oracle.attention import to64

pytestmark = pytest.mark.gpu


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _bytes(x):
    return x.reshape(-1).view(torch.uint8)


def _freqs(n, base=10000.0):
    return torch.tensor(base ** (-np.arange(n) / max(n, 1)), dtype=torch.float32, device="cuda")


def _new(seed, T, H, d, size=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, H, d, generator=g) * size).to(torch.bfloat16).cuda()


def _places(b):
    return np.concatenate([np.arange(x - n, x) for x, n in zip(b.lens, b.nodes)] or [[]]).astype(np.int64)


def bf16_excess(got, exact, pair):
    """How far |got - exact| is past its bound: half a step of bf16 (2^-8 of the value), and the fp32
    rotation: cos and sin to 2^-26 and two roundings (2^-24 of the pair's size each)."""
    return np.abs(to64(got) - exact) - (2.0 ** -8 * np.abs(exact) + 2.0 ** -22 * pair + 1e-38)


def pair_size(x, n, interleaved):
    """|a| + |b| of the pair that an element belongs to."""
    a = np.abs(x)
    s = a.copy()
    i, j = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    s[..., i] = s[..., j] = a[..., i] + a[..., j]
    return s


CASES = [  # d, Hkv, H, page, rot, interleaved, nodes
    (64, 1, 1, 16, 64, False, [1, 1, 1]), (128, 2, 8, 32, 128, False, [3, 0, 200, 1]), (64, 3, 3, 64, 32, True, [17, 16, 15]),
    (128, 16, 16, 128, 64, False, [1, 130]), (128, 8, 32, 16, 128, True, [300]), (128, 2, 6, 16, 16, False, [5, 9, 40]),
    (64, 5, 10, 32, 48, True, [33, 2]), (128, 1, 5, 64, 96, False, [18, 31, 47, 1]), (64, 2, 0, 16, 64, False, [7, 50]),
]


@pytest.mark.parametrize("skew", [0, 5, 15])
@pytest.mark.parametrize("d,Hkv,H,page,rot,inter,nodes", CASES)
def test_append_rotary_to_bf16(d, Hkv, H, page, rot, inter, nodes, skew):
    lens = [n + skew + 37 * i for i, n in enumerate(nodes)]
    b = Batch(1, lens, nodes, Hkv, Hkv, d, page)
    T = sum(nodes)
    k, v = _new(2, T, Hkv, d), _new(3, T, Hkv, d)
    q = _new(4, T, H, d) if H else None
    f = _freqs(rot // 2)
    pos = _places(b)
    want = o8.rotate(to64(k), pos, to64(f), inter)
    old = [x.clone() for x in (b.k, b.v)]
    st = _status()
    out = fm.cache_append_rotary(q, k, v, b.cu, f, b.k, b.v, b.table, b.lens_t, interleaved=inter, status=st)
    assert fm.device_status(st) == 0
    if H:
        rq = o8.rotate(to64(q), pos, to64(f), inter)
        assert bf16_excess(out, rq, pair_size(to64(q), rot // 2, inter)).max() <= 0
        assert torch.equal(out[..., rot:], q[..., rot:])
    else:
        assert out is None
    size = pair_size(to64(k), rot // 2, inter)
    for s, (n, x) in enumerate(zip(nodes, lens)):
        for i in range(n):
            p, row = x - n + i, int(b.cu_np[s]) + i
            at = b.table_np[s][p // page], p % page
            assert bf16_excess(b.k[at], want[row], size[row]).max() <= 0
            assert torch.equal(b.v[at], v[row])
            old[0][at], old[1][at] = b.k[at], b.v[at]
    for new, o in zip((b.k, b.v), old):                      # nothing else is written
        assert torch.equal(new.view(torch.int16), o.view(torch.int16))


def check_codes(b, x, size, pool, scales, old_pool, old_scales):
    """Codes and scales after appending exact values x [T][Hkv][d] (each off by 2^-22 of `size` at
    most before its rounding) to a pool that held old_pool, old_scales."""
    page = b.page
    got, gs = codes64(pool), scales.cpu().numpy().astype(np.float64)
    want, ws = o8.append(x, b.cu_np, codes64(old_pool), old_scales.cpu().numpy().astype(np.float64), b.table_np, b.lens)
    assert np.array_equal(gs, ws, equal_nan=True), "scales"
    new = np.zeros(got.shape[:2], bool)
    for s, (n, length) in enumerate(zip(b.nodes, b.lens)):
        for i in range(n):
            p, row = length - n + i, int(b.cu_np[s]) + i
            at = b.table_np[s][p // page], p % page
            new[at] = True
            sc = gs[at[0], :, at[1] // 16][:, None]
            # half a step of a code: 2^-4 of the value, 2^-10 of the scale below its normal ones
            bound = np.maximum(2.0 ** -4 * np.abs(x[row]), 2.0 ** -10 * sc) * (1 + 2.0 ** -10) + 2.0 ** -22 * size[row]
            assert (np.abs(got[at] * sc - x[row]) <= bound).all(), (s, i)
    assert np.array_equal(got[~new], want[~new], equal_nan=True), "codes of other tokens"
    return ((got != want) & ~(np.isnan(got) & np.isnan(want))).sum()


@pytest.mark.parametrize("skew", [0, 5, 15])
@pytest.mark.parametrize("d,Hkv,H,page,rot,inter,nodes", CASES)
def test_append_rotary_to_codes(d, Hkv, H, page, rot, inter, nodes, skew):
    lens = [n + skew + 37 * i for i, n in enumerate(nodes)]
    b = Batch8(1, lens, nodes, Hkv, Hkv, d, page)
    T = sum(nodes)
    # the second sequence's values are large, so that the scales of its blocks grow
    k, v = _new(2, T, Hkv, d), _new(3, T, Hkv, d)
    if len(nodes) > 1:
        k[b.cu_np[1]:b.cu_np[2]] *= 50
        v[b.cu_np[1]:b.cu_np[2]] *= 900
    q = _new(4, T, H, d) if H else None
    f = _freqs(rot // 2)
    pos = _places(b)
    old = [x.clone() for x in (b.k, b.k_scale, b.v, b.v_scale)]
    st = _status()
    out = fm.cache_append_rotary(q, k, v, b.cu, f, b.k, b.v, b.table, b.lens_t, interleaved=inter,
                                 k_scale=b.k_scale, v_scale=b.v_scale, status=st)
    assert fm.device_status(st) == 0
    if H:
        rq = o8.rotate(to64(q), pos, to64(f), inter)
        assert bf16_excess(out, rq, pair_size(to64(q), rot // 2, inter)).max() <= 0
    x = o8.rotate(to64(k), pos, to64(f), inter)
    flips = check_codes(b, x, pair_size(to64(k), rot // 2, inter), b.k, b.k_scale, old[0], old[1])
    assert flips <= 2 + x.size * 2.0 ** -16            # values next to the middle of two codes
    assert check_codes(b, to64(v), np.zeros(v.shape), b.v, b.v_scale, old[2], old[3]) == 0


@pytest.mark.parametrize("Hkv,d,page", [(1, 64, 16), (8, 128, 64)])
def test_append_codes_without_rotation(Hkv, d, page):
    nodes = [1, 0, 40, 16, 1]
    b = Batch8(5, [n + 11 * i for i, n in enumerate(nodes)], nodes, Hkv, Hkv, d, page)
    k, v = _new(6, sum(nodes), Hkv, d, 3.0), _new(7, sum(nodes), Hkv, d, 1e-3)
    old = [x.clone() for x in (b.k, b.k_scale, b.v, b.v_scale)]
    st = _status()
    assert fm.cache_append(k, v, b.cu, b.k, b.v, b.table, b.lens_t, k_scale=b.k_scale, v_scale=b.v_scale, status=st) is None
    assert fm.device_status(st) == 0
    z = np.zeros(k.shape)
    assert check_codes(b, to64(k), z, b.k, b.k_scale, old[0], old[1]) == 0
    assert check_codes(b, to64(v), z, b.v, b.v_scale, old[2], old[3]) == 0


def test_token_by_token_as_in_one_call():
    """A block that is filled token by token by growing values: each growth rounds the codes again, so
    they are compared to the oracle's, which does the same."""
    b = Batch8(8, [40], [40], 2, 2, 64, 32)
    k, v = _new(9, 40, 2, 64), _new(10, 40, 2, 64)
    v *= torch.exp2(torch.arange(40, device="cuda").float() / 4)[:, None, None].to(torch.bfloat16)
    want, ws = codes64(b.v), b.v_scale.cpu().numpy().astype(np.float64)
    for i in range(40):
        fm.cache_append(k[i:i + 1], v[i:i + 1], ints([0, 1]), b.k, b.v, b.table, ints([i + 1]), k_scale=b.k_scale,
                        v_scale=b.v_scale)
        want, ws = o8.append(to64(v[i:i + 1]), [0, 1], want, ws, b.table_np, [i + 1])
    assert same_codes(b.v, want) and np.array_equal(b.v_scale.cpu().numpy(), ws, equal_nan=True)


def test_values_not_finite_and_out_of_range():
    b = Batch8(11, [20], [20], 1, 1, 64, 16)
    k, v = _new(12, 20, 1, 64), _new(13, 20, 1, 64)
    v[3, 0, 5], v[3, 0, 6], v[4, 0, 7] = float("inf"), float("-inf"), float("nan")
    v[16:] = 0
    k[:16] = 3e38
    old = [x.clone() for x in (b.k, b.k_scale, b.v, b.v_scale)]
    fm.cache_append(k, v, b.cu, b.k, b.v, b.table, b.lens_t, k_scale=b.k_scale, v_scale=b.v_scale)
    for pool, scales, x, at in ((b.k, b.k_scale, k, 0), (b.v, b.v_scale, v, 2)):
        want, ws = o8.append(to64(x), b.cu_np, codes64(old[at]), old[at + 1].cpu().numpy().astype(np.float64), b.table_np, [20])
        assert same_codes(pool, want) and np.array_equal(scales.cpu().numpy(), ws, equal_nan=True)
    t = b.table_np[0]
    assert b.v_scale[t[1], 0, 0] == 2.0 ** -60 and b.k_scale[t[0], 0, 0] == 2.0 ** 60
    assert (b.k[t[0]].float() == 448).all()
    assert b.v[t[0], 3, 0, 5].float() == 448 and b.v[t[0], 4, 0, 7].float().isnan()


@pytest.mark.parametrize("pos", [0, 1, -1, 131071, (1 << 30) + 12345, -(1 << 31), (1 << 31) - 1])
@pytest.mark.parametrize("inter", [False, True])
def test_far_positions(pos, inter):
    b = Batch(14, [3], [3], 2, 2, 128, 16)
    q, k = _new(15, 3, 2, 128), _new(16, 3, 2, 128)
    f = _freqs(64)
    f[7], f[20] = -0.3, 7.5                        # any finite frequency
    p = ints([pos, 0, pos])
    out = fm.cache_append_rotary(q, k, k, b.cu, f, b.k, b.v, b.table, b.lens_t, positions=p, interleaved=inter)
    want = o8.rotate(to64(q), [pos, 0, pos], to64(f), inter)
    # the angle itself: 2^-33 of a turn
    assert (bf16_excess(out, want, pair_size(to64(q), 64, inter)) - 2.0 ** -30 * 8).max() <= 0
    assert torch.equal(out[1], q[1])


def test_frequencies_of_all_sizes():
    b = Batch(14, [3], [3], 2, 2, 128, 16)
    q, k = _new(15, 3, 2, 128), _new(16, 3, 2, 128)
    f = _freqs(64)
    sizes = [0.0, -0.0, 1e-42, 2.0 ** -100, 2.0 ** -40 * 1.3, 2.0 ** -9 * 0.999, 2.0 ** -9, -(2.0 ** -8), 1.7, 1e4,
             2.0 ** 22 + 0.5, 2.0 ** 23 + 1, 2.0 ** 24, -(2.0 ** 24) * 1.1, 2.0 ** 25 * 1.3]
    f[:len(sizes)] = torch.tensor(sizes)
    pos = [1000, 3, -999]
    out = fm.cache_append_rotary(q, k, k, b.cu, f, b.k, b.v, b.table, b.lens_t, positions=ints(pos))
    want = o8.rotate(to64(q), pos, to64(f), False)
    # (angles up to 2^36 in the oracle's long doubles, of 2^-64 or less)
    assert (bf16_excess(out, want, pair_size(to64(q), 64, False)) - 2.0 ** -27 * 8).max() <= 0


def test_frequencies_not_finite_make_their_pairs_nan():
    b = Batch(14, [2], [2], 1, 1, 64, 16)
    q, k = _new(15, 2, 1, 64), _new(16, 2, 1, 64)
    f = _freqs(32)
    f[3], f[4] = float("inf"), float("nan")
    out = fm.cache_append_rotary(q, k, k, b.cu, f, b.k, b.v, b.table, b.lens_t)
    bad = out.isnan().any(0).any(0).nonzero().flatten().tolist()
    assert bad == [3, 4, 35, 36] and out[..., bad].isnan().all()


@pytest.mark.parametrize("codes", [False, True])
def test_strides_in_place_and_rows_behind_the_last(codes):
    nodes, lens = [20, 3], [30, 8]
    b = (Batch8 if codes else Batch)(17, lens, nodes, 4, 2, 64, 16)
    T = 23
    q, k, v = _new(18, T + 4, 4, 64), _new(19, T + 4, 2, 64), _new(20, T + 4, 2, 64)
    f = _freqs(24)
    kw = dict(k_scale=b.k_scale, v_scale=b.v_scale) if codes else {}
    first = [x.clone() for x in (b.k, b.v, *kw.values())]
    out = torch.full_like(q, 7.0)
    fm.cache_append_rotary(q, k, v, b.cu, f, b.k, b.v, b.table, b.lens_t, q_out=out, **kw)
    assert (out[T:] == 7).all()
    after = [x.clone() for x in (b.k, b.v, *kw.values())]
    # again from strided inputs, the queries in place
    for x, y in zip((b.k, b.v, *kw.values()), first):
        x.copy_(y)
    wide = torch.full((T + 4, 11, 80), float("nan"), dtype=torch.bfloat16, device="cuda")
    parts = [wide[:, 0:4, 8:72], wide[:, 5:7, 16:], wide[:, 8:10, :64]]
    for p, x in zip(parts, (q, k, v)):
        p.copy_(x)
    got = fm.cache_append_rotary(*parts, b.cu, f, b.k, b.v, b.table, b.lens_t, q_out=parts[0], **kw)
    assert got.data_ptr() == parts[0].data_ptr()
    assert torch.equal(got[:T], out[:T]) and torch.equal(got[T:], q[T:])
    for x, y in zip((b.k, b.v, *kw.values()), after):
        assert torch.equal(_bytes(x), _bytes(y))


@pytest.mark.parametrize("codes", [False, True])
def test_append_skips_what_is_out_of_range(codes):
    nodes = [4, 3, 5, 2, 20]
    b = (Batch8 if codes else Batch)(21, [x + 14 for x in nodes], nodes, 2, 2, 64, 16)
    q, k = _new(22, 34, 2, 64), _new(23, 34, 2, 64)
    b.lens_t[0] = 2
    b.lens_t[1] = b.max_pages * 16 + 1
    b.table[2, 1] = -1                                  # the second page: places 16 to 18
    b.table[3, 0] = b.k.shape[0]                        # places 14, 15
    kw = dict(k_scale=b.k_scale, v_scale=b.v_scale) if codes else {}
    old = b.v.clone()
    out, st = torch.full_like(q, 7.0), _status()
    fm.cache_append_rotary(q, k, k, b.cu, _freqs(32), b.k, b.v, b.table, b.lens_t, q_out=out, status=st, **kw)
    assert fm.device_status(st) == _abi.FM_ERR_CACHE
    assert (out[:7] == 7).all() and not (out[7:] == 7).all(2).all(1).any()
    diff = (b.v.view(torch.uint8) != old.view(torch.uint8)).flatten(2).any(2).cpu().numpy()
    may = np.zeros_like(diff)
    may[b.table_np[2][0]] = True
    may[b.table_np[4][:3]] = True
    assert not diff[~may].any() and diff[b.table_np[4][1]].all() and diff[b.table_np[2][0], 14:].all()


@pytest.mark.parametrize("B", [31, 33, 1025, 2500])
@pytest.mark.parametrize("codes", [False, True])
def test_append_to_many_sequences(B, codes):
    nodes = [(0, 1, 0, 0, 3, 1, 1, 18)[(i * i) % 8] for i in range(B)]
    lens = [n + i % 20 for i, n in enumerate(nodes)]
    b = (Batch8 if codes else Batch)(24, lens, nodes, 1, 1, 64, 16)
    k, v = _new(25, sum(nodes), 1, 64), _new(26, sum(nodes), 1, 64)
    st = _status()
    if codes:
        old, olds = b.v.clone(), b.v_scale.clone()
        fm.cache_append(k, v, b.cu, b.k, b.v, b.table, b.lens_t, k_scale=b.k_scale, v_scale=b.v_scale, status=st)
        assert check_codes(b, to64(v), np.zeros(v.shape), b.v, b.v_scale, old, olds) == 0
    else:
        want = oc.append(v.view(torch.int16).cpu().numpy(), b.cu_np, b.v.view(torch.int16).cpu().numpy(), b.table_np, lens)
        fm.cache_append_rotary(None, k, v, b.cu, _freqs(8), b.k, b.v, b.table, b.lens_t, status=st)
        assert np.array_equal(b.v.view(torch.int16).cpu().numpy(), want)
    assert fm.device_status(st) == 0


# ------------------------------------------------------------------ accept
@pytest.mark.parametrize("Hkv,d,page,L", [(1, 64, 16, 1), (2, 128, 32, 3), (9, 128, 16, 2), (17, 64, 64, 1)])
def test_accept(Hkv, d, page, L):
    rng = np.random.default_rng(30)
    nodes = [1, 5, 70, 33, 0, 16, 200, 40]
    lens = [n + x for n, x in zip(nodes, (0, 3, 14, 16, 5, 31, 100, 9))]
    b = Batch8(31, lens, nodes, Hkv, Hkv, d, page)
    acc = [np.sort(rng.choice(n, int(rng.integers(0, n + 1)), replace=False)).tolist() if n else [] for n in nodes]
    acc[2], acc[7] = list(range(70)), [39]
    most = max(len(x) for x in acc) + 1
    a = np.full((len(nodes), most), 5)
    for i, x in enumerate(acc):
        a[i, :len(x)] = x
    pools, scales = [], []
    for p, s in ((b.k, b.k_scale), (b.v, b.v_scale)):
        # layers of their own scales
        e = torch.from_numpy(rng.integers(-3, 4, (L, *s.shape))).cuda()
        pools.append(torch.stack([p.view(torch.uint8)] * L).contiguous().view(F8))
        scales.append((s * torch.exp2(e.float())).contiguous())
    want = [o8.accept(acc, b.cu_np, codes64(p), s.cpu().numpy(), b.table_np, lens) for p, s in zip(pools, scales)]
    old_scales = [s.clone() for s in scales]
    one = L == 1
    st = _status()
    out = fm.cache_accept(ints(a), ints([len(x) for x in acc]), b.cu, *(p[0] if one else p for p in pools), b.table,
                          b.lens_t, k_scale=scales[0][0] if one else scales[0], v_scale=scales[1][0] if one else scales[1],
                          status=st)
    assert fm.device_status(st) == 0 and out.tolist() == want[0][2]
    for p, s, old, (wc, ws, _) in zip(pools, scales, old_scales, want):
        assert np.array_equal(s.cpu().numpy(), ws, equal_nan=True)
        assert same_codes(p, wc)


@pytest.mark.parametrize("acc,count", [([3, 2], 2), ([1, 1], 2), ([0, 5], 2), ([-1, 2], 2), ([0, 1], 6), ([0, 1], -1)])
def test_accept_leaves_sequences_with_bad_lists(acc, count):
    b = Batch8(32, [30, 25], [5, 5], 2, 2, 64, 16)
    old = b.k.clone()
    st = _status()
    a = ints([acc, [0, 3]])
    out = fm.cache_accept(a, ints([count, 2]), b.cu, b.k, b.v, b.table, b.lens_t, k_scale=b.k_scale, v_scale=b.v_scale,
                          status=st)
    assert fm.device_status(st) == _abi.FM_ERR_CACHE and out.tolist() == [30, 22]
    mine = b.table_np[0][:2]
    assert torch.equal(b.k.view(torch.uint8)[mine], old.view(torch.uint8)[mine])


def test_accept_releases_pages_and_takes_none():
    b = Batch8(33, [70, 33], [60, 20], 2, 2, 64, 16)
    ref = torch.zeros(b.k.shape[0], dtype=torch.int32, device="cuda")
    for row, n in zip(b.table_np, b.lens):
        ref[row[:-(-n // 16)].tolist()] = 1
    out = fm.cache_accept(ints([[1, 2], [0, 0]]), ints([2, 0]), b.cu, b.k, b.v, b.table, b.lens_t, ref=ref,
                          k_scale=b.k_scale, v_scale=b.v_scale)
    assert out.tolist() == [12, 13]
    held = set(b.table_np[0][:1]) | set(b.table_np[1][:1])
    assert {i for i, r in enumerate(ref.tolist()) if r} == held


# ------------------------------------------------------------------ pages
@pytest.mark.parametrize("Hkv,d,page,L", [(2, 64, 16, 2), (3, 128, 64, 1), (8, 64, 128, 3)])
def test_reserve_copies_shared_last_pages_with_their_scales(Hkv, d, page, L):
    g = torch.Generator().manual_seed(40)
    P, B, width = 12, 3, 4
    k, v = (torch.randint(0, 255, (L, P, page, Hkv, d), generator=g, dtype=torch.uint8).cuda() for _ in range(2))
    ks, vs = (torch.rand(L, P, Hkv, page // 16, generator=g).cuda() for _ in range(2))
    n = page + page // 2 + 1                        # two pages, the second shared by all rows
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    table[:, 0], table[:, 1] = 7, 4
    ref = torch.zeros(P, dtype=torch.int32, device="cuda")
    ref[7], ref[4] = 3, 3
    old = [x.clone() for x in (k, v, ks, vs)]
    fm.pages_reserve(ints([1, 0, page]), k.view(F8), v.view(F8), table, ints([n] * B), ref, k_scale=ks, v_scale=vs)
    t = table.cpu().numpy()
    assert t[1, 1] == 4 and t[0, 1] != 4 and t[2, 1] != 4
    fill = n - page
    for row in (0, 2):
        new = int(t[row, 1])
        for x, y in ((k, old[0]), (v, old[1])):
            assert torch.equal(x[:, new, :fill], y[:, 4, :fill])
        for x, y in ((ks, old[2]), (vs, old[3])):
            assert torch.equal(x[:, new, :, :-(-fill // 16)], y[:, 4, :, :-(-fill // 16)])
    kept = [p for p in range(P) if p not in (t[0, 1], t[2, 1])]
    for x, y in zip((k, v, ks, vs), old):
        assert torch.equal(x[:, kept], y[:, kept])


@pytest.mark.parametrize("Hkv,d,page,L", [(2, 64, 16, 2), (3, 128, 64, 1), (8, 64, 128, 3)])
def test_compact_moves_scales_with_pages(Hkv, d, page, L):
    g = torch.Generator().manual_seed(41)
    P = 20
    k, v = (torch.randint(0, 255, (L, P, page, Hkv, d), generator=g, dtype=torch.uint8).cuda() for _ in range(2))
    ks, vs = (torch.rand(L, P, Hkv, page // 16, generator=g).cuda() for _ in range(2))
    rows = [[19, 2, 11], [5, 17], [0]]
    table = torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    ref = torch.zeros(P, dtype=torch.int32, device="cuda")
    for b, r in enumerate(rows):
        table[b, :len(r)] = ints(r)
        ref[r] = 1
    new, want_ref, moves, live = oc.compact(rows, ref.tolist())
    old = [x.clone() for x in (k, v, ks, vs)]
    n = fm.pages_compact(k.view(F8), v.view(F8), table, ints([len(r) * page for r in rows]), ref, k_scale=ks, v_scale=vs)
    assert int(n) == live and ref.tolist() == want_ref
    to = dict(moves)
    for b, r in enumerate(new):
        assert table[b, :len(r)].tolist() == r
    for p in sum(rows, []):
        for x, y in zip((k, v, ks, vs), old):
            assert torch.equal(x[:, to.get(p, p)], y[:, p])


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("H,Hkv,d,page", [(4, 2, 64, 16), (8, 2, 128, 32)])
def test_drafting_and_verifying_equals_decoding_token_by_token(H, Hkv, d, page, codes):
    """A prompt, then drafted trees whose accepted nodes are kept, with rotated queries and keys; and the
    same tokens one by one.  A token's query, key and value are functions of its name."""
    g = torch.Generator().manual_seed(50)
    words, layers = 40, 2
    emb = [torch.randn(layers, words, n, d, generator=g).to(torch.bfloat16).cuda() for n in (H, Hkv, Hkv)]
    f, scale = _freqs(d // 4), d ** -0.5
    rng = np.random.default_rng(51)
    prompts = [rng.integers(0, words, n).tolist() for n in (21, 5)]

    class Cache:
        def __init__(self):
            dt = F8 if codes else torch.bfloat16
            self.k, self.v = (torch.zeros(layers, 30, page, Hkv, d, device="cuda").to(dt) for _ in range(2))
            self.kw = dict(k_scale=fm.cache_scales(self.k), v_scale=fm.cache_scales(self.v)) if codes else {}
            self.table = torch.full((2, 10), -1, dtype=torch.int32, device="cuda")
            self.lens, self.ref = ints([0, 0]), torch.zeros(30, dtype=torch.int32, device="cuda")

        def layer(self, i):
            return {n: x[i] for n, x in self.kw.items()}

        def step(self, tokens, parents=None, depth=None):
            n = [len(t) for t in tokens]
            fm.pages_reserve(ints(n), self.k, self.v, self.table, self.lens, self.ref, **self.kw)
            cu = ints(np.concatenate([[0], np.cumsum(n)]))
            flat = torch.tensor(sum(tokens, [])).cuda()
            pos = None
            if depth is not None:
                pos = ints(np.concatenate([int(x) - m + np.array(dd) for x, m, dd in zip(self.lens.tolist(), n, depth)]))
            out = []
            for i in range(layers):
                q, k, v = (e[i][flat] for e in emb)
                q = fm.cache_append_rotary(q, k, v, cu, f, self.k[i], self.v[i], self.table, self.lens, positions=pos,
                                           **self.layer(i))
                par = None if parents is None else ints(sum(parents, []))
                out.append(fm.tree_forward(q, self.k[i], self.v[i], self.table, self.lens, cu, scale, parents=par,
                                           max_nodes=max(n), **self.layer(i))[0])
            return out, cu

    tree, plain = Cache(), Cache()
    a, _ = tree.step(prompts)
    b, _ = plain.step(prompts)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    for turn in range(4):
        nodes = [rng.integers(0, words, 9).tolist() for _ in range(2)]
        parents = [[-1, 0, 0, 1, 1, 2, 3, 6, 5], [-1, 0, 1, 1, 0, 4, 5, 6, 2]]
        depth = []
        for p in parents:
            dd = []
            for x in p:
                dd.append(0 if x < 0 else dd[x] + 1)
            depth.append(dd)
        paths = [[0, 1, 3, 6, 7], [0, 4, 5]] if turn % 2 else [[0, 2, 5], [0, 1, 2, 8]]
        drafted, cu = tree.step(nodes, parents, depth)
        most = max(len(p) for p in paths)
        tree.lens = fm.cache_accept(ints([p + [0] * (most - len(p)) for p in paths]), ints([len(p) for p in paths]), cu,
                                    tree.k, tree.v, tree.table, tree.lens, ref=tree.ref, **tree.kw)
        for i in range(most):
            tokens = [[nodes[s][p[i]]] if i < len(p) else [] for s, p in enumerate(paths)]
            single, c2 = plain.step(tokens)
            for s, p in enumerate(paths):
                if i < len(p):
                    row, at = int(cu[s]) + p[i], int(c2[s])
                    for x, y in zip(drafted, single):
                        # codes: other nodes of a block may have grown its scale, which rounds again (two
                        # roundings of 2^-4 of a value between the caches); bf16: the same cache, other orders of sums
                        tol = 0.25 if codes else 0.02
                        assert (x[row].float() - y[at].float()).abs().max() < tol
        assert tree.lens.tolist() == plain.lens.tolist()


def test_captured_append_replays_with_growing_lengths():
    b = Batch8(60, [64, 64], [1, 1], 2, 2, 64, 16)
    q, k, v = _new(61, 2, 4, 64), _new(62, 2, 2, 64), _new(63, 2, 2, 64)
    f, out = _freqs(32), torch.empty(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    start = [x.clone() for x in (b.k, b.v, b.k_scale, b.v_scale)]

    def call():
        fm.cache_append_rotary(q, k, v, b.cu, f, b.k, b.v, b.table, b.lens_t, q_out=out, k_scale=b.k_scale,
                               v_scale=b.v_scale)

    def run(how):
        for x, y in zip((b.k, b.v, b.k_scale, b.v_scale), start):
            x.copy_(y)
        got = []
        for n in range(40, 60):
            b.lens_t.fill_(n)
            how()
            got.append(out.clone())
        torch.cuda.synchronize()
        return [_bytes(x).clone() for x in (b.k, b.v, b.k_scale, b.v_scale)], got

    want = run(call)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    got = run(g.replay)
    for x, y in zip(got[0] + got[1], want[0] + want[1]):
        assert torch.equal(x, y)


def test_on_another_stream():
    b = Batch8(64, [50, 20], [3, 20], 2, 2, 64, 16)
    q, k = _new(65, 23, 2, 64), _new(66, 23, 2, 64)
    f = _freqs(32)
    b2 = Batch8(64, [50, 20], [3, 20], 2, 2, 64, 16)
    want = fm.cache_append_rotary(q, k, k, b.cu, f, b.k, b.v, b.table, b.lens_t, k_scale=b.k_scale, v_scale=b.v_scale)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = fm.cache_append_rotary(q, k, k, b2.cu, f, b2.k, b2.v, b2.table, b2.lens_t, k_scale=b2.k_scale,
                                 v_scale=b2.v_scale, stream=s)
    none = fm.cache_append_rotary(None, k, k, b2.cu, f, b2.k, b2.v, b2.table, b2.lens_t, k_scale=b2.k_scale,
                                  v_scale=b2.v_scale, stream=s)
    s.synchronize()
    assert none is None and torch.equal(got, want)
    assert torch.equal(b.k.view(torch.uint8), b2.k.view(torch.uint8))


def test_the_binding_refuses_wrong_types_and_shapes():
    b = Batch8(70, [20], [4], 4, 2, 64, 32)
    k = _new(71, 4, 2, 64)
    f = _freqs(32)
    good = dict(k_scale=b.k_scale, v_scale=b.v_scale)
    bf16 = torch.zeros(b.k.shape, dtype=torch.bfloat16, device="cuda")
    bad = [
        dict(args=(k, k, b.cu, b.k, b.v), kw={}),                                        # codes without scales
        dict(args=(k, k, b.cu, bf16, bf16), kw=good),                                    # scales of bf16 pools
        dict(args=(k, k, b.cu, b.k, b.v), kw=dict(k_scale=b.k_scale)),
        dict(args=(k, k, b.cu, b.k, b.v), kw=dict(k_scale=b.k_scale, v_scale=b.v_scale[:-1])),
        dict(args=(k, k, b.cu, b.k, b.v), kw=dict(k_scale=b.k_scale, v_scale=b.v_scale.double())),
        dict(args=(k, k, b.cu, b.k, b.v), kw=dict(k_scale=b.k_scale, v_scale=b.v_scale.cpu())),
        dict(args=(k, k, b.cu, b.k, b.v), kw=dict(k_scale=b.k_scale, v_scale=b.v_scale.repeat(1, 1, 2)[:, :, ::2])),
        dict(args=(k.float(), k, b.cu, b.k, b.v), kw=good),
        dict(args=(k[:3], k, b.cu, b.k, b.v), kw=good),
    ]
    for c in bad:
        with pytest.raises(ValueError):
            fm.cache_append(*c["args"], b.table, b.lens_t, **c["kw"])
    q = _new(72, 4, 4, 64)
    rotary = lambda q=q, f=f, **kw: fm.cache_append_rotary(q, k, k, b.cu, f, b.k, b.v, b.table, b.lens_t, **good, **kw)  # noqa: E731
    for call in (lambda: rotary(q=q[:3]), lambda: rotary(q=q[..., :32]), lambda: rotary(f=f[:12]),
                 lambda: rotary(f=_freqs(40)), lambda: rotary(f=f.double()), lambda: rotary(f=None),
                 lambda: rotary(positions=ints([0, 1, 2])), lambda: rotary(positions=b.cu.long()),
                 lambda: rotary(q_out=q[:3]), lambda: rotary(q_out=q.float()),
                 lambda: rotary(stream=torch.cuda.Stream(), positions=b.cu.cpu()),
                 lambda: fm.tree_forward(q, b.k, b.v, b.table, b.lens_t, b.cu, 0.1),
                 lambda: fm.tree_forward(q, bf16, bf16, b.table, b.lens_t, b.cu, 0.1, **good)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(fm.FMError):
        rotary(q=_new(73, 4, 3, 64))
