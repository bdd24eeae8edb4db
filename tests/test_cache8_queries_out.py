"""Where the append with rotation may write its queries: refusals of overlaps on the host and without a
GPU, and slices of one buffer, which do not overlap."""
import ctypes

import numpy as np
import pytest
import torch

import masked_attention_bound_gb300 as fm
from masked_attention_bound_gb300 import _abi
from test_cache8_abi import L, _append, _cache, _rotary  # noqa: F401

Q = 1 << 29
INVALID = _abi.FM_ERR_INVALID


# bytes from q (5 tokens of 4 heads of 64, strides 256 and 64) and strides of q_out
@pytest.mark.parametrize("off,strides", [
    (128, (256, 64)), (-128, (256, 64)), (512, (256, 64)), (-4 * 512, (256, 64)), (112, (256, 64)), (5 * 512 - 16, (256, 64)),
    (0, (512, 64)), (0, (256, 72)), (0, (64, 256)), (512, (320, 64)), (-16, (256, 64))])
@pytest.mark.parametrize("codes", [True, False])
def test_queries_that_overlap_are_refused(L, off, strides, codes):  # noqa: F811
    R = _rotary(q=Q, q_out=Q + off)
    R.o_stride[:] = strides
    assert _append(L, R=R, codes=codes) == INVALID


@pytest.mark.parametrize("off", [(2 * (640 * t + 64 * h)) for t in (-4, -1, 0, 1, 4) for h in (-3, 0, 3)] + [-16, 16, 640])
def test_overlaps_within_one_buffer_are_refused(L, off):  # noqa: F811
    """Tokens of ten heads, of which q and q_out are four each."""
    if off == 0:
        off = 2 * 64
    R = _rotary(q=Q, q_out=Q + off)
    R.q_stride[:] = R.o_stride[:] = (640, 64)
    assert _append(L, R=R) == INVALID


@pytest.mark.parametrize("which", ["a0", "a1"])
@pytest.mark.parametrize("off", [0, 16, 256, -1024, 4 * 512])
def test_queries_over_new_keys_or_values_are_refused(L, which, off):  # noqa: F811
    R = _rotary(q=Q, q_out=(1 << 31) + off)
    assert _append(L, R=R, ks=(256, 64), vs=(256, 64), **{which: ctypes.c_void_p(1 << 31)}) == INVALID


def test_many_heads_are_looked_through_at_once(L):  # noqa: F811
    """Spans that cross with other head strides are refused without a look at each pair of heads."""
    C = _cache(Hkv=40000)
    R = _rotary(H=40000, q=1 << 40, q_out=(1 << 40) + 128)
    R.q_stride[:] = (40000 * 128, 128)
    R.o_stride[:] = (40000 * 128, 256)
    assert _append(L, C=C, R=R, ks=(40000 * 64, 64), vs=(40000 * 64, 64)) == INVALID
    R.o_stride[:] = (40000 * 128, 128)
    R.q_out = (1 << 40) + 16
    assert _append(L, C=C, R=R, ks=(40000 * 64, 64), vs=(40000 * 64, 64)) == INVALID


@pytest.mark.gpu
@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("T", [1, 23])
@pytest.mark.parametrize("step", [1, 2])
def test_slices_of_one_buffer(T, codes, step):
    """q, k, v and q_out side by side in each token (heads one after the other, and every second one), in
    place, and one after the other in one allocation."""
    H, Hkv, d, page = 4, 2, 64, 16
    g = torch.Generator().manual_seed(1)
    x = torch.randn(T, 2 * H + 2 * Hkv, step, d, generator=g).to(torch.bfloat16).cuda()
    heads = x[:, :, 0]
    q, k, v, out = heads[:, :H], heads[:, H:H + Hkv], heads[:, H + Hkv:H + 2 * Hkv], heads[:, H + 2 * Hkv:]
    dt = torch.float8_e4m3fn if codes else torch.bfloat16
    pools = [torch.zeros(3, page, Hkv, d, device="cuda").to(dt) for _ in range(2)]
    kw = dict(k_scale=fm.cache_scales(pools[0]), v_scale=fm.cache_scales(pools[1])) if codes else {}
    table = torch.tensor([[2, 0]], dtype=torch.int32, device="cuda")
    lens, cu = (torch.tensor(n, dtype=torch.int32, device="cuda") for n in ([T + 3], [0, T]))
    freqs = torch.tensor(10.0 ** -np.arange(16.0), dtype=torch.float32, device="cuda")

    def call(q, out):
        return fm.cache_append_rotary(q, k, v, cu, freqs, *pools, table, lens, q_out=out, **kw)

    want = call(q.clone(), None)
    got = call(q, out)
    assert got.data_ptr() == out.data_ptr() and torch.equal(out, want)
    both = torch.cat([q, q]).contiguous()
    call(both[:T], both[T:])
    assert torch.equal(both[:T], q) and torch.equal(both[T:], want)
    if step == 2:                          # heads between heads, the token stride the same
        pairs = x[:, :H]
        pairs[:, :, 0] = q
        call(pairs[:, :, 0], pairs[:, :, 1])
        assert torch.equal(pairs[:, :, 1], want)
    rows = torch.empty(H, 2, T, d, dtype=torch.bfloat16, device="cuda").permute(1, 2, 0, 3)    # heads before tokens
    rows[0] = q
    call(rows[0], rows[1])
    assert torch.equal(rows[0], q) and torch.equal(rows[1], want)
    call(q, q)
    assert torch.equal(q, want)
    with pytest.raises(fm.FMError):
        call(heads[:, 1:1 + H], heads[:, :H])
