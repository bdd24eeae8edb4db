"""Appending to blocks of e4m3 codes that have tokens, by groups of threads of all sizes: within a warp, a
warp, and several, of which some find that their head's scale grows and others not."""
import numpy as np
import pytest
import torch

import masked_attention_bound_gb300 as fm
from cache8_cases import Batch8
from oracle.attention import to64
from test_gpu_cache8_pages import _new, _status, check_codes

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 8, 9, 15])
@pytest.mark.parametrize("Hkv", [1, 8, 11])
@pytest.mark.parametrize("by", ["token", "head"])
def test_scales_of_some_heads_grow(d, n, Hkv, by):
    """Sizes from 2^-6 to 2^6 by token and head (of three tokens one is large), or by sequence and head."""
    B = 40
    b = Batch8(80, [n + 1 + i % (16 - n) for i in range(B)], [n] * B, Hkv, Hkv, d, 16)
    k, v = _new(81, B * n, Hkv, d), _new(82, B * n, Hkv, d)
    for i, x in enumerate((k, v)):
        e = torch.tensor([(7 * h + 3 * (s if by == "token" else s // n) + i) % 5 - 2
                          for s in range(B * n) for h in range(Hkv)], device="cuda")
        x *= torch.exp2(3.0 * e.view(B * n, Hkv, 1)).to(torch.bfloat16)
    old = [x.clone() for x in (b.k, b.k_scale, b.v, b.v_scale)]
    st = _status()
    fm.cache_append(k, v, b.cu, b.k, b.v, b.table, b.lens_t, k_scale=b.k_scale, v_scale=b.v_scale, status=st)
    assert fm.device_status(st) == 0
    z = np.zeros(k.shape)
    assert check_codes(b, to64(k), z, b.k, b.k_scale, old[0], old[1]) == 0
    assert check_codes(b, to64(v), z, b.v, b.v_scale, old[2], old[3]) == 0
    grown = b.k_scale != old[1]
    assert grown.any() and (by == "token" or (~grown).any())
