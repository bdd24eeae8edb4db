"""The arithmetic by which the tcgen05 kernels over e4m3 codes hold a bf16 query: a row's elements times a
power of two that brings the largest to [2^7, 2^8), as the nearest e4m3 code and the nearest e5m2 code of
the rest."""
import torch


def test_two_parts_are_the_value():
    # every positive bf16 below 2^8
    x = torch.arange(((127 + 8) << 7), dtype=torch.int32).to(torch.int16).view(torch.bfloat16).to(torch.float16)
    exact = torch.arange(((127 + 8) << 7), dtype=torch.int32).to(torch.int16).view(torch.bfloat16).double()
    hi = x.float().to(torch.float8_e4m3fn).to(torch.float16)
    rest = x - hi
    assert torch.equal(rest.double(), x.double() - hi.double())        # the difference is exact in f16
    lo = rest.float().to(torch.float8_e5m2)
    off = (hi.double() + lo.double() - exact).abs()
    assert hi.isfinite().all() and (off[exact >= 2.0 ** -6] == 0).all()
    # below: half a step of e5m2 (2^-13 in its binade) of a rest of 2^-10 at most; 2^-21 of the row's largest
    assert off.max() <= 2.0 ** -14
