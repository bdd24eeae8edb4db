"""Refusals of the entry points of the cache of e4m3 codes and of the append with rotation, on the host
and without a GPU."""
import ctypes

import pytest
import torch

import masked_attention_bound_gb300 as fm
from masked_attention_bound_gb300 import _abi, build

INVALID, UNSUPPORTED, WORKSPACE = _abi.FM_ERR_INVALID, _abi.FM_ERR_UNSUPPORTED, _abi.FM_ERR_WORKSPACE


@pytest.fixture(scope="module")
def L():
    build.build()
    return _abi.lib()


def _cache(**kw):
    C = _abi.FmCache()
    C.B, C.Hkv, C.d, C.page_size, C.n_pages, C.max_pages, C.layers = 2, 2, 64, 16, 10, 4, 1
    C.k_stride[:] = C.v_stride[:] = (20480, 2048, 128, 64)
    for name, value in kw.items():
        setattr(C, name, value)
    return C


def _p(i):
    """A pointer that is never followed: every call here is refused on the host."""
    return ctypes.c_void_p((i + 1) << 28)


def _rotary(**kw):
    R = _abi.FmRotary()
    R.rot, R.interleaved, R.freqs, R.positions, R.H = 32, 0, 1 << 28, 0, 4
    R.q, R.q_out = 1 << 29, 1 << 30
    R.q_stride[:] = R.o_stride[:] = (256, 64)
    for name, value in kw.items():
        setattr(R, name, value)
    return R


def _append(L, C=None, R=None, total=5, ks=(128, 64), vs=(128, 64), codes=True, **null):
    args = [_p(i) for i in range(9)]    # k, v, cu, k_pool, v_pool, k_scale, v_scale, table, lens
    if not codes:
        args[5] = args[6] = None
    for name, value in null.items():
        args[int(name[1:])] = value
    st = [(ctypes.c_int64 * 2)(*s) for s in (ks, vs)]
    R = _rotary() if R is None else R
    return L.fm_cache_append_rotary(ctypes.byref(C or _cache()), ctypes.byref(R), args[0], args[1], *st, args[2], total,
                                    *args[3:], None, None)


def _tree(L, C, scale=0.1, ws=1 << 28, ws_bytes=1 << 30, max_nodes=3, **null):
    D = _abi.FmTreeDesc()
    D.H, D.total, D.max_nodes = 4, 5, max_nodes
    D.q_stride[:] = D.o_stride[:] = (256, 64)
    args = [_p(i) for i in range(10)]   # q, k, v, ks, vs, table, lens, cu, o, lse
    for name, value in null.items():
        args[int(name[1:])] = value
    return L.fm_tree_fwd_fp8(ctypes.byref(C), ctypes.byref(D), *args[:8], None, scale, args[8], args[9],
                             ctypes.c_void_p(ws), ws_bytes, None, None)


def _accept(L, C, lens_out=_p(9), most=1, **null):
    args = [_p(i) for i in range(9)]    # accept, n, cu, k, v, ks, vs, table, lens
    for name, value in null.items():
        args[int(name[1:])] = value
    return L.fm_cache_accept_fp8(ctypes.byref(C), args[0], most, *args[1:], lens_out, None, None, None)


def _reserve(L, C, ws=1 << 28, ws_bytes=1 << 40, **null):
    args = [_p(i) for i in range(8)]    # grow, k, v, ks, vs, table, lens, ref
    for name, value in null.items():
        args[int(name[1:])] = value
    return L.fm_pages_reserve_fp8(ctypes.byref(C), *args, args[5], args[6], args[7], _p(8), ctypes.c_void_p(ws),
                                  ws_bytes, None, None)


def _compact(L, C, ws=1 << 28, ws_bytes=1 << 40, **null):
    args = [_p(i) for i in range(7)]    # k, v, ks, vs, table, lens, ref
    for name, value in null.items():
        args[int(name[1:])] = value
    return L.fm_pages_compact_fp8(ctypes.byref(C), *args, args[4], args[6], _p(7), ctypes.c_void_p(ws), ws_bytes,
                                  None, None)


@pytest.mark.parametrize("field,value,code", [
    ("B", 0, INVALID), ("Hkv", 0, INVALID), ("d", 96, UNSUPPORTED), ("page_size", 8, UNSUPPORTED),
    ("page_size", 48, UNSUPPORTED), ("page_size", 256, UNSUPPORTED), ("n_pages", 0, INVALID),
    ("n_pages", (1 << 24) + 1, UNSUPPORTED), ("max_pages", 0, INVALID), ("max_pages", (1 << 26) + 1, UNSUPPORTED),
    ("layers", 0, INVALID), ("B", 1 << 30, UNSUPPORTED), ("Hkv", 1 << 16, UNSUPPORTED)])
def test_bad_caches(L, field, value, code):
    C = _cache(**{field: value})
    R = _rotary(H=0)
    assert _append(L, C, R) == code and _append(L, C, R, codes=False) == code
    assert _tree(L, C) == code and _accept(L, C) == code and _reserve(L, C) == code and _compact(L, C) == code


@pytest.mark.parametrize("which", ["k_stride", "v_stride"])
@pytest.mark.parametrize("i,value", [(0, 0), (1, 2040), (2, -128), (3, 1 << 36), (2, 136)])
def test_bad_pool_strides(L, which, i, value):
    C = _cache()
    getattr(C, which)[i] = value
    assert {_append(L, C), _tree(L, C), _accept(L, C), _reserve(L, C), _compact(L, C)} == {INVALID}


def test_null_and_unaligned_pointers(L):
    C = _cache()
    for i in range(9):
        assert _append(L, **{f"a{i}": None}) == INVALID
        assert _accept(L, C, **{f"a{i}": None}) == INVALID
    for i in range(10):
        assert _tree(L, C, **{f"a{i}": None}) == INVALID
    for i in range(8):
        assert _reserve(L, C, **{f"a{i}": None}) == INVALID
    for i in range(7):
        assert _compact(L, C, **{f"a{i}": None}) == INVALID
    odd = ctypes.c_void_p((1 << 28) + 8)
    for i in (0, 1, 3, 4):
        assert _append(L, **{f"a{i}": odd}) == INVALID and _append(L, codes=False, **{f"a{i}": odd}) == INVALID
    for i in (0, 1, 2, 8):
        assert _tree(L, C, **{f"a{i}": odd}) == INVALID
    by2 = ctypes.c_void_p((1 << 28) + 2)
    for i in (3, 4):
        assert _tree(L, C, **{f"a{i}": by2}) == INVALID


@pytest.mark.parametrize("field,value,code", [
    ("rot", -16, INVALID), ("rot", 8, INVALID), ("rot", 40, INVALID), ("rot", 80, INVALID), ("freqs", 0, INVALID),
    ("freqs", 2, INVALID), ("H", -2, INVALID), ("H", 3, INVALID), ("q", 0, INVALID), ("q", 8, INVALID),
    ("q_out", 0, INVALID), ("q_out", 24, INVALID), ("H", 1 << 29, UNSUPPORTED)])
def test_bad_rotations(L, field, value, code):
    assert _append(L, R=_rotary(**{field: value})) == code
    assert _append(L, R=_rotary(**{field: value}), codes=False) == code


@pytest.mark.parametrize("which", ["q_stride", "o_stride"])
@pytest.mark.parametrize("i,value", [(0, 0), (1, 60), (0, -256), (1, 1 << 36)])
def test_bad_query_strides(L, which, i, value):
    R = _rotary()
    getattr(R, which)[i] = value
    assert _append(L, R=R) == INVALID


def test_bad_appends(L):
    assert _append(L, total=0) == INVALID and _append(L, total=1 << 29) == UNSUPPORTED
    for s in ((0, 64), (124, 64), (128, -64), (128, 1 << 36)):
        assert _append(L, ks=s) == INVALID and _append(L, vs=s) == INVALID
    # blocks of the batch are counted in 31 bits
    assert _append(L, _cache(B=(1 << 30) + 8, max_pages=1, Hkv=1), _rotary(H=0)) == UNSUPPORTED
    # one scale without the other
    assert _append(L, a5=None) == INVALID and _append(L, codes=False, a6=_p(6)) == INVALID


def test_bad_attention(L):
    for s in (0.0, -1.0, float("nan"), float("inf"), 1e-39, 3e38):
        assert _tree(L, _cache(), scale=s) == INVALID
    for ws, size in ((0, 1 << 30), ((1 << 28) + 128, 1 << 30), (1 << 28, 100)):
        assert _tree(L, _cache(), ws=ws, ws_bytes=size) == WORKSPACE
    assert _tree(L, _cache(), max_nodes=0) == INVALID


def test_bad_page_calls(L):
    C = _cache()
    assert _accept(L, C, most=0) == INVALID and _accept(L, C, lens_out=_p(8)) == INVALID
    for f in (_reserve, _compact):
        assert f(L, C, ws=0) == WORKSPACE and f(L, C, ws=(1 << 28) + 4) == WORKSPACE and f(L, C, ws_bytes=8) == WORKSPACE


def test_the_binding_refuses_before_it_looks_at_a_device():
    k = torch.zeros(4, 16, 2, 64).to(torch.float8_e4m3fn)
    t = torch.zeros(2, 3, dtype=torch.int32)
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    s = fm.cache_scales(k)
    assert s.shape == (4, 2, 1) and s.dtype == torch.float32
    assert fm.cache_scales(torch.zeros(3, 4, 64, 2, 64)).shape == (3, 4, 2, 4)
    with pytest.raises(ValueError):
        fm.cache_scales(k[0])
    with pytest.raises(ValueError):
        fm.cache_append_rotary(x, x, x, t[0], torch.ones(8), k, k, t, t[:, 0], k_scale=s, v_scale=s)
    with pytest.raises(ValueError):
        fm.cache_append(x, x, t[0], k, k, t, t[:, 0], k_scale=s, v_scale=s)
    with pytest.raises(ValueError):
        fm.cache_accept(t, t[:, 0], t[0], k, k, t, t[:, 0], k_scale=s, v_scale=s)
    with pytest.raises(TypeError):
        fm.cache.lib(), fm.cache._load().append_rotary(x)
