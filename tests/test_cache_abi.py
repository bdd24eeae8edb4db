"""Refusals of the paged-cache entry points, on the host and without a GPU."""
import ctypes
import itertools

import pytest
import torch

import masked_attention_bound_gb300 as fm
from masked_attention_bound_gb300 import _abi, build, cache

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


def _desc(**kw):
    D = _abi.FmTreeDesc()
    D.H, D.total, D.max_nodes = 4, 5, 3
    D.q_stride[:] = D.o_stride[:] = (256, 64)
    for name, value in kw.items():
        setattr(D, name, value)
    return D


def _p(i):
    """A pointer that is never followed: every call here is refused on the host."""
    return ctypes.c_void_p((i + 1) << 28)


def _tree(L, C, D, q=0, parents=8, scale=0.1, ws=9, ws_bytes=1 << 30, **null):
    args = [_p(i) for i in range(7)]
    for name, value in null.items():
        args[int(name[1:])] = value
    return L.fm_tree_fwd(ctypes.byref(C), ctypes.byref(D), args[0], args[1], args[2], args[3], args[4], args[5],
                         None if parents is None else _p(parents), scale, args[6], _p(7),
                         None if ws is None else ctypes.c_void_p(ws), ws_bytes, None, None)


BAD_CACHE = [("B", 0, INVALID), ("Hkv", 0, INVALID), ("d", 96, UNSUPPORTED), ("page_size", 8, UNSUPPORTED),
             ("page_size", 48, UNSUPPORTED), ("page_size", 256, UNSUPPORTED), ("n_pages", 0, INVALID),
             ("n_pages", (1 << 24) + 1, UNSUPPORTED), ("max_pages", 0, INVALID),
             ("max_pages", (1 << 26) + 1, UNSUPPORTED), ("layers", 0, INVALID), ("B", 1 << 30, UNSUPPORTED), ("Hkv", 1 << 16, UNSUPPORTED)]


@pytest.mark.parametrize("field,value,code", BAD_CACHE)
def test_bad_caches(L, field, value, code):
    C = _cache(**{field: value})
    nul, st = ctypes.c_void_p(0), (ctypes.c_int64 * 2)(128, 64)
    assert _tree(L, C, _desc()) == code
    assert L.fm_tree_workspace_size(ctypes.byref(C), ctypes.byref(_desc())) == 0
    assert L.fm_cache_append(ctypes.byref(C), _p(0), _p(1), st, st, _p(2), 3, _p(3), _p(4), _p(5), _p(6), None,
                             None) == code
    assert L.fm_cache_accept(ctypes.byref(C), _p(0), 1, _p(1), _p(2), _p(3), _p(4), _p(5), _p(6), _p(7), nul, None,
                             None) == code
    assert L.fm_pages_reserve(ctypes.byref(C), _p(0), _p(1), _p(2), _p(3), _p(4), _p(5), _p(3), _p(4), _p(5), _p(6),
                              _p(7), 1 << 40, None, None) == code
    assert L.fm_pages_compact(ctypes.byref(C), _p(1), _p(2), _p(3), _p(4), _p(5), _p(3), _p(5), _p(6), _p(7), 1 << 40,
                              None, None) == code
    if field not in ("Hkv", "d", "layers"):
        assert L.fm_pages_fork(ctypes.byref(C), _p(0), _p(1), _p(2), _p(3), _p(4), _p(5), _p(3), None, None) == code
        assert L.fm_pages_workspace_size(ctypes.byref(C)) == 0


@pytest.mark.parametrize("which", ["k_stride", "v_stride"])
@pytest.mark.parametrize("i,value", [(0, 0), (1, 2044), (2, -128), (3, 1 << 36)])
def test_bad_pool_strides(L, which, i, value):
    C = _cache()
    getattr(C, which)[i] = value
    assert _tree(L, C, _desc()) == INVALID


@pytest.mark.parametrize("field,value,code", [("H", 0, INVALID), ("H", 5, INVALID), ("total", 0, INVALID),
                                              ("max_nodes", 0, INVALID), ("max_nodes", 257, UNSUPPORTED),
                                              ("total", 1 << 29, UNSUPPORTED)])
def test_bad_tree_descriptions(L, field, value, code):
    assert _tree(L, _cache(), _desc(**{field: value})) == code


@pytest.mark.parametrize("i,code", [(i, INVALID) for i in range(7)])
def test_null_pointers(L, i, code):
    assert _tree(L, _cache(), _desc(), **{f"a{i}": None}) == code


@pytest.mark.parametrize("i", [0, 1, 2, 6])
def test_unaligned_tensors(L, i):
    assert _tree(L, _cache(), _desc(), **{f"a{i}": ctypes.c_void_p((1 << 28) + 8)}) == INVALID


@pytest.mark.parametrize("scale", [0.0, -1.0, float("nan"), float("inf"), 1e-39, 3e38])
def test_bad_scales(L, scale):
    assert _tree(L, _cache(), _desc(), scale=scale) == INVALID


def test_workspaces(L):
    C, D = _cache(), _desc()
    n = L.fm_tree_workspace_size(ctypes.byref(C), ctypes.byref(D))
    assert n > 0
    assert _tree(L, C, D, ws=None) == WORKSPACE
    assert _tree(L, C, D, ws=(1 << 30) + 128) == WORKSPACE
    assert _tree(L, C, D, ws=1 << 30, ws_bytes=n - 1) == WORKSPACE
    m = L.fm_pages_workspace_size(ctypes.byref(C))
    for ws, size in ((None, m), ((1 << 30) + 4, m), (1 << 30, m - 1)):
        assert L.fm_pages_reserve(ctypes.byref(C), _p(0), _p(1), _p(2), _p(3), _p(4), _p(5), _p(3), _p(4), _p(5),
                                  _p(6), ws, size, None, None) == WORKSPACE
        assert L.fm_pages_compact(ctypes.byref(C), _p(1), _p(2), _p(3), _p(4), _p(5), _p(3), _p(5), _p(6), ws, size,
                                  None, None) == WORKSPACE


def test_overlapping_outputs(L):
    C = _cache()
    off = lambda i: ctypes.c_void_p(((i + 1) << 28) + 4)  # noqa: E731
    # fork: table and lens need new arrays
    for t, ln, rf in ((_p(1), _p(5), _p(3)), (_p(4), _p(2), _p(3)), (off(1), _p(5), _p(3)), (_p(4), off(2), _p(3)),
                      (_p(4), _p(5), off(3))):
        assert L.fm_pages_fork(ctypes.byref(C), _p(0), _p(1), _p(2), _p(3), t, ln, rf, None, None) == INVALID
    for t, ln, rf in ((off(3), _p(4), _p(5)), (_p(3), off(4), _p(5)), (_p(3), _p(4), off(5))):
        assert L.fm_pages_reserve(ctypes.byref(C), _p(0), _p(1), _p(2), _p(3), _p(4), _p(5), t, ln, rf, _p(6), _p(7),
                                  1 << 40, None, None) == INVALID
    assert L.fm_cache_accept(ctypes.byref(C), _p(0), 1, _p(1), _p(2), _p(3), _p(4), _p(5), _p(6), _p(6), None, None,
                             None) == INVALID
    assert L.fm_cache_accept(ctypes.byref(C), _p(0), 0, _p(1), _p(2), _p(3), _p(4), _p(5), _p(6), _p(7), None, None,
                             None) == INVALID


def test_append_refusals(L):
    C, good = _cache(), (ctypes.c_int64 * 2)(128, 64)
    call = lambda ks=good, total=3, k=_p(0): L.fm_cache_append(  # noqa: E731
        ctypes.byref(C), k, _p(1), ks, good, _p(2), total, _p(3), _p(4), _p(5), _p(6), None, None)
    assert call(total=0) == INVALID and call(k=ctypes.c_void_p(0)) == INVALID
    assert call(k=ctypes.c_void_p(8)) == INVALID
    for i, x in ((0, 0), (0, 4), (1, -8)):
        s = (ctypes.c_int64 * 2)(128, 64)
        s[i] = x
        assert call(ks=s) == INVALID


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    t = torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError):
        cache.make_cache(k, k, t)
    with pytest.raises(ValueError):
        cache.make_cache(k[0], k[0], t)
    with pytest.raises(ValueError):
        cache.make_cache(k, k[:2], t)
    with pytest.raises(ValueError):
        fm.tree_forward(k[:, 0], k, k, t, t[:, 0], t[0], 0.1)
    with pytest.raises(ValueError):
        fm.pages_fork(t[:, 0], 16, t, t[:, 0], t[0])


def test_status_names(L):
    for c in (_abi.FM_ERR_CACHE, _abi.FM_ERR_PAGES):
        assert len(_abi.status_string(c)) > 5 and _abi.STATUS_NAMES[c].startswith("FM_ERR")


def test_a_workspace_of_the_attention_serves_every_smaller_description(L):
    """No kernel that fewer nodes, tokens or a narrower table choose needs more than the size given for
    more of them."""
    for d, G, B in itertools.product((64, 128), (1, 3, 4, 8, 40, 300), (1, 2, 40, 1000)):
        need = {}
        for width, total, nodes in itertools.product((4, 20, 41, 200), (1, 4, 20, 128, 129, 600),
                                                     (1, 2, 3, 4, 5, 16, 17, 31, 32, 33, 40, 63, 64, 65, 128, 200, 256)):
            C = _cache(d=d, B=B, max_pages=width)
            D = _desc(H=2 * G, total=total, max_nodes=nodes)
            need[width, total, nodes] = L.fm_tree_workspace_size(ctypes.byref(C), ctypes.byref(D))
        assert min(need.values()) > 0
        for size, n in need.items():
            for axis in range(3):        # the next smaller value of one axis
                less = max((x for x in need if all(x[a] == size[a] or a == axis for a in range(3))
                            and x[axis] < size[axis]), key=lambda x: x[axis], default=size)
                assert need[less] <= n, (d, G, B, less, size)
