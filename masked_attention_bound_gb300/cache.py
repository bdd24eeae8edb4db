"""The paged K/V cache: binding of the ``fm_cache_*``, ``fm_tree_*`` and
``fm_pages_*`` entry points of ``include/fm.h``.

Pools are bf16 CUDA tensors [pages][page_size][Hkv][d] of one layer, or
[layers][pages][page_size][Hkv][d]; page_size is 16, 32, 64 or 128, d 64 or
128, d is contiguous and the other strides are multiples of 8 elements.
``table`` [B][max_pages], ``lens`` [B], ``ref`` [pages], ``cu`` [B + 1],
``parents`` [total] and the other index arrays are contiguous int32 tensors on
the pools' device.

A step of a model that drafts trees:

    pages_reserve(n, k, v, table, lens, ref, ...)     # room for n[b] nodes each
    cache_append(k_new, v_new, cu, k[layer], v[layer], table, lens)     # per layer
    o, lse = tree_forward(q, k[layer], v[layer], table, lens, cu, scale, parents=parents)
    lens = cache_accept(accept, n_accept, cu, k, v, table, lens, ref=ref)  # after verification

Calls are enqueued on ``stream`` (default: the current stream of the tensors'
device), allocate there what the caller leaves out, and do not synchronise.  Arguments that the host can check raise
ValueError or FMError; what the kernels find wrong (a length, page, node or
row out of range, too few free pages) is or-ed into ``status``, an int32 CUDA
tensor of one element that the caller zeroes and reads with
``device_status(status)``.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools

import torch

from ._abi import FmCache, FmTreeDesc, check, lib

_I64x2 = ctypes.c_int64 * 2


_HERE = contextlib.nullcontext()


def _on(t, stream):
    """Context in which a call on tensor t's device runs and allocates: memory that the call
    allocates then belongs to the stream that uses it."""
    if stream is not None:
        if stream.device != t.device:
            raise ValueError("stream must belong to the tensors' device")
        return torch.cuda.stream(stream)
    if not t.is_cuda:
        raise ValueError("the cache's tensors must be on a CUDA device")
    return _HERE if t.device.index == torch.cuda.current_device() else torch.cuda.device(t.device)


def _stream(t):
    return torch.cuda.current_stream(t.device).cuda_stream


def _ints(where, like, **named):
    """Checks index tensors; the values None are left out."""
    for name, (t, shape) in named.items():
        if t is None:
            continue
        if t.dtype is not torch.int32 or not t.is_contiguous() or t.device != like.device \
                or t.shape != shape:
            raise ValueError(f"{where}: {name} must be a contiguous int32 tensor of shape "
                             f"{tuple(shape)} on {like.device}")


def _status_ptr(where, status, like):
    if status is None:
        return None
    if status.dtype is not torch.int32 or status.numel() < 1 or status.device != like.device:
        raise ValueError(f"{where}: status must be an int32 tensor on {like.device}")
    return status.data_ptr()


def _bf16(where, like, **named):
    for name, t in named.items():
        if t.dtype is not torch.bfloat16 or not t.is_cuda or t.device != like.device:
            raise ValueError(f"{where}: {name} must be a bf16 CUDA tensor on {like.device}")
        if t.stride(-1) != 1 and t.shape[-1] != 1:
            raise ValueError(f"{where}: {name}'s head_dim must be the contiguous dimension")


@functools.lru_cache(maxsize=256)
def _cache_desc(B, max_pages, shape, k_stride, v_stride) -> FmCache:
    layers = shape[0] if len(shape) == 5 else 1
    C = FmCache()
    C.B, C.max_pages = B, max_pages
    C.layers, (C.n_pages, C.page_size, C.Hkv, C.d) = layers, shape[-4:]
    # without a layer axis, or with one layer, its stride is never used
    C.k_stride[:] = k_stride[:-1] if layers > 1 else (8, *k_stride[-4:-1])
    C.v_stride[:] = v_stride[:-1] if layers > 1 else (8, *v_stride[-4:-1])
    return C


def make_cache(k_pool, v_pool, table) -> FmCache:
    """The ``fm_cache`` description of pools and a page table (not to be changed)."""
    shape = k_pool.shape
    if len(shape) not in (4, 5) or v_pool.shape != shape or table.dim() != 2:
        raise ValueError("pools must have one shape, [layers][pages][page_size][Hkv][d] or "
                         "[pages][page_size][Hkv][d], and the page table two dimensions")
    _bf16("make_cache", table, k_pool=k_pool, v_pool=v_pool)
    return _cache_desc(table.shape[0], table.shape[1], tuple(shape), k_pool.stride(), v_pool.stride())


def _one_layer(where, k_pool):
    if k_pool.dim() != 4:
        raise ValueError(f"{where}: give one layer's pools, [pages][page_size][Hkv][d]")


def cache_append(k, v, cu, k_pool, v_pool, table, lens, status=None, stream=None):
    """Write new tokens' K and V ([total][Hkv][d], packed by ``cu``) to one layer's
    pools: sequence b's are its last cu[b + 1] - cu[b] of lens[b] cached tokens."""
    _one_layer("cache_append", k_pool)
    C = make_cache(k_pool, v_pool, table)
    _bf16("cache_append", k_pool, k=k, v=v)
    if k.dim() != 3 or v.shape != k.shape or k.shape[1:] != k_pool.shape[2:]:
        raise ValueError("cache_append: k and v must be [total][Hkv][d]")
    B = C.B
    _ints("cache_append", k_pool, cu=(cu, (B + 1,)), table=(table, table.shape), lens=(lens, (B,)))
    if k.shape[0] == 0:
        return
    with _on(k_pool, stream):
        check(lib().fm_cache_append(ctypes.byref(C), k.data_ptr(), v.data_ptr(),
                                    _I64x2(*k.stride()[:2]), _I64x2(*v.stride()[:2]), cu.data_ptr(),
                                    k.shape[0], k_pool.data_ptr(), v_pool.data_ptr(),
                                    table.data_ptr(), lens.data_ptr(),
                                    _status_ptr("cache_append", status, k_pool),
                                    _stream(k_pool)), "fm_cache_append")


@functools.lru_cache(maxsize=256)
def _tree_desc(H, total, max_nodes, q_stride, o_stride) -> FmTreeDesc:
    D = FmTreeDesc()
    D.H, D.total, D.max_nodes = H, total, max_nodes
    D.q_stride[:], D.o_stride[:] = q_stride, o_stride
    return D


def tree_workspace(q, k_pool, v_pool, table, max_nodes=None) -> torch.Tensor:
    """Scratch of ``tree_forward`` for a program that keeps its own (one per call in flight)."""
    C = make_cache(k_pool, v_pool, table)
    total = max(q.shape[0], 1)
    D = _tree_desc(q.shape[1], total, max_nodes or total, q.stride()[:2], q.stride()[:2])
    with _on(q, None):
        n = lib().fm_tree_workspace_size(ctypes.byref(C), ctypes.byref(D))
    if n == 0:
        raise ValueError("tree_workspace: sizes that fm_tree_fwd does not take")
    return torch.empty(n, dtype=torch.uint8, device=q.device)


def tree_forward(q, k_pool, v_pool, table, lens, cu, scale, parents=None, max_nodes=None, o=None,
                 lse=None, ws=None, status=None, stream=None):
    """Attention of packed query tokens over one layer's cache: O [total][H][d] bf16 and
    LSE [H][total] fp32.  Sequence b's cu[b + 1] - cu[b] query tokens are the last of its
    lens[b] cached tokens.  ``parents`` [total]: the drafted tree (the node's parent within
    its sequence, -1 for a root, -2 for padding); without it every token sees the ones before
    it.  ``max_nodes``: an upper bound of a sequence's query tokens (default: total); a close
    one picks the faster kernel."""
    _one_layer("tree_forward", k_pool)
    C = make_cache(k_pool, v_pool, table)
    if q.dim() != 3 or q.shape[2] != C.d:
        raise ValueError("tree_forward: q must be [total][H][d]")
    total, H = q.shape[0], q.shape[1]
    dev = q.device
    with _on(q, stream):
        if o is None:
            o = torch.empty(q.shape, dtype=q.dtype, device=dev)
        if lse is None:
            lse = torch.empty(H, total, dtype=torch.float32, device=dev)
        if ws is None:
            ws = tree_workspace(q, k_pool, v_pool, table, max_nodes)
    _bf16("tree_forward", k_pool, q=q, o=o)
    if o.shape != q.shape or lse.shape != (H, total) or lse.dtype is not torch.float32 \
            or not lse.is_contiguous() or lse.device != dev:
        raise ValueError("tree_forward: o must have q's shape and lse be a contiguous fp32 [H][total]")
    B = C.B
    _ints("tree_forward", k_pool, table=(table, table.shape), lens=(lens, (B,)), cu=(cu, (B + 1,)),
          parents=(parents, (total,)))
    if total == 0:
        return o, lse
    D = _tree_desc(H, total, max_nodes or (min(total, 256) if parents is not None else total),
                   q.stride()[:2], o.stride()[:2])
    with _on(q, stream):
        check(lib().fm_tree_fwd(ctypes.byref(C), ctypes.byref(D), q.data_ptr(), k_pool.data_ptr(),
                                v_pool.data_ptr(), table.data_ptr(), lens.data_ptr(), cu.data_ptr(),
                                None if parents is None else parents.data_ptr(), scale,
                                o.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(),
                                _status_ptr("tree_forward", status, k_pool), _stream(q)),
              "fm_tree_fwd")
    return o, lse


def cache_accept(accept, n_accept, cu, k_pool, v_pool, table, lens, lens_out=None, ref=None,
                 status=None, stream=None):
    """Keep the accepted nodes of each sequence's tree: node accept[b][i] (ascending, the first
    n_accept[b] count) moves to the i-th place after the context, in all layers.  With ``ref``
    the pages past a row's new length lose its hold.  Returns the new lengths (``lens_out``,
    which may not be ``lens``)."""
    C = make_cache(k_pool, v_pool, table)
    B = C.B
    if lens_out is None:
        with _on(lens, stream):
            lens_out = torch.empty_like(lens)
    if accept.dim() != 2:
        raise ValueError("cache_accept: accept must be [B][max_accept]")
    _ints("cache_accept", k_pool, accept=(accept, (B, accept.shape[1])), n_accept=(n_accept, (B,)),
          cu=(cu, (B + 1,)), table=(table, table.shape), lens=(lens, (B,)), lens_out=(lens_out, (B,)),
          ref=(ref, (C.n_pages,)))
    with _on(k_pool, stream):
        check(lib().fm_cache_accept(ctypes.byref(C), accept.data_ptr(), accept.shape[1],
                                    n_accept.data_ptr(), cu.data_ptr(), k_pool.data_ptr(),
                                    v_pool.data_ptr(), table.data_ptr(), lens.data_ptr(),
                                    lens_out.data_ptr(), None if ref is None else ref.data_ptr(),
                                    _status_ptr("cache_accept", status, k_pool),
                                    _stream(k_pool)), "fm_cache_accept")
    return lens_out


@functools.lru_cache(maxsize=256)
def _pages_desc(B, max_pages, page_size, n_pages) -> FmCache:
    C = FmCache()
    C.B, C.max_pages, C.page_size, C.n_pages = B, max_pages, page_size, n_pages
    return C


def pages_fork(parent, page_size, table, lens, ref, table_out=None, lens_out=None, ref_out=None,
               status=None, stream=None):
    """Rows after a step of a search or a scheduler: new row b shares the pages of old row
    parent[b] (-1: empty).  Returns (table_out, lens_out, ref_out); ``ref_out`` may be ``ref``
    (the default), the other two are new."""
    with _on(table, stream):
        table_out = torch.empty_like(table) if table_out is None else table_out
        lens_out = torch.empty_like(lens) if lens_out is None else lens_out
    ref_out = ref if ref_out is None else ref_out
    if table.dim() != 2 or ref.dim() != 1 or not table.is_cuda:
        raise ValueError("pages_fork: table must be [B][max_pages] and ref [pages], on a CUDA device")
    B, n = table.shape[0], ref.shape
    _ints("pages_fork", table, parent=(parent, (B,)), table=(table, table.shape), lens=(lens, (B,)),
          ref=(ref, n), table_out=(table_out, table.shape), lens_out=(lens_out, (B,)),
          ref_out=(ref_out, n))
    C = _pages_desc(B, table.shape[1], page_size, n[0])
    with _on(table, stream):
        check(lib().fm_pages_fork(ctypes.byref(C), parent.data_ptr(), table.data_ptr(),
                                  lens.data_ptr(), ref.data_ptr(), table_out.data_ptr(),
                                  lens_out.data_ptr(), ref_out.data_ptr(),
                                  _status_ptr("pages_fork", status, table), _stream(table)),
              "fm_pages_fork")
    return table_out, lens_out, ref_out


def pages_workspace(k_pool, v_pool, table) -> torch.Tensor:
    """Scratch of ``pages_reserve`` and ``pages_compact`` for a program that keeps its own."""
    C = make_cache(k_pool, v_pool, table)
    n = lib().fm_pages_workspace_size(ctypes.byref(C))
    if n == 0:
        raise ValueError("pages_workspace: sizes that fm_pages_reserve does not take")
    return torch.empty(n, dtype=torch.uint8, device=table.device)


def pages_reserve(grow, k_pool, v_pool, table, lens, ref, table_out=None, lens_out=None,
                  ref_out=None, info=None, ws=None, status=None, stream=None):
    """Room for grow[b] more tokens of every row, in place by default: free pages in ascending
    order, and a copy of a shared last page that the row will write.  All or nothing.  Returns
    ``info``: int32 [2], free pages after the call and pages asked for (more than were free:
    nothing was done)."""
    C = make_cache(k_pool, v_pool, table)
    B, n = C.B, (C.n_pages,)
    table_out = table if table_out is None else table_out
    lens_out = lens if lens_out is None else lens_out
    ref_out = ref if ref_out is None else ref_out
    with _on(table, stream):
        if info is None:
            info = torch.empty(2, dtype=torch.int32, device=table.device)
        if ws is None:
            ws = pages_workspace(k_pool, v_pool, table)
    _ints("pages_reserve", k_pool, grow=(grow, (B,)), table=(table, table.shape), lens=(lens, (B,)),
          ref=(ref, n), table_out=(table_out, table.shape), lens_out=(lens_out, (B,)),
          ref_out=(ref_out, n), info=(info, (2,)))
    with _on(k_pool, stream):
        check(lib().fm_pages_reserve(ctypes.byref(C), grow.data_ptr(), k_pool.data_ptr(),
                                     v_pool.data_ptr(), table.data_ptr(), lens.data_ptr(),
                                     ref.data_ptr(), table_out.data_ptr(), lens_out.data_ptr(),
                                     ref_out.data_ptr(), info.data_ptr(), ws.data_ptr(), ws.numel(),
                                     _status_ptr("pages_reserve", status, k_pool),
                                     _stream(k_pool)), "fm_pages_reserve")
    return info


def pages_compact(k_pool, v_pool, table, lens, ref, table_out=None, ref_out=None, n_live=None,
                  ws=None, status=None, stream=None):
    """Move the held pages to the front of the pool, [0, n_live), in place by default.  Returns
    ``n_live``: int32 [1]."""
    C = make_cache(k_pool, v_pool, table)
    B, n = C.B, (C.n_pages,)
    table_out = table if table_out is None else table_out
    ref_out = ref if ref_out is None else ref_out
    with _on(table, stream):
        if n_live is None:
            n_live = torch.empty(1, dtype=torch.int32, device=table.device)
        if ws is None:
            ws = pages_workspace(k_pool, v_pool, table)
    _ints("pages_compact", k_pool, table=(table, table.shape), lens=(lens, (B,)), ref=(ref, n),
          table_out=(table_out, table.shape), ref_out=(ref_out, n), n_live=(n_live, (1,)))
    with _on(k_pool, stream):
        check(lib().fm_pages_compact(ctypes.byref(C), k_pool.data_ptr(), v_pool.data_ptr(),
                                     table.data_ptr(), lens.data_ptr(), ref.data_ptr(),
                                     table_out.data_ptr(), ref_out.data_ptr(), n_live.data_ptr(),
                                     ws.data_ptr(), ws.numel(),
                                     _status_ptr("pages_compact", status, k_pool),
                                     _stream(k_pool)), "fm_pages_compact")
    return n_live
