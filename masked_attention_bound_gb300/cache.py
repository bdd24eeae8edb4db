"""The paged K/V cache: the ``fm_cache_*``, ``fm_tree_*`` and ``fm_pages_*``
entry points of ``include/fm.h`` on torch tensors.

Pools are bf16 CUDA tensors [pages][page_size][Hkv][d] of one layer, or
[layers][pages][page_size][Hkv][d]; page_size is 16, 32, 64 or 128, d 64 or
128, d is contiguous and the other strides are multiples of 8 elements.
``table`` [B][max_pages], ``lens`` [B], ``ref`` [pages], ``cu`` [B + 1],
``parents`` [total] and the other index arrays are contiguous int32 tensors on
the pools' device.

A step of a model that drafts trees:

    pages_reserve(n, k, v, table, lens, ref)          # room for n[b] nodes each
    cache_append(k_new, v_new, cu, k[layer], v[layer], table, lens)     # per layer
    o, lse = tree_forward(q, k[layer], v[layer], table, lens, cu, scale, parents=parents,
                          max_nodes=64)               # no sequence has more
    lens = cache_accept(accept, n_accept, cu, k, v, table, lens, ref=ref)  # after verification

These are operators of inference: no gradient flows through them.

Calls are enqueued on ``stream`` (default: the current stream of the tensors'
device), allocate there what the caller leaves out, and do not synchronise.
Arguments that the host can check raise ValueError or FMError; what the
kernels find wrong (a length, page, node or row out of range, too few free
pages) is or-ed into ``status``, an int32 CUDA tensor of one element that the
caller zeroes and reads with ``device_status(status)``.

The calls go through the module ``_fmcache`` (csrc/fm_binding.cpp), which
checks the tensors and calls the C ABI; without it they raise.
"""
from __future__ import annotations

import ctypes

import torch

from ._abi import FmCache, FmTreeDesc, lib

_module = None


def _load():
    """The compiled binding.  Raises if it has not been built."""
    global _module
    lib()      # its own message if nothing has been built; the module links to it
    try:
        from . import _fmcache
    except ImportError as e:
        raise RuntimeError("the _fmcache module is missing or does not load: build it first "
                           "(python -m masked_attention_bound_gb300.build)") from e
    _module = _fmcache
    return _module


def _call(name, stream, *args):
    m = _module or _load()
    if stream is None:
        return getattr(m, name)(*args)
    if stream.device != args[0].device:
        raise ValueError("stream must belong to the tensors' device")
    with torch.cuda.stream(stream):        # memory that the call allocates belongs to it too
        return getattr(m, name)(*args)


def make_cache(k_pool, v_pool, table) -> FmCache:
    """The ``fm_cache`` description of pools and a page table, for calls of the C ABI."""
    if k_pool.dim() not in (4, 5) or v_pool.shape != k_pool.shape or table.dim() != 2:
        raise ValueError("pools must have one shape, [layers][pages][page_size][Hkv][d] or "
                         "[pages][page_size][Hkv][d], and the page table two dimensions")
    for t in (k_pool, v_pool):
        if t.dtype is not torch.bfloat16 or not t.is_cuda or t.device != table.device:
            raise ValueError("pools must be bf16 CUDA tensors on the page table's device")
        if t.stride(-1) != 1:
            raise ValueError("head_dim must be the contiguous dimension")
    if max(*k_pool.shape, *table.shape) >= 1 << 31:
        raise ValueError("pools and page tables have fewer than 2^31 layers, pages, rows and entries of a row")
    C = FmCache()
    C.B, C.max_pages = table.shape
    C.layers = k_pool.shape[0] if k_pool.dim() == 5 else 1
    C.n_pages, C.page_size, C.Hkv, C.d = k_pool.shape[-4:]
    for to, t in ((C.k_stride, k_pool), (C.v_stride, v_pool)):
        # a dimension of one element is never stepped along
        s = [8 if n == 1 else x for n, x in zip(t.shape[:-1], t.stride()[:-1])]
        to[:] = s if t.dim() == 5 else [8, *s]
    return C


def cache_append(k, v, cu, k_pool, v_pool, table, lens, status=None, stream=None):
    """Write new tokens' K and V ([total][Hkv][d], packed by ``cu``) to one layer's
    pools: sequence b's are its last cu[b + 1] - cu[b] of lens[b] cached tokens."""
    _call("append", stream, k, v, cu, k_pool, v_pool, table, lens, status)


def tree_workspace(q, k_pool, v_pool, table, max_nodes=None) -> torch.Tensor:
    """Scratch of ``tree_forward`` for a program that keeps its own (one per call in flight).  It
    serves every call of up to ``max_nodes`` and q's tokens, with the same heads and any table."""
    C = make_cache(k_pool, v_pool, table)
    D = FmTreeDesc()
    total = max(q.shape[0], 1)
    D.H, D.total, D.max_nodes = q.shape[1], total, max_nodes or total
    D.q_stride[:] = D.o_stride[:] = (8, 8)
    with torch.cuda.device(q.device):
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
    it.  ``max_nodes``: an upper bound of a sequence's query tokens (default: total, with
    ``parents`` at most 256); a close one picks the faster kernel, and a batch of several
    sequences should give it (128 single tokens over up to 255 tokens of context, 4 query heads
    per K/V head: 31 us with 1, 60 with the default, which plans for 128 tokens a sequence; over
    up to 8192 tokens 481 and 493)."""
    return _call("tree", stream, q, k_pool, v_pool, table, lens, cu, scale, parents, max_nodes, o, lse,
                 ws, status)


def cache_accept(accept, n_accept, cu, k_pool, v_pool, table, lens, lens_out=None, ref=None,
                 status=None, stream=None):
    """Keep the accepted nodes of each sequence's tree: node accept[b][i] (ascending, the first
    n_accept[b] count) moves to the i-th place after the context, in all layers.  With ``ref``
    the pages past a row's new length lose its hold.  Returns the new lengths (``lens_out``,
    which may not be ``lens``)."""
    return _call("accept", stream, accept, n_accept, cu, k_pool, v_pool, table, lens, lens_out, ref, status)


def pages_fork(parent, page_size, table, lens, ref, table_out=None, lens_out=None, ref_out=None,
               status=None, stream=None):
    """Rows after a step of a search or a scheduler: new row b shares the pages of old row
    parent[b] (-1: empty).  Returns (table_out, lens_out, ref_out); ``ref_out`` may be ``ref``
    (the default), the other two are new."""
    return _call("fork", stream, parent, page_size, table, lens, ref, table_out, lens_out, ref_out, status)


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
    return _call("reserve", stream, grow, k_pool, v_pool, table, lens, ref, table_out, lens_out, ref_out,
                 info, ws, status)


def pages_compact(k_pool, v_pool, table, lens, ref, table_out=None, ref_out=None, n_live=None,
                  ws=None, status=None, stream=None):
    """Move the held pages to the front of the pool, [0, n_live), in place by default.  Returns
    ``n_live``: int32 [1]."""
    return _call("compact", stream, k_pool, v_pool, table, lens, ref, table_out, ref_out, n_live, ws, status)
