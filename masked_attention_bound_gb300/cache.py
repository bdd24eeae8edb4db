"""The paged K/V cache: the ``fm_cache_*``, ``fm_tree_*`` and ``fm_pages_*``
entry points of ``include/fm.h`` on torch tensors.

Pools are CUDA tensors [pages][page_size][Hkv][d] of one layer, or
[layers][pages][page_size][Hkv][d]; page_size is 16, 32, 64 or 128, d 64 or
128, d is contiguous.  They hold bf16, with the other strides multiples of 8
elements, or e4m3 codes (torch.float8_e4m3fn, strides multiples of 16).  A
cache of codes comes with ``k_scale`` and ``v_scale``, contiguous fp32 tensors
[pages][Hkv][page_size / 16] (with the layers in front where the pools have
them; ``cache_scales`` makes them): a value is its code times the scale of its
block of 16 tokens and head.  It takes half the bytes.  Attention over it takes
0.5 to 0.65 of the time where reading them is what it waits for (up to 16 rows,
query tokens times heads, a sequence and K/V head); with more it is bound by
other things: trees of 32 nodes of 4 heads take about as long as over bf16,
trees of 64 and pieces of prompts up to a fifth longer.
``table`` [B][max_pages], ``lens`` [B], ``ref`` [pages], ``cu`` [B + 1],
``parents`` [total] and the other index arrays are contiguous int32 tensors on
the pools' device.

A step of a model that drafts trees:

    pages_reserve(n, k, v, table, lens, ref)          # room for n[b] nodes each
    cache_append(k_new, v_new, cu, k[layer], v[layer], table, lens)     # per layer, or with
    q = cache_append_rotary(q, k_new, v_new, cu, freqs, k[layer], v[layer], table, lens,
                            positions=context_and_depth)                # rotated by position
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

SCALE_BLOCK = 16          # tokens of a head that share a scale in a cache of codes

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
    if stream.device != next(a.device for a in args if isinstance(a, torch.Tensor)):
        raise ValueError("stream must belong to the tensors' device")
    with torch.cuda.stream(stream):        # memory that the call allocates belongs to it too
        return getattr(m, name)(*args)


def make_cache(k_pool, v_pool, table) -> FmCache:
    """The ``fm_cache`` description of pools and a page table, for calls of the C ABI."""
    if k_pool.dim() not in (4, 5) or v_pool.shape != k_pool.shape or table.dim() != 2:
        raise ValueError("pools must have one shape, [layers][pages][page_size][Hkv][d] or "
                         "[pages][page_size][Hkv][d], and the page table two dimensions")
    for t in (k_pool, v_pool):
        if t.dtype not in (torch.bfloat16, torch.float8_e4m3fn) or not t.is_cuda or t.device != table.device:
            raise ValueError("pools must be bf16 or float8_e4m3fn CUDA tensors on the page table's device")
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
        s = [16 if n == 1 else x for n, x in zip(t.shape[:-1], t.stride()[:-1])]
        to[:] = s if t.dim() == 5 else [16, *s]
    return C


def cache_scales(pool) -> torch.Tensor:
    """Scales of a pool of e4m3 codes, one for each block of 16 tokens of a head, all 1.
    (Appending gives a block its scale; the initial values have no part in a result.)"""
    if pool.dim() not in (4, 5) or pool.shape[-3] % SCALE_BLOCK:
        raise ValueError("a pool has the shape [layers][pages][page_size][Hkv][d] or [pages][page_size][Hkv][d]")
    *front, page_size, heads, _ = pool.shape
    return torch.ones(*front, heads, page_size // SCALE_BLOCK, dtype=torch.float32, device=pool.device)


def cache_append(k, v, cu, k_pool, v_pool, table, lens, status=None, stream=None, k_scale=None,
                 v_scale=None):
    """Write new tokens' K and V ([total][Hkv][d], packed by ``cu``) to one layer's
    pools: sequence b's are its last cu[b + 1] - cu[b] of lens[b] cached tokens.  With pools of
    codes (``k_scale``, ``v_scale``) a block that begins with a new token gets the least power of
    two as its scale that brings its largest value to 448 or less; one that has tokens keeps at
    least its scale, and its codes are rounded again where that grows."""
    _call("append", stream, k, v, cu, k_pool, v_pool, table, lens, k_scale, v_scale, status)


def cache_append_rotary(q, k, v, cu, freqs, k_pool, v_pool, table, lens, positions=None,
                        interleaved=False, q_out=None, k_scale=None, v_scale=None, status=None,
                        stream=None):
    """``cache_append`` with keys and queries rotated by their position on the way: element pair i
    of a head's first 2 n, n = len(freqs) (a multiple of 8), turns by position * freqs[i] radians.  Pairs
    are (x[i], x[i + n]), or neighbours with ``interleaved``.  ``positions`` [total]: by default
    a token's place in its sequence; a drafted node has context + depth.  Returns the rotated queries
    [total][H][d] (``q_out``, which may be ``q`` and overlaps neither it otherwise nor ``k`` and ``v``), or
    None where ``q`` is None."""
    return _call("append_rotary", stream, q, k, v, cu, freqs, k_pool, v_pool, table, lens, positions,
                 interleaved, q_out, k_scale, v_scale, status)


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
                 lse=None, ws=None, status=None, stream=None, k_scale=None, v_scale=None):
    """Attention of packed query tokens over one layer's cache: O [total][H][d] bf16 and
    LSE [H][total] fp32.  Sequence b's cu[b + 1] - cu[b] query tokens are the last of its
    lens[b] cached tokens.  ``parents`` [total]: the drafted tree (the node's parent within
    its sequence, -1 for a root, -2 for padding); without it every token sees the ones before
    it.  ``max_nodes``: an upper bound of a sequence's query tokens (default: total, with
    ``parents`` at most 256); a close one picks the faster kernel, and a batch of several
    sequences should give it (128 single tokens over up to 255 tokens of context, 4 query heads
    per K/V head: 31 us with 1, 41 to 60 with the default, which plans for 128 tokens a sequence; over
    up to 8192 tokens 482 and 498; over codes 23 and 92, 270 and 616).  The largest sequence picks it
    for all: pieces of prompts are better a call of their own beside single tokens (a piece of 480
    tokens and 127 single ones over up to 8192 tokens of codes 751 us together, 82 and 240 apart)."""
    return _call("tree", stream, q, k_pool, v_pool, table, lens, cu, scale, parents, max_nodes, o, lse,
                 ws, k_scale, v_scale, status)


def cache_accept(accept, n_accept, cu, k_pool, v_pool, table, lens, lens_out=None, ref=None,
                 status=None, stream=None, k_scale=None, v_scale=None):
    """Keep the accepted nodes of each sequence's tree: node accept[b][i] (ascending, the first
    n_accept[b] count) moves to the i-th place after the context, in all layers.  With ``ref``
    the pages past a row's new length lose its hold.  Returns the new lengths (``lens_out``,
    which may not be ``lens``)."""
    return _call("accept", stream, accept, n_accept, cu, k_pool, v_pool, table, lens, lens_out, ref, k_scale,
                 v_scale, status)


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
                  ref_out=None, info=None, ws=None, status=None, stream=None, k_scale=None, v_scale=None):
    """Room for grow[b] more tokens of every row, in place by default: free pages in ascending
    order, and a copy of a shared last page that the row will write.  All or nothing.  Returns
    ``info``: int32 [2], free pages after the call and pages asked for (more than were free:
    nothing was done)."""
    return _call("reserve", stream, grow, k_pool, v_pool, table, lens, ref, table_out, lens_out, ref_out,
                 info, ws, k_scale, v_scale, status)


def pages_compact(k_pool, v_pool, table, lens, ref, table_out=None, ref_out=None, n_live=None,
                  ws=None, status=None, stream=None, k_scale=None, v_scale=None):
    """Move the held pages to the front of the pool, [0, n_live), in place by default.  Returns
    ``n_live``: int32 [1]."""
    return _call("compact", stream, k_pool, v_pool, table, lens, ref, table_out, ref_out, n_live, ws, k_scale,
                 v_scale, status)
