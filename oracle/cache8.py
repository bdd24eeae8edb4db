"""The paged cache held in e4m3 codes, and the rotation by position, from their
definitions in numpy float64.

Codes are float64 values of e4m3 (NaN among them), pools [pages][page_size][Hkv][d]
as in ``oracle.cache``; scales [pages][Hkv][page_size / 16].
"""
from __future__ import annotations

import numpy as np

from .fp8 import E4M3_MAX, e4m3

BLOCK = 16
LEAST, MOST = 2.0 ** -60, 2.0 ** 60


def code(x):
    """The nearest code of every value; NaN stays NaN, infinities saturate."""
    x = np.asarray(x, np.float64)
    return np.where(np.isnan(x), np.nan, e4m3(np.clip(np.where(np.isnan(x), 0, x), -E4M3_MAX, E4M3_MAX)))


def as_read(scale):
    """A scale as every operator reads it."""
    s = np.asarray(scale, np.float64)
    return np.clip(np.where(np.isnan(s), LEAST, s), LEAST, MOST)


def scale_for(amax):
    """The least power of two within range that brings amax to 448 or less."""
    s = np.full(np.shape(amax), LEAST)
    for e in range(-60, 60):
        s = np.where(np.asarray(amax) > E4M3_MAX * 2.0 ** e, 2.0 ** (e + 1), s)
    return s


def values(codes, scales):
    """What pools of codes stand for."""
    return codes * np.repeat(as_read(scales), BLOCK, axis=-1).swapaxes(-1, -2)[..., None]


def rotate(x, positions, freqs, interleaved):
    """x [T][heads][d] with pair i of its first 2 len(freqs) elements turned by position * freqs[i]."""
    x, n = np.array(x, np.float64), len(freqs)
    a = np.asarray(positions, np.longdouble)[:, None] * np.asarray(freqs, np.longdouble)
    turn = 2 * np.longdouble("3.14159265358979323846264338327950288")
    a = (a - np.round(a / turn) * turn).astype(np.float64)
    c, s = np.cos(a)[:, None], np.sin(a)[:, None]
    i, j = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    x[..., i], x[..., j] = x[..., i] * c - x[..., j] * s, x[..., j] * c + x[..., i] * s
    return x


def append(x, cu, codes, scales, table, lens):
    """New tokens' values x [T][Hkv][d] to copies of one layer's codes and scales."""
    codes, scales, page = codes.copy(), scales.copy(), codes.shape[1]
    for b in range(len(lens)):
        n = cu[b + 1] - cu[b]
        base = lens[b] - n
        for blk in range(base // BLOCK, -(-lens[b] // BLOCK) if n else 0):
            lo, hi = max(base, blk * BLOCK), min(lens[b], (blk + 1) * BLOCK)
            if lo >= hi:
                continue
            new = x[cu[b] + lo - base:cu[b] + hi - base]
            pg, j = table[b][lo // page], lo % page // BLOCK
            here = codes[pg, j * BLOCK:(j + 1) * BLOCK]
            s = scale_for(np.where(np.isfinite(new), np.abs(new), 0).max((0, 2)))
            if lo % BLOCK:
                old = as_read(scales[pg, :, j])
                s = np.maximum(s, old)
                grown = s > old
                here[:, grown] = code(here[:, grown] * (old / s)[grown][:, None])
            here[lo % BLOCK:lo % BLOCK + hi - lo] = code(new / s[:, None])
            scales[pg, :, j] = s
    return codes, scales


def accept(nodes, cu, codes, scales, table, lens):
    """Accepted nodes (a list per sequence) moved together in copies of [layers] pools and scales."""
    page, out = codes.shape[2], []
    old_codes, old_scales = codes, as_read(scales)
    codes, scales = codes.copy(), scales.copy()
    for b, acc in enumerate(nodes):
        base = lens[b] - (cu[b + 1] - cu[b])
        at = lambda p: (table[b][p // page], p % page)  # noqa: E731
        into = {}
        for i, a in enumerate(acc):
            into.setdefault((base + i) // BLOCK, []).append((base + a, base + i))
        for blk, moves in into.items():
            pg, j = table[b][blk * BLOCK // page], blk * BLOCK % page // BLOCK
            s = old_scales[:, pg, :, j].copy()
            for x, _ in moves:
                p, q = at(x)
                s = np.maximum(s, old_scales[:, p, :, q // BLOCK])
            rows = slice(j * BLOCK, (j + 1) * BLOCK)
            here = code(old_codes[:, pg, rows] * (old_scales[:, pg, :, j] / s)[:, None, :, None])
            for x, y in moves:
                p, q = at(x)
                here[:, y % BLOCK] = code(old_codes[:, p, q] * (old_scales[:, p, :, q // BLOCK] / s)[..., None])
            codes[:, pg, rows] = here
            scales[:, pg, :, j] = s
        out.append(base + len(acc))
    return codes, scales, out
