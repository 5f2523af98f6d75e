"""Plain numpy fp64 oracle of rotary positions with several axes, and of a paged K/V cache.

TEST INFRASTRUCTURE, NOT PRODUCT CODE (see cowa_oracle).  Imports nothing from the library.

Rotation: pair i of a head's elements turns by angle(t, i) = pos[axis(i)][t] * inv_freq[i], the pairs
being dealt out to the axes in order by `sections`:

    (a, b) -> scale (a cos - b sin, b cos + a sin)

Pair i is elements (i, i + r/2), or (2i, 2i + 1) if interleaved, r = 2 len(inv_freq); the rest of the
head passes through.  The transpose is the rotation by the negated angle.
"""

from __future__ import annotations

import numpy as np

__all__ = ["angles", "rope", "gather_pages"]


def angles(pos, inv_freq, sections) -> np.ndarray:
    """[tokens, r/2] float64 from pos [axes, tokens] (integers) and inv_freq (the float32 values used)."""
    pos = np.asarray(pos, dtype=np.float64)
    f = np.asarray(inv_freq, dtype=np.float32).astype(np.float64)
    axis = np.repeat(np.arange(len(sections)), sections)
    assert axis.size == f.size
    return pos[axis].T * f


def rope(x, pos, inv_freq, sections=None, interleaved=False, scale=1.0, transpose=False) -> np.ndarray:
    """x [tokens, H, d] float64 rotated (or, transpose, its gradient pulled back)."""
    inv_freq = np.asarray(inv_freq, dtype=np.float32)
    h = inv_freq.size
    a = angles(pos, inv_freq, [h] if sections is None else sections)
    c = (scale * np.cos(a))[:, None]
    s = (scale * np.sin(a))[:, None] * (-1.0 if transpose else 1.0)
    y = np.array(x, dtype=np.float64)
    i = np.arange(h)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
    xa, xb = x[..., ia], x[..., ib]
    y[..., ia] = xa * c - xb * s
    y[..., ib] = xb * c + xa * s
    return y


def gather_pages(pool, table, n, fill=0):
    """A paged pool read back as a contiguous cache.

    pool [n_pages, page_size, H, d] (H = 1 with a table per head), table [B, max_pages] or
    [B, Hkv, max_pages]; returns [B, Hkv, n, d] of positions 0..n-1, `fill` where the entry lies
    outside the pool, and the bool array [B, Hkv, n] of the positions that have a page."""
    n_pages, ps, hp, d = pool.shape
    per_head = table.ndim == 3
    B, H = table.shape[0], table.shape[1] if per_head else hp
    out = np.full((B, H, n, d), fill, dtype=pool.dtype)
    has = np.zeros((B, H, n), dtype=bool)
    s = np.arange(n)
    for b in range(B):
        for g in range(H):
            page = (table[b, g] if per_head else table[b])[s // ps]
            ok = (page >= 0) & (page < n_pages)
            out[b, g, ok] = pool[page[ok], (s % ps)[ok], 0 if per_head else g]
            has[b, g] = ok
    return out, has
