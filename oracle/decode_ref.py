"""Plain numpy forms of the operators from a step's hidden states to its tokens,
independent of the HIP code: the int8 cache of keys and values, attention over
it, and the draw of a token.  Attention and the draw are the definitions in 64
bits; the cache's codes and values take the fp32 roundings that the operators
document, so they can be compared exactly.
"""

from __future__ import annotations

import numpy as np

from .operators_ref import quantize_rows_steps


def cache_rows_steps(x):
    """Keys or values [tokens, heads, d] (fp32) -> (codes int8, scale fp32 [tokens, heads])."""
    n, h, d = x.shape
    q, s = quantize_rows_steps(np.asarray(x, np.float32).reshape(n * h, d))
    return q.reshape(n, h, d).astype(np.int8), s.reshape(n, h)


def cache_write(codes, scale, x, slots):
    """Writes rows into codes [pages, heads, page_size, d] and scale in place; slots outside are skipped."""
    pages, _, size, _ = codes.shape
    q, s = cache_rows_steps(x)
    for i, slot in enumerate(slots):
        if 0 <= slot < pages * size:
            codes[slot // size, :, slot % size] = q[i]
            scale[slot // size, :, slot % size] = s[i]


def cache_read(codes, scale, slots):
    """fp32 rows [tokens, heads, d]: the rounded product of code and scale, 0 for slots outside."""
    pages, heads, size, d = codes.shape
    out = np.zeros((len(slots), heads, d), np.float32)
    for i, slot in enumerate(slots):
        if 0 <= slot < pages * size:
            with np.errstate(all="ignore"):
                out[i] = codes[slot // size, :, slot % size].astype(np.float32) * scale[slot // size, :, slot % size, None]
    return out


def attention(q, k, ks, v, vs, pages, visible, scale):
    """(out, sizes) in 64 bits of q [seqs, cols, heads, d] over the cache.

    ``sizes`` holds what the error of a result is measured by, for each row:
    the sum of weight times |value| of every output value, the largest sum of
    |q| |k| scale of a score, the largest |score|, the positions that count."""
    q = np.asarray(q, np.float64)
    seqs, cols, heads, d = q.shape
    n_pages, kv, size, _ = k.shape
    group = heads // kv
    out, absolute = np.zeros(q.shape), np.zeros(q.shape)
    dots, largest, count = np.zeros(q.shape[:3]), np.zeros(q.shape[:3]), np.zeros(q.shape[:3], np.int64)
    for s in range(seqs):
        for c in range(cols):
            n = min(max(int(visible[s][c]), 0), len(pages[s]) * size)
            at = np.array([i for i in range(n) if 0 <= pages[s][i // size] < n_pages], np.int64)
            if not len(at):
                continue
            where, place = np.asarray(pages[s])[at // size], at % size
            for h in range(kv):
                keys, key_scale = k[where, h, place].astype(np.float64), ks[where, h, place].astype(np.float64)
                values = v[where, h, place].astype(np.float64) * vs[where, h, place].astype(np.float64)[:, None]
                for a in range(h * group, (h + 1) * group):
                    t = keys @ q[s, c, a] * key_scale * scale
                    w = np.exp(t - t.max())
                    w /= w.sum()
                    out[s, c, a] = w @ values
                    absolute[s, c, a] = w @ np.abs(values)
                    dots[s, c, a] = (np.abs(keys) @ np.abs(q[s, c, a]) * key_scale).max() * abs(scale)
                    largest[s, c, a] = np.abs(t).max()
                    count[s, c, a] = len(at)
    return out, (absolute, dots, largest, count)


def sample_row(z, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, log of the probability it is drawn with) of one row of logits."""
    z = np.asarray(z, np.float64)
    drawn = z > -np.inf                                       # false for NaN
    if not drawn.any():
        return -1, -np.inf
    best = z[drawn].max()
    order = np.array(sorted(np.flatnonzero(drawn), key=lambda i: (-z[i], i)))
    if not temperature > 0:
        return int(order[0]), 0.0
    with np.errstate(all="ignore"):
        x = np.where(z == best, 0.0, -np.inf if np.isinf(best) else (z - best) / temperature)
    w = np.where(drawn, np.exp(x), 0.0)
    if top_k > 0:
        order = order[:top_k]
    if top_p < 1:
        mass = np.cumsum(w[order])
        before = np.concatenate([[0.0], mass[:-1]])
        keep = before < top_p * mass[-1]
        keep[0] = True
        order = order[keep]
    order = np.sort(order[(w[order] >= min(min_p, 1.0)) | (np.arange(len(order)) == 0)])
    mass = np.cumsum(w[order])
    i = min(int(np.searchsorted(mass, u * mass[-1], side="right")), len(order) - 1)
    while w[order[i]] == 0:                                   # u at the end of the mass
        i -= 1
    return int(order[i]), float(x[order[i]] - np.log(mass[-1]))
