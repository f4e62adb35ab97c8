"""The target's side of a step in float64: rotary positions, a paged cache's append and commit, attention of a
drafted block over it.  Plain loops over sequences and rows; numpy only."""
from __future__ import annotations

import math

import numpy as np


def rope_frequencies(rotary_dim, base=10000.0, scaling="none", factor=1.0, low=1.0, high=32.0, original_len=0):
    """(frequencies, magnitude) of the rotary pairs, with the scalings for long contexts."""
    r = rotary_dim
    if scaling == "base":
        base = base * factor ** (r / (r - 2.0))
    i = np.arange(r // 2)
    f = base ** (-2.0 * i / r)
    mag = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "turns":
        g = np.clip((original_len * f / (2 * math.pi) - low) / (high - low), 0.0, 1.0)
        f = f * g + (1.0 - g) * f / factor
    elif scaling == "dims":
        def dim_of(turns):
            return r * math.log(original_len / (2 * math.pi * turns)) / (2 * math.log(base))
        d0 = min(max(math.floor(dim_of(high)), 0), r - 1)
        d1 = min(max(math.ceil(dim_of(low)), 0), r - 1)
        h = np.clip((i - d0) / max(d1 - d0, 0.001), 0.0, 1.0)
        f = f * (1.0 - h) + h * f / factor
        mag = 1.0 + 0.1 * math.log(factor)
    return f, mag


def rope(x, positions, inv_freq, style="half", magnitude=1.0, backward=False):
    """x [rows, heads, dim] with its first 2 len(inv_freq) elements turned pair by pair."""
    x = np.array(x, dtype=np.float64)
    half = len(inv_freq)
    ang = np.asarray(positions, np.float64)[:, None] * np.asarray(inv_freq, np.float64)
    c, s = magnitude * np.cos(ang)[:, None], magnitude * np.sin(ang)[:, None] * (-1.0 if backward else 1.0)
    if style == "half":
        a, b = x[..., :half].copy(), x[..., half:2 * half].copy()
        x[..., :half], x[..., half:2 * half] = a * c - b * s, a * s + b * c
    else:
        a, b = x[..., 0:2 * half:2].copy(), x[..., 1:2 * half:2].copy()
        x[..., 0:2 * half:2], x[..., 1:2 * half:2] = a * c - b * s, a * s + b * c
    return x


def ancestors(parents, n):
    """sees[i][j]: row j is row i or an ancestor of it.  parents None: a chain."""
    sees = np.zeros((n, n), bool)
    for i in range(n):
        j = i
        while True:
            sees[i, j] = True
            if j == 0:
                break
            j = j - 1 if parents is None else int(parents[j - 1])
    return sees


def slots(page_table, page_size, n):
    """(page, place) of tokens 0..n-1 of one sequence."""
    t = np.arange(n)
    return np.asarray(page_table)[t // page_size], t % page_size


def append(k_cache, v_cache, k, v, context, page_table, parents=None, inv_freq=None, style="half", magnitude=1.0, q=None):
    """One sequence's block: k, v [n, heads, dim] written in place into the caches [pages, size, heads, dim]; returns the
    rotated queries."""
    n, size = len(k), k_cache.shape[1]
    if inv_freq is not None:
        pos = context + ancestors(parents, n).sum(1) - 1
        k = rope(k, pos, inv_freq, style, magnitude)
        q = None if q is None else rope(q, pos, inv_freq, style, magnitude)
    page, place = slots(page_table, size, context + n)
    k_cache[page[context:], place[context:]] = k
    v_cache[page[context:], place[context:]] = v
    return q


def attend(q, k_cache, v_cache, context, page_table, scale, parents=None):
    """One sequence's rows q [n, heads, dim] over its cached tokens and its block: (out, lse, sum of w |v|, largest
    sum of |q_d k_d| scale over the tokens a row sees).  Tokens a row does not see do not enter at all."""
    n, H, D = q.shape
    G = H // k_cache.shape[2]
    page, place = slots(page_table, k_cache.shape[1], context + n)
    k, v = k_cache[page, place], v_cache[page, place]
    sees = np.concatenate([np.ones((n, context), bool), ancestors(parents, n)], 1)
    out, lse = np.zeros((n, H, D)), np.full((n, H), -np.inf)
    wabs, big = np.zeros((n, H, D)), np.zeros((n, H))
    for i in range(n):
        ki, vi = k[sees[i]], v[sees[i]]
        for h in range(H):
            kh, vh = ki[:, h // G], vi[:, h // G]
            s = scale * (kh @ q[i, h])
            top = s.max()
            w = np.exp(s - top)
            z = w.sum()
            w = w / z
            out[i, h], wabs[i, h] = w @ vh, w @ np.abs(vh)
            lse[i, h] = top + math.log(z)
            big[i, h] = abs(scale) * (np.abs(kh) @ np.abs(q[i, h])).max()
    return out, lse, wabs, big


def commit(k_cache, v_cache, context, page_table, accept_len, path):
    """One sequence: the accepted nodes' slots move to the slots after row 0's, in caches [layers, pages, size, heads, dim]."""
    size = k_cache.shape[2]
    page, place = slots(page_table, size, context + 1 + (max(path[:accept_len]) if accept_len else 0))
    src = [context + int(p) for p in path[:accept_len]]
    for c in (k_cache, v_cache):
        moved = c[:, page[src], place[src]].copy()
        for j in range(accept_len):
            c[:, page[context + 1 + j], place[context + 1 + j]] = moved[:, j]
    return context + 1 + accept_len
