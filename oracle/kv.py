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


# ---- the cache held in 8 bits --------------------------------------------------------------------------------------------------

def e4m3_grid(x):
    """x rounded to the nearest e4m3 number, ties to the even one; |x| at most 448 but for infinities, which become NaN."""
    x = np.asarray(x, np.float64)
    with np.errstate(divide="ignore", invalid="ignore"):
        step = np.exp2(np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6))) - 3)
        y = np.round(x / step) * step   # half to even
    return np.where(np.isfinite(x), y, np.nan)


def scale_exponent(most):
    """The smallest exponent, -120 at least, of a power of two that keeps `most` within 448."""
    m, e = np.frexp(np.asarray(most, np.float64) / 448.0)
    return np.where(np.asarray(most) > 0, np.maximum(e - (m == 0.5), -120), -120).astype(np.int64)


def append8(codes, exps, x, context, page_table):
    """One sequence's block x [n, heads, dim], rotated already, into codes [pages, size, heads, dim] (as the e4m3 numbers they are) and the
    exponents of the scales [pages, heads], both in place."""
    n, size = len(x), codes.shape[1]
    i = 0
    while i < n:
        page, place = int(page_table[(context + i) // size]), (context + i) % size
        m = min(n - i, size - place)
        part = x[i:i + m]
        e = scale_exponent(np.where(np.isfinite(part), np.abs(part), 0.0).max((0, 2)))
        if place:
            e = np.maximum(e, exps[page])
            codes[page, :place] = e4m3_grid(codes[page, :place] * np.exp2(exps[page] - e)[:, None])
        exps[page] = e
        codes[page, place:place + m] = e4m3_grid(part * np.exp2(-e)[:, None])
        i += m


def commit8(codes, exps, context, page_table, accept_len, path):
    """One sequence: the accepted path in codes [layers, pages, size, heads, dim], exps [layers, pages, heads], in place."""
    size = codes.shape[2]

    def at(slot):
        return int(page_table[slot // size]), slot % size
    j = 0
    while j < accept_len:
        page, place = at(context + 1 + j)
        m = min(accept_len - j, size - place)
        src = [at(context + int(p)) for p in path[j:j + m]]
        e = np.max([exps[:, page]] + [exps[:, p] for p, _ in src], 0)
        came = [e4m3_grid(codes[:, p, o] * np.exp2(exps[:, p] - e)[..., None]) for p, o in src]
        codes[:, page, :place] = e4m3_grid(codes[:, page, :place] * np.exp2(exps[:, page] - e)[:, None, :, None])
        exps[:, page] = e
        for k, c in enumerate(came):
            codes[:, page, place + k] = c
        j += m
    return context + 1 + accept_len


# ---- pages ---------------------------------------------------------------------------------------------------------------------

def fork(refs, context, table, src, reserve, size):
    """(table, context, refs, copies) of the new batch: copies (from, to, tokens)."""
    refs, width = [int(r) for r in refs], len(table[0])
    for row in table:
        for p in row:
            if p >= 0:
                refs[p] -= 1
    rows, ctx, keeps = [], [], set()
    for b in src:
        c = int(context[b]) if b >= 0 else 0
        ctx.append(c)
        rows.append([int(p) for p in table[b][:c // size]] if b >= 0 else [])
        for p in rows[-1]:
            refs[p] += 1
    for j, b in enumerate(src):
        if b >= 0 and ctx[j] % size and refs[table[b][ctx[j] // size]] == 0:
            refs[table[b][ctx[j] // size]] = 1
            keeps.add(j)
    free = [p for p, r in enumerate(refs) if r == 0]
    copies = []
    for j, b in enumerate(src):
        if b < 0:
            rows[j] = [-1] * width
            continue
        if j in keeps:
            rows[j].append(int(table[b][ctx[j] // size]))
        while len(rows[j]) * size < ctx[j] + reserve:
            p = free.pop(0) if free else -1
            if len(rows[j]) == ctx[j] // size and ctx[j] % size and p >= 0:
                copies.append((int(table[b][ctx[j] // size]), p, ctx[j] % size))
            rows[j].append(p)
            if p >= 0:
                refs[p] = 1
        rows[j] += [-1] * (width - len(rows[j]))
    return rows, ctx, refs, copies


def compact(refs):
    """(new number of each page, -1 for a free one; refs; pages held)."""
    refs = [int(r) for r in refs]
    held = [p for p, r in enumerate(refs) if r > 0]
    live = len(held)
    holes = iter([p for p in range(live) if refs[p] <= 0])
    to = [-1] * len(refs)
    for p in held:
        to[p] = p if p < live else next(holes)
    after = [0] * len(refs)
    for p in held:
        after[to[p]] = refs[p]
    return to, after, live
