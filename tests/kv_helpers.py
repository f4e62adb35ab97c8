"""Inputs of the cache and attention tests: a paged cache whose unused slots hold NaN, blocks, and the float64
oracle's answers for them."""
from __future__ import annotations

import numpy as np
import torch

from oracle import kv as okv

U32, U16 = 2.0 ** -24, 2.0 ** -9   # unit roundoffs of float32 and bfloat16


def f64(t):
    return t.detach().to("cpu").to(torch.float64).numpy()


def random_tree(rng, B, n):
    return torch.tensor([[rng.integers(0, i) if rng.random() < 0.5 else i - 1 for i in range(1, n)] for _ in range(B)],
                        dtype=torch.int32).reshape(B, n - 1)


class Cache:
    """Paged caches k, v [pages, size, heads, dim] on the GPU with `order` axes in memory, page tables that scatter each
    sequence, and per-sequence contexts; every slot that is no cached token holds NaN."""

    def __init__(self, seed, dtype, contexts, n, kv_heads, dim, page, order="psh", groups=None, together=False):
        self.rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        B = len(contexts)
        each = max((c + n + page - 1) // page for c in contexts) + 1
        P = B * each + 3
        perm = self.rng.permutation(P)
        table = perm[: B * each].reshape(B, each).copy()
        self.groups = groups   # list of (first sequence, prefix length) with whole pages shared
        shape = (P, page, kv_heads, dim)
        data = [torch.full(shape, float("nan"), dtype=torch.float32) for _ in range(2)]
        if groups:
            bounds = [b for b, _ in groups] + [B]
            for (b0, pre), b1 in zip(groups, bounds[1:]):
                table[b0:b1, : pre // page] = table[b0, : pre // page]
        for b, c in enumerate(contexts):
            t = np.arange(c)
            for x in data:
                x[table[b][t // page], t % page] = torch.randn((c, kv_heads, dim), generator=g)
        if groups:   # a prefix's last, partly filled page is every sequence's own copy
            for (b0, pre), b1 in zip(groups, bounds[1:]):
                t = np.arange(pre - pre % page, pre)
                for b in range(b0 + 1, b1):
                    for x in data:
                        x[table[b][t // page], t % page] = x[table[b0][t // page], t % page].clone()
        if together:   # keys and values interleaved in one allocation
            pool = torch.stack(data, 1).to(dtype).cuda()
            self.k, self.v = pool[:, 0], pool[:, 1]
        else:
            axes = {"psh": (0, 1, 2, 3), "phs": (0, 2, 1, 3), "hps": (2, 0, 1, 3)}[order]
            back = tuple(int(i) for i in np.argsort(axes))
            self.k, self.v = (x.to(dtype).permute(axes).contiguous().cuda().permute(back) for x in data)
        self.contexts = list(contexts)
        self.table = torch.tensor(table, dtype=torch.int32)
        self.args = dict(context_len=torch.tensor(contexts, dtype=torch.int32).cuda(), page_table=self.table.cuda())
        if groups:
            self.group_args = dict(group_start=torch.tensor(bounds, dtype=torch.int32).cuda(),
                                   prefix_len=torch.tensor([p for _, p in groups], dtype=torch.int32).cuda())
        else:
            self.group_args = {}

    def put(self, b, first, k, v):
        """Writes rows k, v [n, heads, dim] to slots first.. of sequence b."""
        t = np.arange(first, first + len(k))
        page = self.k.shape[1]
        at = torch.tensor(self.table.numpy()[b][t // page], device="cuda"), torch.tensor(t % page, device="cuda")
        self.k[at] = k.to(self.k.dtype).cuda()
        self.v[at] = v.to(self.v.dtype).cuda()


def check_attend(cache, q, out, lse, scale, rows_of, parents=None, seqs=None):
    """out, lse of sv_kv_attend against the oracle.  rows_of[b] = slice of the flat rows of sequence b.

    Error of a score: D products and sums in float32, and the scaling: ds <= (D + 8) u32 scale sum|q k|.  A weight is
    off by 2 ds relative (its own score and the maximum it is taken from cancel, the sum's do not) plus a few u32 of exp and
    the rescalings; bf16 weights round once more (u16) in the product with v.  So
      |out error| <= (2 ds + (n + 64) u32 [+ u16]) sum w|v| [+ u16 |out|],  |lse error| <= ds + (n + 64) u32 + 4 u32 |lse|,
    with n the number of tokens that a sum runs over (its worst case; sums of partial sums do better)."""
    k64, v64, q64, o64, l64 = f64(cache.k), f64(cache.v), f64(q), f64(out), f64(lse)
    bf16 = q.dtype == torch.bfloat16
    D = q.shape[-1]
    for b in range(len(cache.contexts)) if seqs is None else seqs:
        r = rows_of[b]
        if r.stop == r.start:
            continue
        c = cache.contexts[b]
        par = None if parents is None else parents[b].tolist()
        want, wl, wabs, big = okv.attend(q64[r], k64, v64, c, cache.table[b].numpy(), scale, par)
        n = c + (r.stop - r.start)
        ds = (D + 8) * U32 * big
        tol = (2 * ds + (n + 64) * U32 + (U16 if bf16 else 0.0))[..., None] * wabs + (U16 if bf16 else 0.0) * np.abs(want) + 1e-30
        err = np.abs(o64[r] - want)
        assert np.all(err <= tol), (b, float((err / tol).max()))
        ltol = ds + (n + 64) * U32 + 4 * U32 * np.abs(wl)
        assert np.all(np.abs(l64[r] - wl) <= ltol), (b, float((np.abs(l64[r] - wl) / ltol).max()))
