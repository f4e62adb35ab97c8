"""Caches held in 8 bits for the tests: random codes and scales in any axis order, and the values they stand for."""
from __future__ import annotations

import numpy as np
import torch

from kv_helpers import U32, Cache, f64
from oracle import kv as okv

E4M3 = torch.float8_e4m3fn


def order_axes(x, order):
    """x [pages, size, heads, dim] laid out in memory with its first three axes in the order given."""
    axes = {"psh": (0, 1, 2, 3), "phs": (0, 2, 1, 3), "hps": (2, 0, 1, 3)}[order]
    return x.permute(axes).contiguous().permute(tuple(int(i) for i in np.argsort(axes)))


def values(codes, scale):
    """The numbers that codes [..., size, heads, dim] in scales (bytes) [..., heads] stand for, as float32."""
    e = scale.view(torch.uint8).cpu().double() - 127
    f = torch.where(e == 128, float("nan"), torch.exp2(e))
    return (codes.cpu().float().double() * f[..., None, :, None]).float()


class Cache8(Cache):
    """Cache (its page tables, contexts and groups) whose cached tokens are held in 8 bits; slots that are no cached token hold NaN codes.
    spread: scales are 2^-spread .. 2^spread times what a token needs."""

    def __init__(self, seed, dtype, contexts, n, kv_heads, dim, page, order="psh", groups=None, spread=0):
        super().__init__(seed, torch.float32, contexts, n, kv_heads, dim, page, groups=groups)
        k, v = self.k.cpu(), self.v.cpu()
        for name, x in (("k", k), ("v", v)):
            e = torch.tensor(self.rng.integers(-spread, spread + 1, (x.shape[0], kv_heads)))
            scale = (e - 6 + 127).to(torch.uint8)
            # the data grows with its page's scale, so that a head's pages differ in size as its scales do
            codes = (x * 64).to(E4M3)
            setattr(self, name + "8", order_axes(codes.view(torch.uint8), order).cuda().view(E4M3))
            setattr(self, name + "s", scale.cuda())
        self.dtype = dtype
        self.refresh()

    def refresh(self):
        """k, v: the values, as a cache of the queries' type."""
        self.k, self.v = (values(c, s).to(self.dtype).cuda() for c, s in ((self.k8, self.ks), (self.v8, self.vs)))

    @property
    def args8(self):
        return (self.k8, self.v8, self.ks, self.vs, self.args["context_len"], self.args["page_table"])

    def put(self, b, first, k, v):
        """Codes of rows k, v at slots first.. of sequence b, rounded in whatever scale their page has."""
        t = np.arange(first, first + len(k))
        page = torch.tensor(self.table.numpy()[b][t // self.k8.shape[1]].astype(np.int64))
        place = torch.tensor(t % self.k8.shape[1])
        for c, x in ((self.k8, k), (self.v8, v)):
            c.view(torch.uint8)[page.cuda(), place.cuda()] = (x * 64).clamp(-448, 448).to(E4M3).view(torch.uint8).cuda()


def check_attend8(cache, q, out, lse, scale, rows_of, parents=None):
    """out, lse of sv_kv_attend8 against the oracle over the values, as check_attend, with bf16's half step at its largest: numbers of [1, 2) are 2^-7
    apart, so rounding moves one by up to 2^-8 of it (not 2^-9: 1 + 2^-8 lies in the middle of 1 and 1 + 2^-7).  With ds the error of a score,
      |out error| <= (2 ds + (n + 64) u32 [+ 2^-12, a weight's one binary16 number]) sum w|v| [+ 2^-8 |out|],
    to which two-part bf16 weights add nothing, and a row that sees one token has the last term alone.  In the few-row kernel a query
    element is a binary16 number, exact but for those that end below its normal range: 2^-25 off, where the block's largest is 2^14 or more.  That
    adds 2^-39 max|q| scale max sum|k| to ds."""
    k64, v64, q64, o64, l64 = f64(cache.k), f64(cache.v), f64(q), f64(out), f64(lse)
    bf16 = q.dtype == torch.bfloat16
    for b, r in enumerate(rows_of):
        if r.stop == r.start:
            continue
        par = None if parents is None else parents[b].tolist()
        want, wl, wabs, big = okv.attend(q64[r], k64, v64, cache.contexts[b], cache.table[b].numpy(), scale, par)
        n = cache.contexts[b] + (r.stop - r.start)
        ds = (q.shape[-1] + 8) * U32 * big
        if bf16 and q.shape[-1] <= 128:
            page, place = okv.slots(cache.table[b].numpy(), k64.shape[1], n)
            ds = ds + 2.0 ** -39 * np.nanmax(np.abs(q64[r]), initial=0.0) * abs(scale) * np.abs(k64[page, place]).sum(-1).max(initial=0.0)
        tol = (2 * ds + (n + 64) * U32 + (2.0 ** -12 if bf16 else 0.0))[..., None] * wabs + (2.0 ** -8 if bf16 else 0.0) * np.abs(want) + 1e-30
        err = np.abs(o64[r] - want)
        assert np.all(err <= tol), (b, float((err / tol).max()))
        ltol = ds + (n + 64) * U32 + 4 * U32 * np.abs(wl)
        assert np.all(np.abs(l64[r] - wl) <= ltol), (b, float((np.abs(l64[r] - wl) / ltol).max()))
