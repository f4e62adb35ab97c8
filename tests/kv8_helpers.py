"""Caches held in 8 bits for the tests: random codes and scales in any axis order, and the values they stand for."""
from __future__ import annotations

import numpy as np
import torch

from kv_helpers import Cache

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
