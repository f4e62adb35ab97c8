"""The weights' bits in bf16 attention over codes, few rows.  A weight enters the product with the codes as two binary16 parts: one rounded to 11
bits, and 2^11 times what that leaves, rounded to 11 again: within 2^-22 of it, or 2^-36 where 2^4 is the row's largest weight (half of
binary16's last step, of 2^-11).  With one part it would be off by up to 2^-11.  The values here cancel: sum w v is thousands of times smaller than sum w |v|, so neither the rounding of the output nor
other tokens hide what a weight lacks.

Scores are exact: a query holds one 1, so q.k is an element of k, and the scale is 1.  Twelve tokens count, or twice that; the others' scores are -32.
What is left, relative to sum w |v| where each row's weights add up to 1:
  2^-21            the two parts, and what is left of the tokens at -32 (the tall kernel's two bf16 parts: 2^-16)
  2^-40 sum |v| * the largest weight's share   the parts' end
  2^-19            the exponent x = s log2(e) - m, |x| <= 12: one rounding each of the constant, the maximum and x, and exp2's 2^-22
  (2^-18 beside a token of score 16 that has nearly all the weight, and no value: |x| <= 29)
  (24 + 64) 2^-23  sums in float32, whichever way the products round
and the output's rounding, 2^-8 |out|."""
import numpy as np
import pytest
import torch

from kv8_helpers import E4M3, Cache8
from kv_helpers import f64
from oracle import kv as okv

BF = torch.bfloat16
COUNT = 12


def cancelling(seed, dim):
    """Scores s [COUNT] in [-4, 4] and values v [COUNT, dim], both numbers of e4m3's grid, with a small sum of exp(s) v: the last six tokens make
    up for what is left in turn, each to a sixteenth."""
    rng = np.random.default_rng(seed)
    s = okv.e4m3_grid(rng.uniform(-4, 4, COUNT).astype(np.float32)).astype(np.float64)
    w = np.exp(s)
    v = okv.e4m3_grid((rng.normal(size=(COUNT, dim)) * 16).astype(np.float32)).astype(np.float64)
    for i in range(COUNT - 6, COUNT):
        v[i] = 0.0
        v[i] = okv.e4m3_grid(np.clip(-(w @ v) / w[i], -448, 448).astype(np.float32))
    return s, v


def bound(wabs, want, vabs, top, parts=2.0 ** -21, end=2.0 ** -40, exponent=2.0 ** -19):
    return (parts + exponent + (2 * COUNT + 64) * 2.0 ** -23) * wabs + end * vabs * top + 2.0 ** -8 * np.abs(want) + 1e-30


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lead", [None, 16.0])
def test_bound_tells_the_parts_apart(dim, lead):
    """In the oracle, with the weights rounded to one part and to two, as a share of a row's largest, 2^4: the bound takes two and refuses one, and two
    without the 2^11 where a token of score `lead` has nearly all the weight."""
    refused, refused11 = 0, 0
    for seed in range(20):
        s, v = cancelling(seed, dim)
        if lead:
            s, v = np.append(s, lead), np.append(v, np.zeros((1, dim)), 0)
        w = 16 * np.exp(s - s.max())
        want, wabs, vabs = w @ v / w.sum(), w @ np.abs(v) / w.sum(), np.abs(v).sum(0)
        assert np.median(np.abs(want) / wabs) < 2.0 ** -12
        hi = w.astype(np.float16).astype(np.float64)
        lo = ((w - hi) * 2048).astype(np.float16).astype(np.float64) / 2048
        tol = bound(wabs, want, vabs, 16 / w.sum())
        assert np.all(np.abs((hi + lo) @ v / w.sum() - want) <= tol)
        refused += np.sum(np.abs(hi @ v / w.sum() - want) > tol)
        refused11 += np.sum(np.abs((hi + (w - hi).astype(np.float16)) @ v / w.sum() - want) > tol)
        assert np.sum(np.abs((hi + np.roll(lo, 1)) @ v / w.sum() - want) > tol) > dim // 8
    assert refused > 20 * dim // 4 and (lead is None or refused11 > 20 * dim // 2)


@pytest.mark.gpu
@pytest.mark.parametrize("n,heads,kv,dim", [(1, 2, 2, 128), (5, 8, 2, 128), (4, 16, 2, 64), (3, 4, 2, 96), (32, 2, 2, 128), (8, 4, 1, 48), (60, 4, 2, 128)])
@pytest.mark.parametrize("pre", [0, 128, 144])
@pytest.mark.parametrize("rest,lead", [(0, None), (1, None), (6, None), (0, 16.0)])
def test_two_part_weights(n, heads, kv, dim, pre, rest, lead):
    """Both tensor-core kernels (up to 32 packed rows and more), alone and behind a prefix that holds whole tiles or ends inside one; contexts that blocks
    share; `rest`: a first page (of zeros) whose scale is more than 2^40 times the values', which are then taken as 2^-40 of it with 2^-rest on the weights: their
    end is 2^rest further up; `lead`: a token of that score, without value."""
    import speculative_decoding_verification_gb300 as sv
    page = 16
    ctx = [pre + 40, pre + 127, pre + 700, pre + 6000, pre + 33]
    B = len(ctx)
    c = Cache8(n + dim, BF, ctx, n, kv, dim, page, groups=[(0, pre)] if pre else None)
    for x in (c.k8, c.v8):
        x.view(torch.uint8).zero_()
    c.ks.fill_(127)
    c.vs.fill_(127 - rest)
    low, rng = torch.tensor(-32.0).to(E4M3), np.random.default_rng(n)
    c.k8.view(torch.uint8)[..., 1] = low.view(torch.uint8).cuda()
    for b in range(B):
        for first, end in ((0, pre), (pre, ctx[b])):
            if end - first < 2 * page or (first == 0 and b > 0):   # the prefix is one for all
                continue
            at = first + page + np.sort(rng.choice(end - first - page, COUNT, replace=False))
            p, o = c.table[b].numpy()[at // page].astype(np.int64), at % page
            for h in range(kv):
                s, v = cancelling(100 * b + 10 * h + (first == 0), dim)
                c.k8[p, o, h, 1] = torch.tensor(s, dtype=torch.float32).to(E4M3).cuda()
                c.v8[p, o, h] = torch.tensor(v, dtype=torch.float32).to(E4M3).cuda()
            if lead:
                p, o = int(c.table[b, first // page]), first % page
                c.k8.view(torch.uint8)[p, o, :, 1] = torch.tensor(lead).to(E4M3).view(torch.uint8).cuda()
        if rest:
            c.vs[c.table[b, pre // page].long()] = 127 + 45
    c.refresh()
    q = torch.zeros(B, n, heads, dim, dtype=BF, device="cuda")
    q[..., 1] = 1.0
    out, _ = sv.sv_kv_attend8(q, *c.args8, scale=1.0, **c.group_args)
    k64, v64 = f64(c.k), f64(c.v)
    for b in range(B):
        want, lse, wabs, _ = okv.attend(f64(q[b]), k64, v64, ctx[b], c.table[b].numpy(), 1.0)
        pg, o = okv.slots(c.table[b].numpy(), page, ctx[b] + n)
        vabs = np.abs(v64[pg, o]).sum(0)[np.arange(heads) * kv // heads]
        top = np.exp(k64[pg, o][..., 1].max(0))[np.arange(heads) * kv // heads]
        tall = pre > 0 or n * (heads // kv) > 32
        tol = bound(wabs, want, vabs, (top / np.exp(lse))[..., None], 2.0 ** -16 if tall else 2.0 ** -21, 2.0 ** (rest - 40),
                    2.0 ** -18 if lead else 2.0 ** -19)
        assert np.all(np.abs(f64(out[b]) - want) <= tol), (b, float((np.abs(f64(out[b]) - want) / tol).max()))
        assert np.median(np.abs(want) / wabs.clip(1e-30)) < 2.0 ** -10   # the sums do cancel
