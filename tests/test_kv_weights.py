"""The weights' bits in bf16 attention.  A weight enters the product with V as two bf16 parts that hold it within 2^-16; with the
upper part alone it would be off by up to 2^-7.  The values here cancel: sum w v is hundreds of times smaller than sum w |v|, so the
rounding of the output hides nothing, and a kernel that lost the lower parts, or put them beside the wrong values, fails.

Scores are exact: a query holds one 1, so q.k is an element of k, and the scale is 1.  What is left, relative to sum w |v| where each
row's weights add up to 1:
  2^-16            the two parts (the rest after cutting off 8 bits, rounded to 8 bits)
  2^-19            the exponent x = s log2(e) - m, |x| <= 12: one rounding each of the constant, the maximum and x, and exp2's 2^-22
  (n + 64) 2^-23   sums over n tokens in float32, whichever way the products round
and the output's rounding, 2^-8 |out| (bf16 has 8 significant bits: half the distance of 1 to 1 + 2^-7)."""
import numpy as np
import pytest
import torch

from kv_helpers import Cache, f64
from oracle import kv as okv

BF = torch.bfloat16
U16 = 2.0 ** -8


def bf16(x):
    return f64(torch.tensor(np.asarray(x), dtype=torch.float64).to(BF))


def cancelling(seed, n, dim):
    """Scores s [n] in [-4, 4] and values v [n, dim] of bf16 numbers with a small sum of exp(s) v."""
    rng = np.random.default_rng(seed)
    s = bf16(rng.uniform(-4, 4, n))
    v = bf16(rng.normal(size=(n, dim)))
    last = int(s.argmax())
    w = np.exp(s - s.max())
    v[last] = bf16(v[last] - w @ v)
    return s, v


def bound(n, wabs, want):
    return (2.0 ** -16 + 2.0 ** -19 + (n + 64) * 2.0 ** -23) * wabs + U16 * np.abs(want) + 1e-30


@pytest.mark.parametrize("n,dim", [(3, 64), (40, 128), (127, 64), (260, 128)])
def test_bound_tells_the_parts_apart(n, dim):
    """In the oracle, with the weights cut to one part and to two: the bound takes two and refuses one."""
    s, v = cancelling(n, n, dim)
    w = np.exp(s - s.max())
    want, wabs = w @ v / w.sum(), w @ np.abs(v) / w.sum()

    def cut(x):   # to 8 significant bits, towards zero
        step = 2.0 ** (np.floor(np.log2(np.maximum(x, 1e-30))) - 7)
        return np.floor(x / step) * step
    hi = cut(w)
    lo = bf16(w - hi * (1 - 2.0 ** -24))
    one, two = bf16(hi @ v / w.sum()), bf16((hi + lo) @ v / w.sum())
    assert np.all(np.abs(two - want) <= bound(n, wabs, want))
    assert np.sum(np.abs(one - want) > 4 * bound(n, wabs, want)) > dim // 4
    wrong = bf16((hi + np.roll(lo, 1)) @ v / w.sum())
    assert np.sum(np.abs(wrong - want) > 4 * bound(n, wabs, want)) > dim // 4


@pytest.mark.gpu
@pytest.mark.parametrize("n,heads,kv,dim", [(1, 2, 2, 128), (5, 8, 2, 128), (4, 16, 2, 64), (3, 4, 2, 96), (40, 8, 2, 128), (150, 2, 2, 64),
                                            (70, 4, 1, 96), (130, 4, 2, 128)])
@pytest.mark.parametrize("pre", [0, 128, 144])
def test_two_part_weights(n, heads, kv, dim, pre):
    """Both tensor-core kernels (up to 32 packed rows and more), alone, and behind a prefix that holds whole tiles or ends inside one.  The
    block's own values are zero, so every row's weighted values cancel."""
    import speculative_decoding_verification_gb300 as sv
    ctx = [pre + 40, pre + 127, pre + 128, pre + 230, pre + 5]
    B = len(ctx)
    c = Cache(n, BF, ctx, n, kv, dim, 16, groups=[(0, pre)] if pre else None)
    q = torch.zeros(B, n, heads, dim, dtype=BF, device="cuda")
    q[..., 1] = 1.0
    for b in range(B):
        for first, end in ((0, pre), (pre, ctx[b])):   # the prefix cancels by itself
            if end > first:
                keys, vals = torch.zeros(end - first, kv, dim), torch.zeros(end - first, kv, dim)
                for h in range(kv):
                    s, v = cancelling(7 * h + (first == pre) * (b + 1), end - first, dim)
                    keys[:, h, 1], vals[:, h] = torch.tensor(s), torch.tensor(v)
                c.put(b, first, keys, vals)
        own = torch.zeros(n, kv, dim)
        own[:, :, 1] = -3.0
        c.put(b, ctx[b], own, torch.zeros(n, kv, dim))
    out, _ = sv.sv_kv_attend(q, c.k, c.v, scale=1.0, **c.args, **c.group_args)
    k64, v64 = f64(c.k), f64(c.v)
    for b in range(B):
        want, _, wabs, _ = okv.attend(f64(q[b]), k64, v64, ctx[b], c.table[b].numpy(), 1.0)
        tol = bound(ctx[b] + n, wabs, want)
        assert np.all(np.abs(f64(out[b]) - want) <= tol), (b, float((np.abs(f64(out[b]) - want) / tol).max()))
        assert np.median(np.abs(want) / wabs.clip(1e-30)) < 2.0 ** -5   # the sums do cancel
