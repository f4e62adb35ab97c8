"""GPU tests of a prompt's append to a cache held in 8 bits: thousands of rows of one sequence, whole and in parts."""
import numpy as np
import pytest
import torch

from kv8_helpers import values
from kv_helpers import f64
from oracle import kv as okv
from test_kv8_gpu import BF, F32, AppendCase, exps, same_codes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_gb300 as sv
    sv.load()
    return sv


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,contexts,page,kv,dim", [(2049, [0], 16, 8, 128), (1300, [0, 77], 100, 2, 64), (4000, [5], 64, 1, 96), (515, [0, 1, 300], 7, 9, 16),
                                                    (1000, [24], 1, 3, 48), (777, [1000], 1024, 4, 256)])
def test_a_prompt_is_the_oracles_to_the_bit(sv, dtype, n, contexts, page, kv, dim):
    """Without rotation: codes and scales are the oracle's, other pages and slots as they were."""
    c = AppendCase(n, dtype, contexts, n, kv, kv, dim, page)
    c.run(sv)
    for x, cache, scale, (codes, e) in zip((c.k, c.v), c.caches, c.scales, c.before):
        for b, ctx in enumerate(c.contexts):
            okv.append8(codes, e, f64(x[b]), ctx, c.table[b].numpy())
        np.testing.assert_array_equal(exps(scale), e)
        same_codes(cache, codes)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("style,rotary,page", [("half", 128, 16), ("interleaved", 64, 100)])
def test_a_prompt_is_rotated_at_its_positions(sv, dtype, style, rotary, page):
    """As in the test of short blocks: keys are off by the rotation in float32, 5e-6 of the row's largest, and half a step of their code; queries by
    the same and their rounding."""
    n, ctx, H, kv, dim = 1500, 333, 4, 2, 128
    c = AppendCase(3, dtype, [ctx], n, H, kv, dim, page)
    freq, mag = okv.rope_frequencies(rotary)[0], 0.75
    got = c.run(sv, q=c.q.cuda(), inv_freq=torch.tensor(freq, dtype=F32).cuda(), style=style, magnitude=mag)
    f32freq, pos, t = np.asarray(freq, np.float32).astype(np.float64), ctx + np.arange(n), ctx + np.arange(n)
    q, k = (okv.rope(f64(x[0]), pos, f32freq, style, mag) for x in (c.q, c.k))
    unit = 2.0 ** -9 if dtype is BF else 2.0 ** -24
    assert (np.abs(f64(got[0]) - q) <= 2 * unit * np.abs(q) + 1e-5 * np.abs(f64(c.q[0])).max(-1, keepdims=True) + 1e-30).all()
    p, o = c.table[0].numpy()[t // page], t % page
    for which, x in ((0, k), (1, f64(c.v[0]))):
        have = values(c.caches[which], c.scales[which]).double().numpy()[p, o]
        scale = np.exp2(exps(c.scales[which])[p])[..., None]
        off = 5e-6 * np.abs(f64(c.k[0])).max(-1, keepdims=True) if which == 0 else 0.0
        assert (np.abs(have - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * scale) + 1.0001 * off).all()


def test_a_prompt_in_parts(sv):
    """Parts that end within pages: pages hold what the whole at once would, rounded once more where a part raised the scale."""
    n, page = 600, 32
    whole, parts = (AppendCase(9, BF, [0], n, 2, 2, 64, page) for _ in range(2))
    whole.run(sv)
    table = parts.table.cuda()
    for first, end in ((0, 1), (1, 130), (130, 144), (144, 500), (500, 600)):
        sv.sv_kv_append8(parts.k[:, first:end].contiguous().cuda(), parts.v[:, first:end].contiguous().cuda(), *parts.caches, *parts.scales,
                         torch.tensor([first], dtype=torch.int32).cuda(), table)
    used = parts.table[0, :-(-n // page)].long()
    t = np.arange(n)
    p, o = parts.table[0].numpy()[t // page], t % page
    for i, x in enumerate((whole.k, whole.v)):
        np.testing.assert_array_equal(exps(parts.scales[i])[used], exps(whole.scales[i])[used])   # the largest of a page is the same
        have = values(parts.caches[i], parts.scales[i]).double().numpy()[p, o]
        scale = np.exp2(exps(parts.scales[i])[p])[..., None]
        # a page gets up to three parts: two roundings to coarser scales after the first, each half a step of a subnormal code
        assert (np.abs(have - f64(x[0])) <= 2.0 ** -4 * np.abs(f64(x[0])) + 3 * 2.0 ** -10 * scale).all()
