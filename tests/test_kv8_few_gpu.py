"""GPU tests of the few-row attention kernel over codes: blocks that work on many short sequences one after the other."""
import numpy as np
import pytest
import torch

from kv8_helpers import Cache8, check_attend8
from kv_helpers import random_tree

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_gb300 as sv
    sv.load()
    return sv


def short_sequences(seed, B, n, H, kv, dim, page=32):
    """Contexts of one, two and three tiles of 128 tokens (the block's own among them) in changing order: three, one, two; three, one, one, two; and
    others."""
    rng = np.random.default_rng(seed)
    runs = [(3, 1, 2), (3, 1, 1, 2), (1, 3, 1, 3), (3, 3, 1, 1, 1, 2), (2, 1, 3, 1), (1, 1, 1)]
    tiles = []
    while len(tiles) < B:
        tiles += runs[rng.integers(len(runs))]
    contexts = [128 * t - n - int(rng.integers(0, 90)) for t in tiles[:B]]
    c = Cache8(seed, BF, contexts, n, kv, dim, page, spread=2)
    g = torch.Generator().manual_seed(seed)
    own = torch.randn((2, B * n, kv, dim), generator=g)
    b, t = np.repeat(np.arange(B), n), np.concatenate([x + np.arange(n) for x in contexts])
    at = torch.tensor(c.table.numpy()[b, t // page].astype(np.int64)).cuda(), torch.tensor(t % page).cuda()
    for codes, x in ((c.k8, own[0]), (c.v8, own[1])):
        codes.view(torch.uint8)[at] = (x * 64).clamp(-448, 448).to(codes.dtype).view(torch.uint8).cuda()
    c.refresh()
    return c, torch.randn((B, n, H, dim), generator=g).to(BF).cuda()


@pytest.mark.parametrize("n,H,kv,dim,tree", [(4, 4, 1, 64, False), (7, 4, 1, 128, True), (32, 1, 1, 64, True), (1, 8, 1, 128, False), (3, 8, 2, 128, False),
                                             (5, 6, 3, 80, False)])
@pytest.mark.parametrize("B", [700, 1100])
def test_many_short_sequences_of_one_to_three_tiles(sv, n, H, kv, dim, tree, B):
    c, q = short_sequences(B + dim + n, B, n, H, kv, dim)
    par = random_tree(c.rng, B, n) if tree else None
    kw = dict(parents=par.cuda()) if tree else {}
    out, lse = sv.sv_kv_attend8(q, *c.args8, lse=True, **kw)
    for _ in range(5):
        again = sv.sv_kv_attend8(q, *c.args8, lse=True, **kw)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    check_attend8(c, q.flatten(0, 1), out.flatten(0, 1), lse.flatten(0, 1), dim ** -0.5, [slice(b * n, b * n + n) for b in range(B)], par)
