"""GPU test of the whole target side: decoding with drafted trees gives the tokens of plain greedy decoding, computed here
densely in float64 without a cache: each token's logit is the largest, up to 1e-3, hundreds of times float32's error in two
layers' sums of 256 terms of order one."""
import math
import os
import sys

import pytest
import torch

from oracle import kv as okv

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


def dense_next(model, tokens):
    """Logits after the last of `tokens`, every layer recomputed over the whole sequence in float64 on the host."""
    import tree_step as ex
    x = model.embed.double().cpu()[tokens]
    n = len(tokens)
    freq = model.freq.double().cpu().numpy()
    mask = torch.full((n, n), -math.inf).triu(1).double()
    for qkv, out in zip(model.qkv, model.out):
        q, k, v = (x @ qkv.double().cpu()).unflatten(-1, (-1, ex.DIM)).split([ex.HEADS, ex.KV_HEADS, ex.KV_HEADS], 1)
        q, k = (torch.from_numpy(okv.rope(t.numpy(), range(n), freq, "half", model.magnitude)) for t in (q, k))
        k, v = (t.repeat_interleave(ex.HEADS // ex.KV_HEADS, 1) for t in (k, v))
        s = torch.einsum("ihd,jhd->hij", q, k) / math.sqrt(ex.DIM) + mask
        x = x + torch.einsum("hij,jhd->ihd", torch.softmax(s, -1), v).flatten(1) @ out.double().cpu()
    return (x @ model.head.double().cpu())[-1]


@pytest.mark.parametrize("branches,depth,prompt_len", [(8, 3, 40), (4, 2, 32), (12, 1, 7)])
def test_tree_decoding_is_greedy_decoding(branches, depth, prompt_len):
    import tree_step as ex
    model, prompt, done, counts = ex.decode(rounds=6, branches=branches, depth=depth, prompt_len=prompt_len, seed=3)
    assert sum(map(sum, counts)) > 0   # some drafted tokens were accepted, so paths were moved
    for b, tokens in enumerate(done):
        seq = prompt.tolist() + tokens[:1]
        for t in tokens[1:]:
            logits = dense_next(model, seq)
            assert float(logits[t]) > float(logits.max()) - 1e-3   # the argmax, or as good as tied with it
            seq.append(t)
        assert len(tokens) == 1 + 6 + sum(c[b] for c in counts)
