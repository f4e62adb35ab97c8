"""Greedy decoding with drafted trees through the library, end to end on the target's side.

Three sequences share a prompt.  Each round drafts a tree of `branches` paths of `depth` tokens a sequence, runs a small
target model over the last committed token and the drafted ones (sv_kv_append and sv_kv_attend in every layer), verifies
the tree (sv_tree_verify), and keeps the accepted path in the cache (sv_kv_commit).  The tokens that come out are those of
plain greedy decoding, whatever was drafted.

    python examples/tree_step.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verification_gb300 as sv  # noqa: E402

LAYERS, HEADS, KV_HEADS, DIM, VOCAB, PAGE = 2, 8, 2, 32, 32, 16
WIDTH = HEADS * DIM


class Target:
    """A transformer of attention layers with random weights over a paged cache."""

    def __init__(self, seed=0, device="cuda", dtype=torch.float32):
        g = torch.Generator().manual_seed(seed)

        def w(*shape):
            return (torch.randn(shape, generator=g) / shape[0] ** 0.5).to(device, dtype)
        self.embed = torch.randn((VOCAB, WIDTH), generator=g).to(device, dtype)
        self.qkv = [w(WIDTH, (HEADS + 2 * KV_HEADS) * DIM) for _ in range(LAYERS)]
        self.out = [w(WIDTH, WIDTH) for _ in range(LAYERS)]
        self.head = w(WIDTH, VOCAB)
        freq, self.magnitude = sv.sv_rope_frequencies(DIM, 10000.0, "turns", factor=4.0, low=1.0, high=4.0, original_len=64)
        self.freq = torch.tensor(freq, device=device)

    def step(self, tokens, k_cache, v_cache, context_len, page_table, parents=None, **groups):
        """Logits [B, n, VOCAB] of a block of tokens int64 [B, n], which is appended to the cache."""
        x = self.embed[tokens]
        for i in range(LAYERS):
            q, k, v = (x @ self.qkv[i]).unflatten(-1, (-1, DIM)).split([HEADS, KV_HEADS, KV_HEADS], 2)
            q = sv.sv_kv_append(k, v, k_cache[i], v_cache[i], context_len, page_table, q=q, inv_freq=self.freq, magnitude=self.magnitude,
                                parents=parents)
            a, _ = sv.sv_kv_attend(q, k_cache[i], v_cache[i], context_len, page_table, parents=parents, **groups)
            x = x + a.flatten(2) @ self.out[i]
        return x @ self.head


def decode(rounds=8, branches=8, depth=3, prompt_len=40, seed=0, device="cuda"):
    """Returns (model, prompt, committed tokens of each sequence, accepted counts of each round)."""
    model = Target(seed, device)
    g = torch.Generator().manual_seed(seed + 1)
    B, n = 3, branches * depth + 1
    prompt = torch.randint(0, VOCAB, (prompt_len,), generator=g)
    # page tables: the prompt's whole pages are shared, its last tokens are each sequence's own copy
    shared = prompt_len // PAGE
    each = -(-(prompt_len % PAGE + rounds * (depth + 1) + n) // PAGE)
    pages = torch.randperm(shared + B * each, generator=g).int()
    table = torch.cat([pages[:shared].repeat(B, 1), pages[shared:].view(B, each)], 1).to(device)
    k_cache, v_cache = (torch.zeros((LAYERS, shared + B * each, PAGE, KV_HEADS, DIM), device=device) for _ in range(2))
    context = torch.zeros(B, dtype=torch.int32, device=device)
    if shared:   # the shared pages once, through the first sequence's table
        model.step(prompt[None, : shared * PAGE].to(device), k_cache, v_cache, context[:1], table[:1])
    context += shared * PAGE
    groups = dict(group_start=torch.tensor([0, B], dtype=torch.int32, device=device), prefix_len=context[:1].clone())
    rest = prompt[shared * PAGE:].repeat(B, 1).to(device)
    if rest.shape[1]:
        model.step(rest, k_cache, v_cache, context, table, **groups)
        context += rest.shape[1]
    last = torch.arange(B, device=device)          # each sequence goes on from a token of its own
    done = [[int(t)] for t in last]
    node = torch.arange(n - 1, dtype=torch.int32)
    parents = torch.where(node % depth == 0, 0, node).repeat(B, 1).to(device)
    greedy = torch.zeros(B, device=device)
    uniforms = torch.zeros((B, n), dtype=torch.float64, device=device)
    counts = []
    for _ in range(rounds):
        drafted = torch.randint(0, VOCAB, (B, n - 1), generator=g).to(device)
        first = torch.stack([torch.randperm(VOCAB, generator=g)[:branches] for _ in range(B)]).to(device)
        drafted[:, ::depth] = first                # the branches start with different tokens
        logits = model.step(torch.cat([last[:, None], drafted], 1), k_cache, v_cache, context, table, parents, **groups)
        accepted, tokens, path, _ = sv.sv_tree_verify(logits, logits, parents, drafted.int(), uniforms, greedy)
        context = sv.sv_kv_commit(k_cache, v_cache, context, table, accepted, path)
        last = tokens.gather(1, accepted[:, None].long())[:, 0].long()   # the correction: the next block's row 0
        for b, (row, k) in enumerate(zip(tokens.tolist(), accepted.tolist())):
            done[b] += row[: k + 1]
        counts.append(accepted.tolist())
    return model, prompt, done, counts


if __name__ == "__main__":
    _, _, done, counts = decode()
    for b, tokens in enumerate(done):
        print(f"sequence {b}: {tokens}")
    print("drafted tokens accepted in each round:", counts)
