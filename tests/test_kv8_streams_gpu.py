"""GPU tests of calls on a cache held in 8 bits that overlap (streams, graphs, host threads), that wait in vain, and of caches laid out in other
ways: each result has to equal that of the same call made alone over plain arrays, bit for bit."""
import threading

import numpy as np
import pytest
import torch

from kv8_helpers import E4M3, Cache8, check_attend8
from kv_helpers import random_tree

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_gb300 as sv
    sv.load()
    return sv


class Call:
    """An attention call over its own cache.  Contexts long enough that units are split over blocks, so that the workspace is used."""

    def __init__(self, sv, seed, dtype, B, n, heads, kv, dim, longest, page=16, groups=None, step=37):
        self.sv = sv
        g = torch.Generator().manual_seed(seed)
        ctx = [longest - step * (b % 40) for b in range(B)]
        self.c = Cache8(seed, dtype, ctx, n, kv, dim, page, groups=groups, spread=2)
        for b in range(B):
            self.c.put(b, ctx[b], torch.randn((n, kv, dim), generator=g), torch.randn((n, kv, dim), generator=g))
        self.q = torch.randn((B, n, heads, dim), generator=g).to(dtype).cuda()
        self.alone = self.run(workspace=sv.Workspace())
        torch.cuda.synchronize()

    def run(self, **kw):
        return self.sv.sv_kv_attend8(self.q, *self.c.args8, lse=True, **self.c.group_args, **kw)

    def same(self, got):
        return all(torch.equal(a, b) for a, b in zip(got, self.alone))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_two_streams_without_workspace(sv, dtype):
    calls = [Call(sv, 1, dtype, 7, 4, 8, 2, 128, 3000), Call(sv, 2, dtype, 3, 40, 8, 2, 64, 2500)]
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[], []]
    torch.cuda.synchronize()
    for _ in range(20):
        for call, s, to in zip(calls, streams, got):
            to.append(call.run(stream=s))
    torch.cuda.synchronize()
    assert all(call.same(x) for call, to in zip(calls, got) for x in to)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_replay_after_larger_calls(sv, dtype):
    """A captured call keeps its workspace, whatever is called and allocated afterwards."""
    small, large = Call(sv, 3, dtype, 5, 3, 8, 2, 64, 2000), Call(sv, 4, dtype, 6, 300, 8, 2, 128, 900)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = small.run()
    assert large.same(large.run())
    side = torch.cuda.Stream()
    for _ in range(5):
        torch.cuda.synchronize()
        for t in out:
            t.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        again = large.run()   # beside the replay
        torch.cuda.synchronize()
        assert small.same(out) and large.same(again)


def test_graphs_that_share_a_workspace(sv):
    """Two captured calls of different sizes with one workspace, replayed in turn on one stream."""
    ws = sv.Workspace()
    calls = [Call(sv, 5, BF, 6, 4, 8, 2, 128, 3000), Call(sv, 6, BF, 9, 50, 8, 2, 64, 2500), Call(sv, 7, F32, 3, 2, 8, 2, 64, 3500)]
    for c in calls:
        c.run(workspace=ws)   # at its full size before the captures
    graphs, outs = [], []
    for c in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(c.run(workspace=ws))
    for _ in range(4):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(c.same(o) for c, o in zip(calls, outs))


def test_threads_on_one_stream(sv):
    """Two host threads whose launches alternate on one stream, with kernels that take shared memory by the head width."""
    calls = [Call(sv, 8, BF, 7, 4, 8, 2, 128, 3000), Call(sv, 9, F32, 5, 2, 8, 4, 64, 2500)]
    got, errors = [[], []], []

    def work(call, to):
        try:
            for _ in range(100):
                to.append(call.run())
        except Exception as e:   # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=a) for a in zip(calls, got)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    assert all(call.same(x) for call, to in zip(calls, got) for x in to)


@pytest.mark.parametrize("B,n,heads,kv,dim,longest,pre", [(7, 4, 8, 2, 128, 3000, 0), (9, 3, 4, 4, 64, 2500, 0), (5, 40, 8, 2, 128, 2000, 0),
                                                          (4, 150, 4, 2, 64, 1500, 0), (60, 4, 16, 8, 128, 1700, 1152),
                                                          (160, 1, 8, 8, 64, 500, 0)])
def test_waits_that_give_up(sv, B, n, heads, kv, dim, longest, pre):
    """A barrier that nothing completes: the waits give up, the call ends with a report, and calls after it are as before it."""
    call = Call(sv, n, BF, B, n, heads, kv, dim, longest, groups=[(0, pre)] if pre else None, step=5)
    lib = sv.load()

    def run():
        st = sv.new_stats("cuda")
        return call.run(stats=st), sv.read_stats(st)["status"]
    for limit in (2_000_000, 200_000):   # about 1 and 0.1 ms
        lib.sv_selftest_attend_stall(limit)
        try:
            assert run()[1] == 4   # timed out
        finally:
            lib.sv_selftest_attend_stall(0)
        for _ in range(3):
            again, status = run()
            assert status == 0 and call.same(again)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [4, 40])
def test_ragged_blocks_after_shared_prefixes(sv, dtype, n):
    """Blocks of n, 1, 0, n - 1 and 2 rows over two groups."""
    page, sizes = 16, [n, 1, 0, n - 1, 2]
    contexts = [320, 325, 400, 161, 200]
    c = Cache8(n, dtype, contexts, n, 2, 64, page, groups=[(0, 320), (3, 160)], spread=2)
    g = torch.Generator().manual_seed(n)
    for b, (ctx, m) in enumerate(zip(contexts, sizes)):
        c.put(b, ctx, torch.randn((m, 2, 64), generator=g), torch.randn((m, 2, 64), generator=g))
    c.refresh()
    start = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    q = torch.randn((int(start[-1]), 8, 64), generator=g).to(dtype).cuda()
    st = sv.new_stats("cuda")
    out, lse = sv.sv_kv_attend8(q, *c.args8, row_start=torch.tensor(start).cuda(), max_rows=n, lse=True, stats=st, **c.group_args)
    assert sv.read_stats(st)["status"] == 0
    check_attend8(c, q, out, lse, 64 ** -0.5, [slice(int(a), int(b)) for a, b in zip(start, start[1:])])


def step(sv, caches, scales, table, contexts, tree, q, k, v, freq, acc, path):
    """Append, attention and commit of one block; the caches have a layer axis."""
    one, two = [x[1] for x in (*caches, *scales)], torch.tensor(contexts, dtype=torch.int32).cuda()
    turned = sv.sv_kv_append8(k, v, *one, two, table, q=q, inv_freq=freq, parents=tree)
    out = sv.sv_kv_attend8(turned, *one, two, table, parents=tree, lse=True)
    return (*out, turned, sv.sv_kv_commit8(*caches, *scales, two, table, acc, path))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [6, 50])
def test_interleaved_and_padded_arrays(sv, dtype, n):
    """Keys and values in one allocation, scales of both in one array, heads and rows of one projection, a page table with a pitch, scales of
    the other dtype: the same bits as plain arrays, and nothing between them is touched."""
    rng = np.random.default_rng(n)
    L, P, page, kv, H, D, B = 3, 60, 8, 3, 6, 64, 4
    contexts = [0, 3, 40, 63]
    raw = [torch.tensor((rng.integers(0, 0x78, (L, P, page, kv, D)) | rng.integers(0, 2, (L, P, page, kv, D)) << 7).astype(np.uint8)).cuda() for _ in range(2)]
    byte = [torch.tensor(rng.integers(115, 125, (L, P, kv)).astype(np.uint8)).cuda() for _ in range(2)]
    ids = torch.tensor(rng.permutation(P)[:B * 15].reshape(B, 15).astype(np.int32)).cuda()
    tree = random_tree(rng, B, n).cuda()
    qkv = torch.tensor(rng.normal(size=(B, n, H + 2 * kv, D)), dtype=dtype).cuda()
    q, k, v = qkv[:, :, :H], qkv[:, :, H:H + kv], qkv[:, :, H + kv:]
    freq = torch.tensor(10000.0 ** (-np.arange(32) / 32), dtype=F32).cuda()
    acc = torch.tensor([0, n - 1, 2, 3], dtype=torch.int32).cuda()
    path = torch.tensor(np.stack([np.arange(1, n)] * B).astype(np.int32)).cuda()
    path[2, :2] = torch.tensor([2, 5]).cuda()
    plain = [x.clone() for x in raw], [x.clone() for x in byte]
    want = step(sv, [x.view(E4M3) for x in plain[0]], plain[1], ids, contexts, tree, q.contiguous(), k.contiguous(), v.contiguous(), freq, acc, path)
    pool = torch.full((L, P, 2, kv, page, D + 32), 0xA5, dtype=torch.uint8, device="cuda")
    caches = [pool[:, :, i, :, :, :D].transpose(2, 3) for i in range(2)]
    both = torch.full((P, L, 2 * kv + 1), 0x5A, dtype=torch.uint8, device="cuda")
    scales = [both[:, :, i:i + 2 * kv:2].transpose(0, 1) for i in range(2)]
    for to, x in zip((*caches, *scales), (*raw, *byte)):
        to.copy_(x)
    wide = torch.full((B, 20), -1, dtype=torch.int32, device="cuda")
    wide[:, :15] = ids
    got = step(sv, [x.view(E4M3) for x in caches], [s.view(torch.float8_e8m0fnu) for s in scales], wide[:, :15], contexts, tree, q, k, v, freq, acc, path)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for to, x in zip((*caches, *scales), (*plain[0], *plain[1])):
        assert torch.equal(to.contiguous(), x)
    assert bool((pool[..., D:] == 0xA5).all()) and bool((both[:, :, 2 * kv] == 0x5A).all())


@pytest.mark.parametrize("dtype,n", [(BF, 5), (BF, 40), (F32, 2)])
def test_pages_beyond_four_gigabytes(sv, dtype, n):
    """A step over pages at a large pool's far end is that over the same pages at its start; compaction brings them back."""
    rng = np.random.default_rng(n)
    P, page, kv, H, D, B = 270_000, 16, 8, 16, 128, 3
    contexts = [0, 500, 1000]
    caches = [torch.zeros((2, P // 2, page, kv, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros((2, P // 2, kv), dtype=torch.uint8, device="cuda") for _ in range(2)]
    each = 1064 // page
    low = torch.tensor(rng.permutation(B * each).reshape(B, each).astype(np.int32)).cuda()
    far = low + (P // 2 - B * each)
    for c, s in zip(caches, scales):
        c[:, :B * each] = torch.tensor(rng.integers(0, 0x78, (2, B * each, page, kv, D)).astype(np.uint8)).cuda()
        s[:, :B * each] = torch.tensor(rng.integers(115, 125, (2, B * each, kv)).astype(np.uint8)).cuda()
        c[:, -B * each:], s[:, -B * each:] = c[:, :B * each].clone(), s[:, :B * each].clone()
    tree = random_tree(rng, B, n).cuda()
    q, k, v = (torch.tensor(rng.normal(size=(B, n, h, D)), dtype=dtype).cuda() for h in (H, kv, kv))
    freq = torch.tensor(10000.0 ** (-np.arange(64) / 64), dtype=F32).cuda()
    acc = torch.tensor([0, n - 1, 1], dtype=torch.int32).cuda()
    path = torch.tensor(np.stack([np.arange(1, n)] * B).astype(np.int32)).cuda()
    args = ([x.view(E4M3) for x in caches], scales)
    near = step(sv, *args, low, contexts, tree, q, k, v, freq, acc, path)
    there = step(sv, *args, far, contexts, tree, q, k, v, freq, acc, path)
    assert all(torch.equal(a, b) for a, b in zip(near, there))
    for x in (*caches, *scales):
        assert torch.equal(x[:, :B * each], x[:, -B * each:])
    start = [x[:, :B * each].clone() for x in (*caches, *scales)]
    refs = torch.zeros(P // 2, dtype=torch.int32, device="cuda")
    refs[-B * each:] = 1
    for x in (*caches, *scales):
        x[:, :B * each] = 0
    table, after, live = sv.sv_kv_compact(*args[0], refs, far, k_scale=scales[0], v_scale=scales[1])
    assert int(live) == B * each and torch.equal(table, low) and bool((after[:B * each] == 1).all()) and int(after.sum()) == B * each
    for x, s in zip((*caches, *scales), start):
        assert torch.equal(x[:, :B * each], s)
