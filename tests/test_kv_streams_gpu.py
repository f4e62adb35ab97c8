"""GPU tests of attention calls that overlap: on two streams, in captured graphs, from two host threads.  Every result has to equal
that of the same call made alone, bit for bit (partial sums are joined in a fixed order)."""
import threading

import pytest
import torch

from kv_helpers import Cache

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_gb300 as sv
    sv.load()
    return sv


class Call:
    """An attention call over its own cache.  Contexts long enough that units are split over blocks, so that the workspace is used."""

    def __init__(self, sv, seed, dtype, B, n, heads, kv, dim, longest):
        self.sv = sv
        g = torch.Generator().manual_seed(seed)
        ctx = [longest - 37 * b for b in range(B)]
        c = Cache(seed, dtype, ctx, n, kv, dim, 16)
        self.q = torch.randn((B, n, heads, dim), generator=g).to(dtype).cuda()
        for b in range(B):
            c.put(b, ctx[b], torch.randn((n, kv, dim), generator=g), torch.randn((n, kv, dim), generator=g))
        self.c = c
        self.alone = self.run(workspace=sv.Workspace())
        torch.cuda.synchronize()

    def run(self, **kw):
        return self.sv.sv_kv_attend(self.q, self.c.k, self.c.v, lse=True, **self.c.args, **kw)

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
    for call, s in zip(calls, streams):   # the stream as the current one
        with torch.cuda.stream(s):
            call.late = [call.run() for _ in range(10)]
    torch.cuda.synchronize()
    assert all(call.same(x) for call in calls for x in call.late)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_replay_after_larger_calls(sv, dtype):
    """A captured call keeps its workspace, whatever is called and allocated afterwards."""
    small, large = Call(sv, 3, dtype, 5, 3, 8, 2, 64, 2000), Call(sv, 4, dtype, 6, 300, 8, 2, 128, 900)
    small.run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = small.run()
    assert large.same(large.run())
    fill = [torch.full((1 << 22,), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(40)]
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
    assert all(bool((t == 0x7F).all()) for t in fill)


def test_results_of_another_stream_are_kept(sv):
    """Queries, results and workspaces dropped while the call's own stream is still behind: their memory is not given out before."""
    call = Call(sv, 5, BF, 6, 4, 8, 2, 128, 2000)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    kept = []
    for _ in range(5):
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)   # about 10 ms
        q = call.q.clone()
        s.wait_stream(torch.cuda.current_stream())
        kept.append(sv.sv_kv_attend(q, call.c.k, call.c.v, lse=True, stream=s, workspace=sv.Workspace(), **call.c.args))
        del q
        junk = [torch.full((call.q.numel(),), float("nan"), dtype=BF, device="cuda") for _ in range(4)]
        del junk
    torch.cuda.synchronize()
    assert all(call.same(x) for x in kept)


def test_threads_on_one_stream(sv):
    """Two host threads whose launches alternate on one stream."""
    calls = [Call(sv, 6, BF, 7, 4, 8, 2, 128, 3000), Call(sv, 7, F32, 5, 2, 8, 4, 64, 2500)]
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


def test_threads_with_other_head_widths(sv):
    """The float32 kernel of few rows takes shared memory by the head width: two threads with widths 128 and 64, on streams of their
    own, do not take it from each other."""
    calls = [Call(sv, 8, F32, 2, 1, 2, 1, 128, 100), Call(sv, 9, F32, 2, 1, 2, 1, 64, 100)]
    got, errors = [[], []], []

    def work(call, to):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(3000):
                    last = call.run()
                torch.cuda.current_stream().synchronize()
                to.append(last)
        except Exception as e:   # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=a) for a in zip(calls, got)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    assert all(call.same(x) for call, to in zip(calls, got) for x in to)


@pytest.mark.parametrize("B,n,heads,kv,dim,longest,pre", [(7, 4, 8, 2, 128, 3000, 0), (9, 3, 4, 4, 64, 2500, 0), (5, 40, 8, 2, 128, 2000, 0),
                                                          (4, 150, 4, 2, 64, 1500, 0), (60, 4, 16, 8, 128, 1700, 1152),
                                                          (160, 1, 8, 8, 64, 500, 0)])
def test_waits_that_give_up(sv, B, n, heads, kv, dim, longest, pre):
    """A barrier that nothing completes: the waits give up, the call ends with a report, and calls after it are as before it."""
    g = torch.Generator().manual_seed(n)
    ctx = [longest - 5 * (b % 40) for b in range(B)]
    c = Cache(B, BF, ctx, n, kv, dim, 16, groups=[(0, pre)] if pre else None)
    for b in range(B):
        c.put(b, ctx[b], torch.randn((n, kv, dim), generator=g), torch.randn((n, kv, dim), generator=g))
    q = torch.randn((B, n, heads, dim), generator=g).to(BF).cuda()

    def run():
        st = sv.new_stats("cuda")
        out, lse = sv.sv_kv_attend(q, c.k, c.v, lse=True, stats=st, **c.args, **c.group_args)
        return out, lse, sv.read_stats(st)["status"]
    out, lse, status = run()
    assert status == 0
    lib = sv.load()
    for limit in (2_000_000, 200_000):   # about 1 and 0.1 ms
        lib.sv_selftest_attend_stall(limit)
        try:
            assert run()[2] == 4   # timed out
        finally:
            lib.sv_selftest_attend_stall(0)
        for _ in range(3):
            again = run()
            assert again[2] == 0 and torch.equal(again[0], out) and torch.equal(again[1], lse)


def test_threads_with_other_vocabularies(sv):
    """The same for the top-N kernels, whose shared memory goes by the row length and the count."""
    cases = [(torch.randn(4, 128256, device="cuda"), 64), (torch.randn(4, 20000, device="cuda"), 8), (torch.randn(300, 50000, device="cuda"), 700),
             (torch.randn(2, 4000, device="cuda"), 3)]
    want = [sv.sv_topk_rows(x, n)[:2] for x, n in cases]
    torch.cuda.synchronize()
    got, errors = [[] for _ in cases], []

    def work(x, n, to):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(1500):
                    last = sv.sv_topk_rows(x, n)[:2]
                torch.cuda.current_stream().synchronize()
                to.append(last)
        except Exception as e:   # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=(x, n, to)) for (x, n), to in zip(cases, got)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    assert all(torch.equal(a, b) for w, to in zip(want, got) for x in to for a, b in zip(x, w))
