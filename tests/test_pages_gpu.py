"""GPU tests of a cache's pages: forks and compaction against the oracle, to the bit."""
import numpy as np
import pytest
import torch

from kv8_helpers import order_axes
from oracle import kv as okv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_gb300 as sv
    sv.load()
    return sv


class Pool:
    """Random bytes as a pool of pages, sequences that hold some (a few of them shared), and holders that are no sequence."""

    def __init__(self, seed, layers, page, kv, dim, dtype, B, longest, order="psh", extra=20, kept=3, together=False, shared=0):
        self.rng = rng = np.random.default_rng(seed)
        self.page, self.B = page, B
        self.ctx = rng.integers(0, longest + 1, B)
        took = [-(-int(c) // page) for c in self.ctx]
        self.width = max(took) + 3
        self.pages = P = sum(took) + extra + kept
        ids = [int(p) for p in rng.permutation(P)]
        self.table = np.full((B, self.width), -1, np.int64)
        self.refs = np.zeros(P, np.int64)
        for b in range(B):
            for e in range(took[b]):
                common = b > 0 and e < min(shared, int(self.ctx[b]) // page, int(self.ctx[0]) // page)   # full pages of sequence 0
                self.table[b, e] = self.table[0, e] if common else ids.pop()
                self.refs[self.table[b, e]] += 1
        for p in ids[:kept]:
            self.refs[p] += 2
        if longest > 0 and kept:   # somebody keeps a page of the last sequence too, its partly filled one where it has one
            if took[-1]:
                self.refs[self.table[-1, took[-1] - 1]] += 1
        es = {torch.float32: 4, torch.bfloat16: 2, torch.float8_e4m3fn: 1}[dtype]

        def raw():
            x = torch.tensor(rng.integers(0, 256, (layers, P, page, kv, dim * es)).astype(np.uint8))
            return x
        self.bytes = [raw(), raw()]
        if together:   # keys and values interleaved in one allocation
            both = torch.stack(self.bytes, 2).cuda()
            self.caches = [both[:, :, 0].view(dtype), both[:, :, 1].view(dtype)]
        else:
            self.caches = [torch.stack([order_axes(x, order) for x in c]).cuda() if order == "psh" else
                           self.lay_out(c, order) for c in self.bytes]
            self.caches = [c.view(dtype) for c in self.caches]
        self.scales = [torch.tensor(rng.integers(0, 255, (layers, P, kv)).astype(np.uint8)).cuda() for _ in range(2)] if es == 1 else None
        self.scales_were = [s.cpu().clone() for s in self.scales] if es == 1 else None

    @staticmethod
    def lay_out(c, order):
        axes = {"phs": (0, 1, 3, 2, 4), "hps": (3, 0, 1, 2, 4)}[order]
        return c.permute(axes).contiguous().cuda().permute(tuple(int(i) for i in np.argsort(axes)))

    @property
    def kw(self):
        return dict(k_scale=self.scales[0], v_scale=self.scales[1]) if self.scales else {}

    def dev(self, x):
        return torch.tensor(np.asarray(x).astype(np.int32)).cuda()

    def check_bytes(self, copies):
        """copies: (from, to, tokens), of the bytes as they were."""
        for c, was in zip(self.caches, self.bytes):
            want = was.clone()
            for a, b, t in copies:
                want[:, b, :t] = was[:, a, :t]
            assert torch.equal(c.view(torch.uint8).cpu(), want)
        for s, was in zip(self.scales or [], self.scales_were or []):
            want = was.clone()
            for a, b, _ in copies:
                want[:, b] = was[:, a]
            assert torch.equal(s.cpu(), want)

    def fork(self, sv, src, reserve, **kw):
        return sv.sv_kv_fork(*self.caches, self.dev(self.refs), self.dev(self.ctx), self.dev(self.table), self.dev(src), reserve=reserve, **self.kw, **kw)


E4M3, BF, F32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32
SHAPES = [dict(layers=1, page=16, kv=2, dim=64, dtype=BF, B=1, longest=40), dict(layers=3, page=4, kv=3, dim=48, dtype=E4M3, B=7, longest=30, order="phs"),
          dict(layers=2, page=1, kv=1, dim=16, dtype=F32, B=5, longest=9), dict(layers=2, page=24, kv=8, dim=128, dtype=E4M3, B=12, longest=200, shared=2),
          dict(layers=4, page=7, kv=2, dim=80, dtype=BF, B=40, longest=100, order="hps", shared=5),
          dict(layers=1, page=100, kv=9, dim=16, dtype=F32, B=3, longest=350, together=True), dict(layers=1, page=2, kv=1, dim=16, dtype=E4M3, B=300, longest=60)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("kind", ["same", "beams", "grow", "drop"])
@pytest.mark.parametrize("reserve", [0, 1, 13])
def test_fork_is_the_oracles(sv, shape, kind, reserve):
    B = shape["B"]
    N = 4 * B + 1 if kind == "grow" else B
    p = Pool(reserve + len(kind), **shape, extra=N * (-(-reserve // shape["page"]) + 2) + 10)
    src = {"same": np.arange(B), "beams": p.rng.integers(-1, B, B), "grow": p.rng.integers(0, B, N), "drop": np.full(1, -1)}[kind]
    p.width = max(p.width, -(-(int(p.ctx.max()) + reserve) // p.page))
    p.table = np.pad(p.table, ((0, 0), (0, p.width - p.table.shape[1])), constant_values=-1)
    stats = sv.new_stats("cuda")
    table, ctx, refs = p.fork(sv, src, reserve, stats=stats)
    assert sv.read_stats(stats)["status"] == 0
    rows, wctx, wrefs, copies = okv.fork(p.refs, p.ctx, p.table, src, reserve, p.page)
    assert ctx.tolist() == wctx and refs.tolist() == wrefs
    assert table.tolist() == rows
    p.check_bytes(copies)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("extra,kept", [(0, 0), (3, 1), (700, 5)])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact_is_the_oracles(sv, shape, extra, kept, in_place):
    p = Pool(extra, **dict(shape, extra=max(extra, 1 - kept), kept=kept))
    refs, table = p.dev(p.refs), p.dev(p.table)
    kw = dict(refs_out=refs, table_out=table) if in_place else {}
    moved = torch.empty(p.pages, dtype=torch.int32).cuda()
    stats = sv.new_stats("cuda")
    new, after, live = sv.sv_kv_compact(*p.caches, refs, table, moved_to=moved, stats=stats, **p.kw, **kw)
    assert sv.read_stats(stats)["status"] == 0
    to, wrefs, n = okv.compact(p.refs)
    assert live.tolist() == [n] and moved.tolist() == to and after.tolist() == wrefs
    assert new.tolist() == [[to[e] if e >= 0 else int(e) for e in row] for row in p.table]
    p.check_bytes([(a, b, p.page) for a, b in enumerate(to) if b >= 0 and a != b])
    if not in_place:
        assert refs.tolist() == p.refs.tolist() and table.tolist() == p.table.tolist()


def test_large_pools(sv):
    """More pages and entries than the plan has threads: 40,000 pages, 500 sequences."""
    p = Pool(1, 1, 1, 1, 16, E4M3, 500, 120, extra=9000, shared=3)
    src = p.rng.integers(-1, 500, 700)
    p.table = np.pad(p.table, ((0, 0), (0, 10)), constant_values=-1)
    table, ctx, refs = p.fork(sv, src, 5)
    rows, wctx, wrefs, copies = okv.fork(p.refs, p.ctx, p.table, src, 5, 1)
    assert table.tolist() == rows and ctx.tolist() == wctx and refs.tolist() == wrefs
    p.check_bytes(copies)
    q = Pool(2, 1, 1, 1, 16, E4M3, 500, 120, extra=9000)
    new, after, live = sv.sv_kv_compact(*q.caches, q.dev(q.refs), q.dev(q.table), **q.kw)
    to, wrefs, n = okv.compact(q.refs)
    assert live.tolist() == [n] and after.tolist() == wrefs
    assert new.tolist() == [[to[e] if e >= 0 else int(e) for e in row] for row in q.table]
    q.check_bytes([(a, b, 1) for a, b in enumerate(to) if b >= 0 and a != b])


def test_no_page_is_left(sv):
    """What there is goes to the first sequences; the others' entries are -1 and it is reported."""
    from speculative_decoding_verification_gb300 import _abi
    p = Pool(3, 2, 4, 2, 16, BF, 4, 30, extra=3, kept=0)
    src = np.array([0, 0, 1, 1, 2, 3, 3])
    stats = sv.new_stats("cuda")
    table, ctx, refs = p.fork(sv, src, 4, stats=stats)
    rows, wctx, wrefs, copies = okv.fork(p.refs, p.ctx, p.table, src, 4, 4)
    assert any(-1 in r[:-(-(c + 4) // 4)] for r, c in zip(rows, wctx))
    st = sv.read_stats(stats)
    assert st["status"] == _abi.SV_ERR_NO_PAGE and -1 in rows[st["error_index"]]
    assert table.tolist() == rows and refs.tolist() == wrefs
    p.check_bytes(copies)


def test_bad_device_arrays_are_reported(sv):
    """Sources, contexts, page ids and counts that do not fit: an error in stats, and nothing moved out of place."""
    from speculative_decoding_verification_gb300 import _abi
    p = Pool(4, 2, 4, 2, 16, E4M3, 4, 30, extra=40)
    cap = p.table.shape[1] * 4

    def status(src=(0, 1, 2, 3), **change):
        was = {k: getattr(p, k).copy() for k in change}
        for k, f in change.items():
            f(getattr(p, k))
        stats = sv.new_stats("cuda")
        got = p.fork(sv, src, 2, stats=stats)
        for k, x in was.items():
            setattr(p, k, x)
        st = sv.read_stats(stats)
        return st["status"], st["error_index"], got
    bad = _abi.SV_ERR_INVALID_ARG
    p.ctx[:] = [8, 9, 13, 4]
    p.table[:, :4] = np.arange(16).reshape(4, 4)
    p.table[:, 4:] = -1
    p.refs[:] = 0
    p.refs[:16] = 1
    assert status()[0] == 0
    code, at, (table, ctx, _) = status(src=(0, 4, -2, 1))
    assert code == bad and at in (1, 2) and ctx.tolist() == [8, 0, 0, 9] and (table[1] == -1).all()
    assert status(ctx=lambda x: x.__setitem__(2, -1))[:2] == (bad, 2)
    assert status(ctx=lambda x: x.__setitem__(3, cap - 1))[:2] == (bad, 3)
    assert status(table=lambda x: x.__setitem__((1, 0), p.pages))[:2] == (bad, 1)
    code, at, (table, _, _) = status(table=lambda x: x.__setitem__((1, 0), -7))
    assert (code, at) == (bad, 1) and table[1, 0] == -1
    assert status(refs=lambda x: x.__setitem__(3, 0))[:2] == (bad, 3)
    for refs, entry in ((-1, 3), (0, 3), (1, p.pages + 5)):
        refs_in, table_in = p.refs.copy(), p.table.copy()
        refs_in[3], table_in[0, 3] = refs, entry
        stats = sv.new_stats("cuda")
        new, after, live = sv.sv_kv_compact(*p.caches, p.dev(refs_in), p.dev(table_in), stats=stats, **p.kw)
        assert sv.read_stats(stats)["status"] == bad and live.tolist() == [15 if refs < 1 else 16]
        assert new[0, 3] == entry


def test_in_a_graph_beside_another_stream(sv):
    """Captured once, replayed on new arrays in place, beside calls on a second stream with a pool of their own."""
    p, q = (Pool(s, 2, 8, 2, 64, BF, 30, 90, extra=400) for s in (5, 6))
    src = p.rng.integers(-1, 30, 60)
    args = [p.dev(x) for x in (p.refs, p.ctx, p.table, src)]
    first = [c.clone() for c in p.caches]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = sv.sv_kv_fork(*p.caches, *args, reserve=3)
    want = okv.fork(p.refs, p.ctx, p.table, src, 3, 8)
    qsrc = q.rng.integers(-1, 30, 60)
    qwant = okv.fork(q.refs, q.ctx, q.table, qsrc, 3, 8)
    side = torch.cuda.Stream()
    qargs = [q.dev(x) for x in (q.refs, q.ctx, q.table, qsrc)]
    for _ in range(10):
        for c, f in zip(p.caches, first):
            c.copy_(f)
        torch.cuda.synchronize()
        graph.replay()
        got = sv.sv_kv_fork(*q.caches, *qargs, reserve=3, stream=side)
        torch.cuda.synchronize()
        for (table, ctx, refs), w in ((out, want), (got, qwant)):
            assert table.tolist() == w[0] and ctx.tolist() == w[1] and refs.tolist() == w[2]
        p.check_bytes(want[3])


def test_graphs_that_share_a_workspace(sv):
    """A captured fork and a captured compaction with one workspace, replayed in turn; results in arrays with a pitch and in the inputs' place."""
    p = Pool(8, 2, 8, 2, 64, E4M3, 20, 90, extra=300, shared=3)
    src = p.rng.integers(-1, 20, 50)
    rows, wctx, wrefs, copies = okv.fork(p.refs, p.ctx, p.table, src, 4, 8)
    to, wafter, n = okv.compact(wrefs)
    ws = sv.Workspace()
    inputs = [p.dev(x) for x in (p.refs, p.ctx, p.table, src)]
    refs = inputs[0].clone()
    wide = torch.full((50, p.width + 5), -9, dtype=torch.int32).cuda()
    first = [c.clone() for c in (*p.caches, *p.scales)]

    def fork():
        return sv.sv_kv_fork(*p.caches, refs, *inputs[1:], reserve=4, refs_out=refs, table_out=wide[:, :p.width], workspace=ws, **p.kw)

    def compact():
        return sv.sv_kv_compact(*p.caches, refs, wide[:, :p.width], refs_out=refs, table_out=wide[:, :p.width], workspace=ws, **p.kw)
    fork(), compact()
    graphs = []
    for f in (fork, compact):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            out = f()
    for _ in range(4):
        for c, f in zip((*p.caches, *p.scales, refs), (*first, inputs[0])):
            c.copy_(f)
        graphs[0].replay()
        middle = refs.clone(), wide.clone()
        graphs[1].replay()
        torch.cuda.synchronize()
        assert middle[0].tolist() == wrefs and middle[1][:, :p.width].tolist() == rows and bool((wide[:, p.width:] == -9).all())
        assert refs.tolist() == wafter and int(out[2]) == n
        assert wide[:, :p.width].tolist() == [[to[e] if e >= 0 else int(e) for e in row] for row in rows]
    # a sequence's bytes after both are those of the tokens it continues
    for j, b in enumerate(src):
        for e in range(-(-int(p.ctx[b]) // 8) if b >= 0 else 0):
            t = min(8, int(p.ctx[b]) - 8 * e)
            for c, was in zip(p.caches, p.bytes):
                assert torch.equal(c.view(torch.uint8)[:, wide[j, e].long(), :t].cpu(), was[:, p.table[b, e], :t])


def test_beams_as_they_are_used(sv):
    """Beams over a cache held in 8 bits: append, attend, reorder, now and then compact; each beam's attention is that of a cache of its own that
    was never shared."""
    rng = np.random.default_rng(7)
    B, H, kv, D, page, P = 6, 4, 2, 32, 4, 220
    k8, v8 = (torch.zeros((1, P, page, kv, D), dtype=torch.uint8).cuda().view(E4M3) for _ in range(2))
    ks, vs = (torch.zeros((1, P, kv), dtype=torch.uint8).cuda() for _ in range(2))
    ok8, ov8 = (torch.zeros((1, B * 16, page, kv, D), dtype=torch.uint8).cuda().view(E4M3) for _ in range(2))
    oks, ovs = (torch.zeros((1, B * 16, kv), dtype=torch.uint8).cuda() for _ in range(2))
    own = torch.arange(B * 16, dtype=torch.int32).view(B, 16).cuda()
    table = torch.full((B, 16), -1, dtype=torch.int32).cuda()
    refs, ctx = torch.zeros(P, dtype=torch.int32).cuda(), torch.zeros(B, dtype=torch.int32).cuda()
    stats = sv.new_stats("cuda")

    def ok():
        assert sv.read_stats(stats)["status"] == 0
    for step in range(14):
        n = int(rng.integers(1, 4))
        src = torch.tensor(rng.integers(0, B, B).astype(np.int32)).cuda()
        table, ctx, refs = sv.sv_kv_fork(k8, v8, refs, ctx, table, src, reserve=n, k_scale=ks, v_scale=vs, refs_out=refs, stats=stats)
        ok()
        for c in (ok8, ov8, oks, ovs):   # the other side copies everything
            c = c.view(torch.uint8)
            each = c[0].view(B, -1)
            each.copy_(each[src.long()].clone())
        if step % 4 == 3:
            table, refs, live = sv.sv_kv_compact(k8, v8, refs, table, k_scale=ks, v_scale=vs, refs_out=refs, table_out=table, stats=stats)
            ok()
            assert (table < live).all() and int((refs > 0).sum()) == int(live) and (refs[int(live):] == 0).all()
        q = torch.tensor(rng.normal(size=(B, n, H, D)), dtype=BF).cuda()
        k, v = (torch.tensor(rng.normal(size=(B, n, kv, D)) * 2.0 ** rng.integers(-3, 4), dtype=BF).cuda() for _ in range(2))
        sv.sv_kv_append8(k, v, k8[0], v8[0], ks[0], vs[0], ctx, table, stats=stats)
        ok()
        sv.sv_kv_append8(k, v, ok8[0], ov8[0], oks[0], ovs[0], ctx, own)
        out, _ = sv.sv_kv_attend8(q, k8[0], v8[0], ks[0], vs[0], ctx, table, stats=stats)
        ok()
        want, _ = sv.sv_kv_attend8(q, ok8[0], ov8[0], oks[0], ovs[0], ctx, own)
        assert torch.equal(out, want)
        ctx = ctx + n
    counts = torch.zeros(P, dtype=torch.int32)
    for p in table.cpu().flatten().tolist():
        if p >= 0:
            counts[p] += 1
    assert torch.equal(counts, refs.cpu())
