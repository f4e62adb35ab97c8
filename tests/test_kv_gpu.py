"""GPU tests of the target's side of a step: rotary positions, the cache append, attention over the paged cache and
the commit, against the float64 oracle.  Every slot that holds no token is NaN."""
import numpy as np
import pytest
import torch

from kv_helpers import U16, U32, Cache, check_attend, f64, random_tree
from oracle import kv as okv

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_gb300 as sv
    sv.load()
    return sv


def randn(seed, *shape, dtype=F32):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


# ---- rotary positions --------------------------------------------------------------------------------------------------------

def rope_tol(x, dtype, magnitude=1.0, last=0):
    """An angle is formed from f / 2pi to 2^-49 relative, in three products: within 2e-6 rad plus 1.5e-14 a position.  cos and sin
    are within 2 ulp, a product and a fused product-sum round: (angle + 5 u32) (|a| + |b|) M, then the output's rounding."""
    pair = magnitude * 2.0 * np.abs(x).max()
    return (2e-6 + 1.5e-14 * abs(last) + 5 * U32) * pair + (U16 * pair if dtype == BF else 0.0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("style", ["half", "interleaved"])
@pytest.mark.parametrize("rows,heads,dim,rotary,first", [(1, 1, 2, 2, 0), (3, 5, 64, 64, 7), (17, 3, 80, 80, 100), (5, 2, 128, 64, 131072),
                                                         (4, 7, 96, 34, 1 << 20), (9, 1, 7, 6, 5), (2, 32, 256, 256, 2**31 - 3),
                                                         (6, 2, 128, 128, -4)])
def test_rope(sv, dtype, style, rows, heads, dim, rotary, first):
    x = randn(rows + dim, rows, heads, dim, dtype=dtype)
    f, _ = sv.sv_rope_frequencies(rotary)
    inv = torch.tensor(f).cuda()
    pos = (torch.arange(rows, dtype=torch.int64) + first).to(torch.int32)
    for backward in (False, True):
        got = sv.sv_rope(x, pos.cuda(), inv, style=style, magnitude=1.25, backward=backward)
        want = okv.rope(f64(x), pos.numpy(), f64(inv), style, 1.25, backward)
        assert np.abs(f64(got) - want).max() <= rope_tol(f64(x), dtype, 1.25, first)
        assert torch.equal(got[..., rotary:], x[..., rotary:])
    y = x.clone()
    sv.sv_rope(y, pos.cuda(), inv, style=style, out=y)   # in place
    assert torch.equal(y, sv.sv_rope(x, pos.cuda(), inv, style=style))


@pytest.mark.parametrize("style", ["half", "interleaved"])
def test_rope_gradient(sv, style):
    """backward is the transpose: against differences of the forward along random directions (float32 differences of a linear
    map are exact up to rounding: |dy| 8 u32 over the step)."""
    x, g = randn(1, 6, 3, 64), randn(2, 6, 3, 64)
    pos = torch.tensor([0, 1, 5, 1000, 65536, 3], dtype=torch.int32).cuda()
    inv = torch.tensor(sv.sv_rope_frequencies(48)[0]).cuda()
    gx = sv.sv_rope(g, pos, inv, style=style, magnitude=0.7, backward=True)
    for seed in range(3):
        d = randn(10 + seed, 6, 3, 64)
        up, down = (sv.sv_rope(x + e * d, pos, inv, style=style, magnitude=0.7) for e in (0.5, -0.5))
        slope = float(((up.double() - down.double()) * g.double()).sum())
        terms = float((d.double().abs() * g.double().abs()).sum()) * 2
        assert abs(slope - float((gx.double() * d.double()).sum())) <= 1e-5 * terms


def test_rope_strides_streams_and_empty(sv):
    inv = torch.tensor(sv.sv_rope_frequencies(32)[0]).cuda()
    pos = torch.arange(8, dtype=torch.int32).cuda()
    big = randn(3, 8, 6, 3, 40)
    for view in (big[:, :, 1], big[:, ::2, 2], big[:, :, 0, 3:37], big.permute(0, 2, 1, 3)[:, 1]):
        assert torch.equal(sv.sv_rope(view, pos, inv), sv.sv_rope(view.contiguous(), pos, inv))
    s = torch.cuda.Stream()
    x = big[:, :, 0].contiguous()
    want = sv.sv_rope(x, pos, inv)
    s.wait_stream(torch.cuda.current_stream())
    got = sv.sv_rope(x, pos, inv, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    assert sv.sv_rope(x[:0], pos[:0].contiguous() if pos[:0].numel() else pos, inv).shape == (0, 6, 40)


# ---- append --------------------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,n,heads,kv,dim,page,rotary,style,tree,order", [
    (1, 1, 4, 4, 64, 16, 64, "half", False, "psh"), (3, 5, 8, 2, 128, 16, 128, "half", True, "psh"),
    (2, 7, 6, 3, 80, 5, 40, "interleaved", True, "phs"), (4, 3, 5, 1, 96, 1, 0, "half", False, "hps"),
    (2, 129, 2, 1, 64, 24, 34, "half", True, "psh"), (2, 6, 4, 2, 256, 8, 256, "interleaved", False, "psh")])
def test_append(sv, dtype, B, n, heads, kv, dim, page, rotary, style, tree, order):
    ctx = [0, 13, 40, 31][:B]
    c = Cache(5, dtype, ctx, n, kv, dim, page, order, together=order == "psh" and not tree)
    qkv = randn(6, B, n, heads + 2 * kv, dim, dtype=dtype)
    q, k, v = qkv.split([heads, kv, kv], 2)
    par = random_tree(c.rng, B, n) if tree else None
    inv = torch.tensor(sv.sv_rope_frequencies(rotary)[0]).cuda() if rotary else None
    before_k, before_v = c.k.clone(), c.v.clone()
    st = sv.new_stats("cuda")
    qo = sv.sv_kv_append(k, v, c.k, c.v, q=q, inv_freq=inv, style=style, magnitude=1.1, parents=par.cuda() if tree else None,
                         stats=st, **c.args)
    assert sv.read_stats(st)["status"] == 0
    k64, v64 = f64(before_k), f64(before_v)
    for b in range(B):
        want = okv.append(k64, v64, f64(k[b]), f64(v[b]), ctx[b], c.table[b].numpy(), par[b].tolist() if tree else None,
                          f64(inv) if rotary else None, style, 1.1, f64(q[b]))
        tol = rope_tol(f64(qkv), dtype, 1.1) if rotary else 0.0
        assert np.abs(f64(qo[b]) - (want if rotary else f64(q[b]))).max() <= tol
    got = f64(c.k)
    assert np.array_equal(np.isnan(got), np.isnan(k64)) and np.nanmax(np.abs(got - k64)) <= tol
    assert np.array_equal(f64(c.v), v64, equal_nan=True)
    # without queries the cache comes out the same, bit for bit
    k2, v2 = before_k.clone(), before_v.clone()
    assert sv.sv_kv_append(k, v, k2, v2, inv_freq=inv, style=style, magnitude=1.1, parents=par.cuda() if tree else None, **c.args) is None
    bits = torch.int16 if dtype == BF else torch.int32
    assert torch.equal(k2.view(bits), c.k.view(bits)) and torch.equal(v2.view(bits), c.v.view(bits))


def test_append_ragged_and_reports(sv):
    """Ragged blocks, one of them empty; then a context that does not fit and a bad page: reported, nothing written."""
    rs = [0, 3, 3, 8]
    c = Cache(7, F32, [4, 9, 0], 5, 2, 64, 4)
    k, v, q = randn(1, 8, 2, 64), randn(2, 8, 2, 64), randn(3, 8, 4, 64)
    inv = torch.tensor(sv.sv_rope_frequencies(64)[0]).cuda()
    k64, v64 = f64(c.k), f64(c.v)
    st = sv.new_stats("cuda")
    qo = sv.sv_kv_append(k, v, c.k, c.v, q=q, inv_freq=inv, row_start=torch.tensor(rs, dtype=torch.int32).cuda(), max_rows=5,
                         stats=st, **c.args)
    assert sv.read_stats(st)["status"] == 0
    for b in range(3):
        r = slice(rs[b], rs[b + 1])
        if r.stop > r.start:
            want = okv.append(k64, v64, f64(k[r]), f64(v[r]), c.contexts[b], c.table[b].numpy(), None, f64(inv), q=f64(q[r]))
            assert np.abs(f64(qo[r]) - want).max() <= rope_tol(f64(q), F32)
    assert np.nanmax(np.abs(f64(c.k) - k64)) <= rope_tol(f64(k), F32) and np.array_equal(f64(c.v), v64, equal_nan=True)
    k4, v4 = k[:6].view(3, 2, 2, 64), v[:6].view(3, 2, 2, 64)
    for context, table in (([4, 10000, 0], c.table), ([-1, 9, 0], c.table), ([4, 9, 0], torch.where(c.table >= 0, 10**6, 0).int())):
        kc, vc = c.k.clone(), c.v.clone()
        st = sv.new_stats("cuda")
        sv.sv_kv_append(k4, v4, kc, vc, torch.tensor(context, dtype=torch.int32).cuda(), table.cuda(), stats=st)
        assert sv.read_stats(st)["status"] == 1


# ---- attention -----------------------------------------------------------------------------------------------------------------

def blocks(c, seed, B, n, heads, kv, dim, dtype):
    """Queries, and the block's keys and values put in the cache's slots after the context."""
    q = randn(seed, B, n, heads, dim, dtype=dtype) * 2
    for b in range(B):
        c.put(b, c.contexts[b], randn(seed + 1 + b, n, kv, dim), randn(seed + 101 + b, n, kv, dim))
    return q


ATTEND = [
    # contexts, n, heads, kv_heads, dim, page, tree
    ([0], 1, 1, 1, 64, 16, False),                       # one token that sees itself
    ([1], 1, 8, 1, 128, 16, False),
    ([1000], 5, 32, 8, 128, 16, False),                  # split over many blocks
    ([0, 127, 128, 129, 300], 1, 8, 2, 128, 16, False),  # single tokens, tiles that end exactly
    ([63, 64, 65, 500, 2], 6, 12, 4, 64, 7, False),      # odd pages
    ([17, 200], 33, 6, 2, 96, 24, False),
    ([100, 3], 9, 5, 1, 80, 1, True),                    # pages of one slot
    ([50, 700, 0], 57, 8, 2, 64, 16, True),
    ([200, 31], 129, 4, 2, 128, 32, True),               # the largest tree
    ([260], 129, 16, 1, 128, 100, True),                 # many packed rows a key head
    ([5, 90], 40, 2, 2, 8, 3, False),                    # narrow heads
    ([30, 150], 3, 4, 2, 256, 16, True),                 # wide heads
    ([400, 10], 70, 14, 7, 192, 16, False),
    ([600], 300, 4, 1, 64, 16, False),                   # a chunk of a prompt
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("ctx,n,heads,kv,dim,page,tree", ATTEND)
def test_attend(sv, dtype, ctx, n, heads, kv, dim, page, tree):
    B = len(ctx)
    c = Cache(n + dim, dtype, ctx, n, kv, dim, page)
    q = blocks(c, 40, B, n, heads, kv, dim, dtype)
    par = random_tree(c.rng, B, n) if tree else None
    st = sv.new_stats("cuda")
    out, lse = sv.sv_kv_attend(q, c.k, c.v, parents=par.cuda() if tree else None, lse=True, stats=st, **c.args)
    assert sv.read_stats(st)["status"] == 0
    rows = [slice(b * n, b * n + n) for b in range(B)]
    check_attend(c, q.flatten(0, 1), out.flatten(0, 1), lse.flatten(0, 1), dim ** -0.5, rows, par)
    again, _ = sv.sv_kv_attend(q, c.k, c.v, parents=par.cuda() if tree else None, **c.args)
    assert torch.equal(out, again)   # the order of partial sums is fixed


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("ctx,groups,n,heads,kv,dim,page,tree", [
    ([40, 33, 64], [(0, 32)], 3, 8, 2, 64, 16, False),
    ([1100, 1024, 1300, 1029], [(0, 1024)], 8, 8, 2, 128, 16, False),
    ([300, 290, 513, 520, 514, 7], [(0, 288), (2, 512), (5, 0)], 6, 4, 1, 96, 16, False),   # ragged groups, one without a prefix
    ([45, 45, 50], [(0, 45)], 2, 6, 3, 80, 16, False),                                      # a prefix that ends inside a page
    ([200] * 9, [(0, 192)], 33, 8, 1, 128, 64, True),                                       # tall prefix tiles
    ([700, 650, 810], [(0, 640), (1, 640)], 5, 12, 4, 128, 32, True),                       # groups of one and two
])
def test_attend_shared_prefix(sv, dtype, ctx, groups, n, heads, kv, dim, page, tree):
    B = len(ctx)
    c = Cache(9 + dim, dtype, ctx, n, kv, dim, page, groups=groups)
    q = blocks(c, 41, B, n, heads, kv, dim, dtype)
    par = random_tree(c.rng, B, n) if tree else None
    st = sv.new_stats("cuda")
    out, lse = sv.sv_kv_attend(q, c.k, c.v, parents=par.cuda() if tree else None, lse=True, stats=st, scale=0.11, **c.args, **c.group_args)
    assert sv.read_stats(st)["status"] == 0
    rows = [slice(b * n, b * n + n) for b in range(B)]
    check_attend(c, q.flatten(0, 1), out.flatten(0, 1), lse.flatten(0, 1), 0.11, rows, par)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("grouped", [False, True])
def test_attend_ragged(sv, dtype, grouped):
    """Blocks of different lengths, empty ones among them."""
    lens, ctx = [3, 0, 7, 1, 0], [70, 64, 64, 90, 66]
    rs = np.concatenate([[0], np.cumsum(lens)])
    c = Cache(3, dtype, ctx, 7, 2, 64, 16, groups=[(0, 64)] if grouped else None)
    q = randn(8, int(rs[-1]), 8, 64, dtype=dtype) * 2
    for b in range(5):
        c.put(b, ctx[b], randn(50 + b, lens[b], 2, 64), randn(60 + b, lens[b], 2, 64))
    out, lse = sv.sv_kv_attend(q, c.k, c.v, row_start=torch.tensor(rs, dtype=torch.int32).cuda(), max_rows=7, lse=True, **c.args,
                               **c.group_args)
    check_attend(c, q, out, lse, 0.125, [slice(int(rs[b]), int(rs[b + 1])) for b in range(5)])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("order,together", [("phs", False), ("hps", False), ("psh", True)])
def test_attend_layouts_and_streams(sv, dtype, order, together):
    ctx, n = [130, 5, 257], 4
    c = Cache(4, dtype, ctx, n, 2, 128, 16, order, together=together)
    wide = randn(9, 3, n, 11, 128, dtype=dtype)
    q = wide[:, :, 2:10]
    for b in range(3):
        c.put(b, ctx[b], randn(70 + b, n, 2, 128), randn(80 + b, n, 2, 128))
    room = torch.zeros(3, n, 9, 128, dtype=dtype, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = sv.sv_kv_attend(q, c.k, c.v, out=room[:, :, :8], lse=True, stream=s, workspace=sv.Workspace(), **c.args)
    s.synchronize()
    assert float(room[:, :, 8].abs().max()) == 0.0
    rows = [slice(b * n, b * n + n) for b in range(3)]
    check_attend(c, q.flatten(0, 1), out.flatten(0, 1), lse.flatten(0, 1), 128 ** -0.5, rows)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_attend_hidden_tokens_stay_hidden(sv, dtype, dim, bad):
    """Draft rows whose keys and values are not finite reach only the rows that see them: siblings in a tree, and earlier rows
    of a chain, are those of a finite block bit for bit within the oracle's bound."""
    n, ctx = 9, [37, 140]
    c = Cache(11, dtype, ctx, n, 2, dim, 16)
    q = blocks(c, 42, 2, n, 4, 2, dim, dtype)
    par = torch.tensor([[0, 0, 1, 2, 2, 1, 4, 3]] * 2, dtype=torch.int32)   # rows 2, 4, 5, 7 follow row 2; 4's child is 7
    marked = 4
    for b in range(2):
        keys, vals = randn(7, 1, 2, dim), randn(8, 1, 2, dim)
        keys[..., ::3] = bad
        vals[..., ::5] = bad
        c.put(b, ctx[b] + marked, keys, vals)
    out, lse = sv.sv_kv_attend(q, c.k, c.v, parents=par.cuda(), lse=True, **c.args)
    sees = okv.ancestors(par[0].tolist(), n)[:, marked]
    clean = Cache(11, dtype, ctx, n, 2, dim, 16)
    blocks(clean, 42, 2, n, 4, 2, dim, dtype)
    for b in range(2):
        for i in range(n):
            if sees[i]:
                assert not bool(torch.isfinite(out[b, i]).all())
            else:
                assert bool(torch.isfinite(out[b, i]).all()) and bool(torch.isfinite(lse[b, i]).all())
    ref, _ = sv.sv_kv_attend(q, clean.k, clean.v, parents=par.cuda(), **clean.args)
    hidden = [i for i in range(n) if not sees[i]]
    assert torch.equal(out[:, hidden], ref[:, hidden])
    # a chain: rows before the marked one
    out, _ = sv.sv_kv_attend(q, c.k, c.v, **c.args)
    ref, _ = sv.sv_kv_attend(q, clean.k, clean.v, **clean.args)
    assert torch.equal(out[:, :marked], ref[:, :marked])


def test_attend_values_only_not_finite(sv):
    """Only the value of a hidden token is not finite; a row that sees it gets that value."""
    for dtype, dim in ((BF, 128), (F32, 64)):
        c = Cache(12, dtype, [20], 3, 1, dim, 16)
        q = blocks(c, 43, 1, 3, 2, 1, dim, dtype)
        v = randn(9, 1, 1, dim)
        v[..., 5] = float("inf")
        c.put(0, 22, randn(10, 1, 1, dim), v)
        out, _ = sv.sv_kv_attend(q, c.k, c.v, **c.args)
        assert bool(torch.isfinite(out[0, :2]).all())
        assert bool((out[0, 2, :, 5] == float("inf")).all())
        assert bool(torch.isfinite(out[0, 2, :, :5]).all()) and bool(torch.isfinite(out[0, 2, :, 6:]).all())


def test_attend_large_and_small_scores(sv):
    """Scores that overflow exp without the running maximum, and one that leaves a single token all the weight."""
    for dtype in (BF, F32):
        c = Cache(13, dtype, [300, 1], 2, 2, 64, 16)
        q = blocks(c, 44, 2, 2, 4, 2, 64, dtype) * 40
        out, lse = sv.sv_kv_attend(q, c.k, c.v, lse=True, scale=1.0, **c.args)
        check_attend(c, q.flatten(0, 1), out.flatten(0, 1), lse.flatten(0, 1), 1.0, [slice(0, 2), slice(2, 4)])
        out, lse = sv.sv_kv_attend(q, c.k, c.v, lse=True, scale=0.0, **c.args)   # all weights equal
        check_attend(c, q.flatten(0, 1), out.flatten(0, 1), lse.flatten(0, 1), 0.0, [slice(0, 2), slice(2, 4)])


def test_attend_past_32_bit_offsets(sv):
    """Pages whose element offsets pass 2^32 (a pool of 4.4e9 elements each for keys and values)."""
    page, kv, dim = 256, 8, 128
    P = (1 << 32) // (page * kv * dim) + 40
    k = torch.empty((P, page, kv, dim), dtype=BF, device="cuda")
    v = torch.empty((P, page, kv, dim), dtype=BF, device="cuda")
    ids = [P - 1, 3, P - 2]
    small_k, small_v = randn(1, 3, page, kv, dim, dtype=BF), randn(2, 3, page, kv, dim, dtype=BF)
    k[ids], v[ids] = small_k, small_v
    q = randn(3, 1, 2, 16, dim, dtype=BF)
    ctx = torch.tensor([700], dtype=torch.int32).cuda()
    far, _ = sv.sv_kv_attend(q, k, v, ctx, torch.tensor([ids], dtype=torch.int32).cuda())
    near, _ = sv.sv_kv_attend(q, small_k, small_v, ctx, torch.tensor([[0, 1, 2]], dtype=torch.int32).cuda())
    assert torch.equal(far, near)
    new = randn(4, 1, 2, kv, dim, dtype=BF)
    sv.sv_kv_append(new, new, k, v, ctx, torch.tensor([ids], dtype=torch.int32).cuda())
    assert torch.equal(k[P - 2, 700 - 512:702 - 512], new[0]) and torch.equal(v[P - 2, 700 - 512:702 - 512], new[0])


def test_attend_reports_bad_input(sv):
    """Bad contexts, page ids, prefixes, groups, row starts and parents are reported, and other sequences are not touched."""
    c = Cache(14, BF, [40, 50], 4, 2, 64, 16)
    q = blocks(c, 45, 2, 4, 4, 2, 64, BF)
    par = random_tree(c.rng, 2, 4)
    good, _ = sv.sv_kv_attend(q, c.k, c.v, **c.args)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32).cuda()
    table = c.table.clone()
    table[1, 1] = 10**6
    bad_par = par.clone()
    bad_par[1, 1] = 3
    cases = [dict(context_len=i32(40, 100000)), dict(context_len=i32(40, -3)), dict(page_table=table.cuda()),
             dict(group_start=i32(0, 2), prefix_len=i32(48)), dict(group_start=i32(0, 5), prefix_len=i32(8)),
             dict(group_start=i32(0, 2), prefix_len=i32(-1)), dict(parents=bad_par.cuda())]
    for kw in cases:
        st = sv.new_stats("cuda")
        args = dict(c.args, **kw)
        out, _ = sv.sv_kv_attend(q, c.k, c.v, stats=st, **args)
        assert sv.read_stats(st)["status"] == 1, kw
        if set(kw) <= {"context_len", "page_table"}:
            assert torch.equal(out[0], good[0])
    st = sv.new_stats("cuda")
    sv.sv_kv_attend(q.flatten(0, 1), c.k, c.v, row_start=i32(0, 6, 2), max_rows=4, stats=st, **c.args)
    assert sv.read_stats(st)["status"] == 1


# ---- commit --------------------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layers,N,kv,dim,page", [(1, 1, 1, 64, 16), (3, 8, 2, 80, 5), (2, 128, 8, 128, 16), (5, 30, 3, 256, 1)])
def test_commit(sv, dtype, layers, N, kv, dim, page):
    rng = np.random.default_rng(N)
    ctx = [0, 7, 33, 12]
    c = Cache(15, dtype, ctx, N + 1, kv, dim, page)
    k = torch.randn((layers,) + tuple(c.k.shape), device="cuda").to(dtype)
    v = torch.randn((layers,) + tuple(c.k.shape), device="cuda").to(dtype)
    acc = [0, 1, min(N, 5), N if N < 9 else N // 2]
    path = np.full((4, N), -1, np.int32)
    for b in range(4):
        path[b, : acc[b]] = np.sort(rng.choice(np.arange(1, N + 1), acc[b], replace=False))
    k64, v64 = f64(k), f64(v)
    want = [okv.commit(k64, v64, ctx[b], c.table[b].numpy(), acc[b], path[b]) for b in range(4)]
    st = sv.new_stats("cuda")
    got = sv.sv_kv_commit(k, v, c.args["context_len"], c.args["page_table"], torch.tensor(acc, dtype=torch.int32).cuda(),
                          torch.tensor(path).cuda(), stats=st)
    assert sv.read_stats(st)["status"] == 0
    assert got.tolist() == want
    assert np.array_equal(f64(k), k64) and np.array_equal(f64(v), v64)


def test_commit_reports_bad_paths(sv):
    c = Cache(16, BF, [5, 6, 7, 8], 4, 2, 64, 4)
    k, v = torch.randn((2,) + tuple(c.k.shape), device="cuda").to(BF), torch.randn((2,) + tuple(c.k.shape), device="cuda").to(BF)
    k0, v0 = k.clone(), v.clone()
    for acc, path in (([9, 0, 0, 0], [1, 2, 3]), ([-1, 0, 0, 0], [1, 2, 3]), ([2, 0, 0, 0], [2, 1, 3]), ([2, 0, 0, 0], [3, 4, 5]),
                      ([1, 0, 0, 0], [0, 1, 2])):
        st = sv.new_stats("cuda")
        out = sv.sv_kv_commit(k, v, c.args["context_len"], c.args["page_table"], torch.tensor(acc, dtype=torch.int32).cuda(),
                              torch.tensor([path] * 4, dtype=torch.int32).cuda(), stats=st)
        assert sv.read_stats(st)["status"] == 1 and sv.read_stats(st)["error_index"] == 0
        assert out.tolist() == [5, 7, 8, 9]
        assert torch.equal(k, k0) and torch.equal(v, v0)


# ---- many pieces a block --------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,n,heads,kv,dim,page,tree,pre,longest", [
    (40, 3, 16, 8, 128, 16, False, 0, 700),     # more tiles than blocks: ranges that start and end inside units
    (24, 20, 16, 4, 128, 32, True, 0, 900),     # short tiles of rows
    (12, 40, 16, 4, 64, 64, True, 0, 1500),     # two row tiles that share keys
    (30, 6, 8, 8, 128, 8, False, 0, 40),        # units of one key tile
    (48, 6, 16, 4, 128, 16, False, 1280, 300),  # prefixes of three groups, tall tiles, then own tokens
    (36, 9, 16, 8, 64, 96, True, 2016, 130),    # a prefix that is no whole number of tiles
    (20, 5, 8, 4, 96, 24, False, 1200, 260),    # pages that no box fits
])
def test_attend_many_pieces(sv, dtype, B, n, heads, kv, dim, page, tree, pre, longest):
    """Thousands of key tiles, so that every block walks several pieces of several units; a sample of the sequences is checked."""
    rng = np.random.default_rng(B)
    ctx = [pre + int(x) for x in rng.integers(0, longest + 1, B)]
    groups = [(0, pre), (B // 3, pre), (2 * B // 3 + 1, pre)] if pre else None
    c = Cache(B + dim, dtype, ctx, n, kv, dim, page, groups=groups)
    q = blocks(c, 46, B, n, heads, kv, dim, dtype)
    par = random_tree(c.rng, B, n) if tree else None
    st = sv.new_stats("cuda")
    out, lse = sv.sv_kv_attend(q, c.k, c.v, parents=par.cuda() if tree else None, lse=True, stats=st, **c.args, **c.group_args)
    assert sv.read_stats(st)["status"] == 0
    rows = [slice(b * n, b * n + n) for b in range(B)]
    seqs = sorted({0, 1, B // 3, B // 2, 2 * B // 3, B - 2, B - 1})
    check_attend(c, q.flatten(0, 1), out.flatten(0, 1), lse.flatten(0, 1), dim ** -0.5, rows, par, seqs)
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    again, _ = sv.sv_kv_attend(q, c.k, c.v, parents=par.cuda() if tree else None, **c.args, **c.group_args)
    assert torch.equal(out, again)


@pytest.mark.parametrize("B,n,heads,kv,dim,page,tree,pre,longest", [
    (24, 6, 16, 4, 128, 100, False, 0, 900),    # groups of 8 tokens, one in 25 of them over two pages
    (16, 4, 8, 4, 64, 9, False, 0, 700),        # nearly all of them
    (12, 30, 8, 2, 96, 20, True, 0, 800),       # tall tiles
    (20, 5, 8, 4, 80, 12, False, 1100, 260),    # prefixes that end inside a page and a group
    (16, 3, 8, 4, 128, 40, False, 0, 600),      # whole groups, no power of two
    (16, 3, 8, 4, 128, 7, False, 0, 600),       # pages smaller than a group
])
def test_attend_odd_pages(sv, B, n, heads, kv, dim, page, tree, pre, longest):
    """Page sizes that groups of 8 tokens do not divide into, over whole tiles; a bad page behind a good one is reported and the other
    sequences stay."""
    rng = np.random.default_rng(page)
    ctx = [pre + int(x) for x in rng.integers(longest // 2, longest + 1, B)]
    groups = [(0, pre), (B // 2, pre)] if pre else None
    c = Cache(B + page, BF, ctx, n, kv, dim, page, groups=groups)
    q = blocks(c, 47, B, n, heads, kv, dim, BF)
    par = random_tree(c.rng, B, n) if tree else None
    kw = dict(parents=par.cuda() if tree else None, **c.group_args)
    st = sv.new_stats("cuda")
    out, lse = sv.sv_kv_attend(q, c.k, c.v, lse=True, stats=st, **kw, **c.args)
    assert sv.read_stats(st)["status"] == 0
    rows = [slice(b * n, b * n + n) for b in range(B)]
    check_attend(c, q.flatten(0, 1), out.flatten(0, 1), lse.flatten(0, 1), dim ** -0.5, rows, par, [0, 1, B // 2, B - 1])
    table = c.table.clone()
    last = B - 1
    table[last, (ctx[last] - 1) // page] = c.k.shape[0]
    st = sv.new_stats("cuda")
    bad, _ = sv.sv_kv_attend(q, c.k, c.v, stats=st, **kw, **dict(c.args, page_table=table.cuda()))
    assert sv.read_stats(st)["status"] == 1
    assert torch.equal(bad[:last], out[:last])


@pytest.mark.parametrize("dtype,B,n,heads,kv,dim,page,tree,pre,longest", [
    (F32, 40, 2, 8, 4, 80, 16, False, 700, 500),     # 4 packed rows
    (F32, 30, 4, 6, 2, 128, 24, True, 333, 300),     # 12, a prefix that ends inside a page
    (F32, 24, 1, 8, 1, 64, 8, False, 1000, 20),      # 8 of one token
    (F32, 12, 3, 8, 2, 200, 16, False, 150, 400),    # wide heads
    (BF, 16, 4, 8, 2, 192, 32, False, 500, 300),
])
def test_attend_few_rows_beside_prefixes(sv, dtype, B, n, heads, kv, dim, page, tree, pre, longest):
    """Own tokens of few packed rows in a launch behind the prefixes', in every arithmetic."""
    rng = np.random.default_rng(dim)
    ctx = [pre + int(x) for x in rng.integers(0, longest + 1, B)]
    c = Cache(B + n, dtype, ctx, n, kv, dim, page, groups=[(0, pre), (B // 3, pre), (B // 2, pre)])
    q = blocks(c, 48, B, n, heads, kv, dim, dtype)
    par = random_tree(c.rng, B, n) if tree else None
    kw = dict(parents=par.cuda() if tree else None, **c.args, **c.group_args)
    st = sv.new_stats("cuda")
    out, lse = sv.sv_kv_attend(q, c.k, c.v, lse=True, stats=st, **kw)
    assert sv.read_stats(st)["status"] == 0
    rows = [slice(b * n, b * n + n) for b in range(B)]
    check_attend(c, q.flatten(0, 1), out.flatten(0, 1), lse.flatten(0, 1), dim ** -0.5, rows, par, [0, 1, B // 3, B // 2, B - 1])
    assert torch.equal(out, sv.sv_kv_attend(q, c.k, c.v, **kw)[0])
