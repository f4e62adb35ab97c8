"""GPU parity of the cache held in 8 bits: append, attention and commit against the float64 oracle and against the same calls over the values
that the codes stand for."""
from types import SimpleNamespace

import numpy as np
import pytest
import torch

from kv8_helpers import E4M3, Cache8, check_attend8, order_axes, values
from kv_helpers import f64, random_tree
from oracle import kv as okv

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_gb300 as sv
    sv.load()
    return sv


def exps(scale):
    return scale.view(torch.uint8).cpu().numpy().astype(np.int64) - 127


def same_codes(got, want64):
    """Codes against the oracle's numbers, NaN for NaN."""
    g = got.cpu().float().double().numpy()
    np.testing.assert_array_equal(g, want64)


def random_codes(rng, shape, most=0x77):
    """Finite codes up to 2^(most >> 3) or so, both signs."""
    c = rng.integers(0, most + 1, shape) | rng.integers(0, 2, shape) << 7
    return torch.tensor(c.astype(np.uint8))


class AppendCase:
    def __init__(self, seed, dtype, contexts, n, H, kv, dim, page, order="psh", scale_dtype=torch.uint8, low=100, high=130, size=1.0):
        self.rng = np.random.default_rng(seed)
        rng, B = self.rng, len(contexts)
        each = max((c + n + page - 1) // page for c in contexts) + 1
        P = B * each + 2
        self.table = torch.tensor(rng.permutation(P)[:B * each].reshape(B, each).astype(np.int32))
        self.contexts, self.page = contexts, page
        self.caches, self.scales, self.before = [], [], []
        for _ in range(2):
            c, s = random_codes(rng, (P, page, kv, dim)), torch.tensor(rng.integers(low, high, (P, kv)).astype(np.uint8))
            self.before.append((c.view(E4M3).double().numpy().copy(), s.numpy().astype(np.int64) - 127))
            self.caches.append(order_axes(c, order).cuda().view(E4M3))
            self.scales.append(s.cuda().view(scale_dtype))
        self.q = torch.tensor(rng.normal(size=(B, n, H, dim)), dtype=dtype)
        self.k, self.v = (torch.tensor(size * rng.normal(size=(B, n, kv, dim)) * 2.0 ** rng.integers(-9, 4, (B, n, kv, 1)), dtype=dtype)
                          for _ in range(2))

    def run(self, sv, **kw):
        return sv.sv_kv_append8(self.k.cuda(), self.v.cuda(), *self.caches, *self.scales,
                                torch.tensor(self.contexts, dtype=torch.int32).cuda(), self.table.cuda(), **kw)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,page,kv,dim,order", [(1, 16, 2, 64, "psh"), (5, 16, 8, 128, "phs"), (40, 8, 3, 80, "hps"), (33, 100, 17, 16, "psh"),
                                                 (3, 1, 1, 256, "psh"), (19, 3, 9, 48, "phs")])
def test_append_is_the_oracles_to_the_bit(sv, dtype, n, page, kv, dim, order):
    """Without rotation nothing is rounded but to the codes: codes and scales are the oracle's, those of slots past the block and of other
    pages as they were."""
    c = AppendCase(n + page, dtype, [0, 7, 16, 100, 3 * page - 1], n, kv, kv, dim, page, order, torch.float8_e8m0fnu if n == 5 else torch.uint8)
    assert c.run(sv) is None
    for x, cache, scale, (codes, e) in zip((c.k, c.v), c.caches, c.scales, c.before):
        for b, ctx in enumerate(c.contexts):
            okv.append8(codes, e, f64(x[b]), ctx, c.table[b].numpy())
        np.testing.assert_array_equal(exps(scale), e)
        same_codes(cache, codes)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("style,rotary,tree,n,page", [("half", 64, False, 6, 16), ("interleaved", 32, True, 12, 8), ("half", 26, False, 21, 24),
                                                      ("interleaved", 26, True, 9, 16), ("half", 0, True, 5, 16)])
def test_append_rotates(sv, dtype, style, rotary, tree, n, page):
    """Keys: off by the rotation in float32 (two products and a sum of elements up to m, an angle good to 4e-6: 5e-6 m in all) and half a step
    of their code.  Queries: rounded once."""
    c = AppendCase(n, dtype, [0, 30, 1001], n, 6, 2, 64, page)
    par = random_tree(c.rng, 3, n) if tree else None
    freq, mag = okv.rope_frequencies(rotary)[0] if rotary else None, 1.25 if rotary else 1.0
    kw = dict(inv_freq=torch.tensor(freq, dtype=F32).cuda(), style=style, magnitude=mag) if rotary else {}
    got = c.run(sv, q=c.q.cuda(), parents=par.cuda() if tree else None, **kw)
    f32freq = np.asarray(freq, np.float32).astype(np.float64) if rotary else None
    for b, ctx in enumerate(c.contexts):
        pos = ctx + okv.ancestors(par[b].tolist() if tree else None, n).sum(1) - 1
        turn = (lambda x: okv.rope(f64(x[b]), pos, f32freq, style, mag)) if rotary else (lambda x: f64(x[b]))
        q = turn(c.q)
        unit = 2.0 ** -9 if dtype is BF else 2.0 ** -24
        assert (np.abs(f64(got[b]) - q) <= 2 * unit * np.abs(q) + 1e-5 * np.abs(f64(c.q[b])).max(-1, keepdims=True) + 1e-30).all()
        t = ctx + np.arange(n)
        p, o = c.table[b].numpy()[t // page], t % page
        for which, x in ((0, turn(c.k)), (1, f64(c.v[b]))):
            have = values(c.caches[which], c.scales[which]).double().numpy()[p, o]
            scale = np.exp2(exps(c.scales[which])[p])[..., None]
            off = 5e-6 * mag * np.abs(f64(c.k[b] if which == 0 else c.v[b])).max(-1, keepdims=True) if which == 0 else 0.0
            assert (np.abs(have - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * scale) + 1.0001 * off).all()
            # the scale is the smallest that holds the page's largest: at least as large as needed, and not twice that
            most = {}
            for i in range(n):
                most[p[i]] = np.maximum(most.get(p[i], 0.0), np.abs(x[i]).max(-1))
            for page_id, m in most.items():
                e = exps(c.scales[which])[page_id]
                assert (m * (1 - 1e-5) <= 448 * np.exp2(e)).all()
                need = okv.scale_exponent(m * (1 + 1e-5))
                if page_id != p[0] or ctx % page == 0:
                    assert (e <= need).all()


def test_append_of_what_is_not_finite_and_of_extremes(sv):
    """NaN and infinities become NaN and do not enter the scale; the largest and smallest numbers; a block of zeros; cached tokens of a page whose
    scale grows by 2^1 to 2^30."""
    c = AppendCase(3, F32, [5, 0, 12], 6, 2, 2, 32, 8)
    inf = float("inf")
    c.k[0, 1, 0, :4] = torch.tensor([inf, -inf, float("nan"), 1.0])
    c.k[0, 0, 1] = torch.tensor(3.4e38)
    c.k[1] = 0.0
    c.v[1, 2, 0] = torch.finfo(F32).smallest_normal
    c.v[1, 2, 1, 7] = 1e-45
    c.v[2] *= 2.0 ** 40
    c.run(sv)
    for x, cache, scale, (codes, e) in zip((c.k, c.v), c.caches, c.scales, c.before):
        for b, ctx in enumerate(c.contexts):
            okv.append8(codes, e, f64(x[b]), ctx, c.table[b].numpy())
        np.testing.assert_array_equal(exps(scale), e)
        same_codes(cache, codes)
    assert exps(c.scales[0]).max() == 120 and exps(c.scales[0]).min() >= -120


def test_append_ragged_and_in_place(sv):
    """Ragged blocks (one empty), queries rotated in place; the same as block by block."""
    c = AppendCase(11, BF, [3, 20, 9], 9, 4, 2, 64, 8)
    sizes = [9, 0, 4]
    start = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    freq = torch.tensor(okv.rope_frequencies(64)[0], dtype=F32).cuda()
    q, k, v = (torch.cat([x[b, :s] for b, s in enumerate(sizes)]).cuda() for x in (c.q, c.k, c.v))
    ctx, table = torch.tensor(c.contexts, dtype=torch.int32).cuda(), c.table.cuda()
    ragged = [x.clone() for x in (*c.caches, *c.scales)]
    out = sv.sv_kv_append8(k, v, *ragged, ctx, table, q=q.clone(), inv_freq=freq, row_start=torch.tensor(start).cuda(), max_rows=9)
    one = [x.clone() for x in (*c.caches, *c.scales)]
    for b, s in enumerate(sizes):
        if s:
            r = slice(start[b], start[b + 1])
            own = q[None, r].clone()
            got = sv.sv_kv_append8(k[None, r], v[None, r], *one, ctx[b:b + 1], table[b:b + 1], q=own, q_out=own, inv_freq=freq)
            assert got is own and torch.equal(own[0], out[r])
    for x, y in zip(ragged, one):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def check_both(sv, c, q, kw, rows_of, par=None):
    """sv_kv_attend8 against the oracle over the values; where a block has more rows than the kernel for few takes, in bf16, it is sv_kv_attend
    over the values to the bit."""
    bits = q.dtype is BF and q.shape[-1] <= 128 and q.shape[1] * (q.shape[2] // c.k.shape[2]) > 32
    scale = kw.pop("scale", q.shape[-1] ** -0.5)
    stats = sv.new_stats("cuda")
    out, lse = sv.sv_kv_attend8(q, *c.args8, scale=scale, lse=True, stats=stats, **kw)
    assert sv.read_stats(stats)["status"] == 0
    check_attend8(c, q.flatten(0, 1) if q.dim() == 4 else q, out.flatten(0, 1) if q.dim() == 4 else out,
                 lse.flatten(0, 1) if q.dim() == 4 else lse, scale, rows_of, par)
    if bits:
        plain = sv.sv_kv_attend(q, c.k, c.v, *c.args8[4:], scale=scale, lse=True, **kw)
        assert torch.equal(out, plain[0]) and torch.equal(lse, plain[1])
    return out, lse


def filled(seed, dtype, contexts, n, H, kv, dim, page, order="psh", groups=None, spread=0):
    c = Cache8(seed, dtype, contexts, n, kv, dim, page, order, groups, spread)
    g = torch.Generator().manual_seed(seed)
    for b, ctx in enumerate(contexts):
        c.put(b, ctx, torch.randn((n, kv, dim), generator=g), torch.randn((n, kv, dim), generator=g))
    c.refresh()
    q = torch.randn((len(contexts), n, H, dim), generator=g).to(dtype).cuda()
    return c, q, [slice(b * n, b * n + n) for b in range(len(contexts))]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,H,kv,dim,page,order", [(1, 4, 4, 64, 16, "psh"), (6, 8, 2, 128, 16, "psh"), (4, 6, 2, 80, 24, "phs"), (33, 8, 2, 128, 8, "hps"),
                                                   (1, 8, 1, 128, 100, "psh"), (9, 4, 2, 96, 7, "phs"), (140, 4, 2, 64, 32, "psh"), (3, 2, 2, 16, 3, "psh"),
                                                   (5, 4, 1, 256, 16, "psh"), (2, 2, 1, 48, 1, "psh"), (300, 2, 1, 128, 64, "phs")])
def test_attend_over_codes(sv, dtype, n, H, kv, dim, page, order):
    c, q, rows = filled(n + dim, dtype, [0, 1, 127, 128, 700], n, H, kv, dim, page, order, spread=3)
    check_both(sv, c, q, {}, rows)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,dim,page", [(17, 64, 16), (57, 128, 24), (5, 128, 16)])
def test_attend_trees(sv, dtype, n, dim, page):
    c, q, rows = filled(n, dtype, [3, 250, 0], n, 4, 2, dim, page, spread=2)
    par = random_tree(c.rng, 3, n)
    check_both(sv, c, q, dict(parents=par.cuda()), rows, par)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,page,prefixes", [(6, 16, (320, 160)), (1, 16, (1024, 16)), (40, 8, (264, 128)), (3, 24, (0, 500))])
def test_attend_shared_prefixes(sv, dtype, n, page, prefixes):
    contexts = [prefixes[0] + x for x in (0, 5, 130)] + [prefixes[1] + x for x in (1, 40)]
    c = Cache8(n, dtype, contexts, n, 2, 128, page, groups=[(0, prefixes[0]), (3, prefixes[1])], spread=2)
    g = torch.Generator().manual_seed(n)
    for b, ctx in enumerate(contexts):
        c.put(b, ctx, torch.randn((n, 2, 128), generator=g), torch.randn((n, 2, 128), generator=g))
    # a prefix's last, partly filled page is every sequence's own copy: its scales too
    for b0, bs, pre in ((0, (1, 2), prefixes[0]), (3, (4,), prefixes[1])):
        if pre % page:
            for b in bs:
                for s in (c.ks, c.vs):
                    s[c.table[b, pre // page].long()] = s[c.table[b0, pre // page].long()]
    c.refresh()
    q = torch.randn((5, n, 8, 128), generator=g).to(dtype).cuda()
    check_both(sv, c, q, dict(c.group_args), [slice(b * n, b * n + n) for b in range(5)])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [-0.3, 0.0, 40.0])
def test_attend_scales_of_either_sign_and_scale_bytes_at_the_ends(sv, dtype, scale):
    """Scales from 2^-100 to 2^30 beside one another."""
    c, q, rows = filled(5, dtype, [40, 300], 4, 4, 2, 64, 8, spread=2)
    c.vs.copy_(torch.tensor(c.rng.integers(27, 157, tuple(c.vs.shape)).astype(np.uint8)))
    c.ks.copy_(torch.tensor(c.rng.integers(100, 121, tuple(c.ks.shape)).astype(np.uint8)))
    c.refresh()
    check_both(sv, c, q, dict(scale=scale), rows)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [3, 40])
@pytest.mark.parametrize("large", [100, 127, 150])
def test_a_first_page_of_zeros_before_the_largest_values(sv, dtype, n, large):
    """Keys and values of zeros (their scale is the least, and counts as 2^-40) before pages of values up to 2^31, whose scales are at most 2^64 above
    that, as far as the sum of the weights holds those of the zeros: a weight times its scale is 2^(4 - 40 - 64 - d) there or more, d bits below its
    row's largest, and float32 ends at 2^-126, so what is lost is below 2^-26.  A context that is split over blocks beside short ones."""
    c, q, rows = filled(n + large, dtype, [9000, 40, 300], n, 4, 2, 64, 16)
    for b in range(3):
        first = c.table[b, 0].long()
        for codes, scale in ((c.k8, c.ks), (c.v8, c.vs)):
            codes.view(torch.uint8)[first] = 0
            scale[first] = 7
        c.vs[c.table[b, 1:].long()] = torch.tensor(c.rng.integers(large - 30, large + 1, (c.table.shape[1] - 1, 2)).astype(np.uint8)).cuda()
    c.refresh()
    check_both(sv, c, q, {}, rows)


@pytest.mark.parametrize("dtype,n,dim", [(BF, 4, 128), (BF, 60, 64), (F32, 4, 64), (BF, 3, 192), (F32, 40, 128)])
def test_hidden_tokens_cannot_reach_a_row(sv, dtype, n, dim):
    """NaN codes, NaN scales, pages that nobody sees: slots past the block and a tree's other branches.  A value of NaN that a row sees makes it NaN and no other."""
    c, q, rows = filled(n, dtype, [100, 30], n, 4, 2, dim, 16)
    used = torch.zeros(c.ks.shape[0], dtype=torch.bool)
    for b, ctx in enumerate(c.contexts):
        used[c.table[b, :(ctx + n + 15) // 16].long()] = True
    for s in (c.ks, c.vs):
        s[~used.cuda()] = 255
    c.refresh()
    check_both(sv, c, q, {}, rows)
    # row 1's own value is NaN in one element of head 0: later rows see it, row 0 does not
    t = c.contexts[0] + 1
    c.v8.view(torch.uint8)[c.table[0, t // 16].long(), t % 16, 0, 5] = 0x7F
    out, _ = sv.sv_kv_attend8(q, *c.args8)
    bad = torch.isnan(out).cpu()
    want = torch.zeros_like(bad)
    want[0, 1:, :2, 5] = True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("dtype,n,dim", [(BF, 6, 128), (BF, 7, 64), (BF, 60, 64), (F32, 2, 64), (F32, 20, 96)])
@pytest.mark.parametrize("most", [13, 30, 60, 110])
def test_query_rows_of_very_different_size(sv, dtype, n, dim, most):
    """Rows (each head's) between 2^-most and 1 beside rows of zeros, with scores up to some 2^3 and, by the scale, 2^20 (at 2^22 float32 no longer tells
    scores apart)."""
    c, q, rows = filled(n + most, dtype, [200, 0, 33], n, 4, 2, dim, 16, spread=2)
    size = torch.tensor(2.0 ** -c.rng.integers(0, most + 1, (3, n, 4, 1)), dtype=F32)
    size[0, 0, 1] = 0.0
    size[0, 1, 2] = 2.0 ** -most
    size[0, 2 % n, 3] = 1.0
    q = (q.float().cpu() * size).to(dtype).cuda()
    for scale in (dim ** -0.5, 2.0 ** (min(most, 18) - 4)):
        check_both(sv, c, q, dict(scale=scale), rows)


@pytest.mark.parametrize("dtype,n", [(BF, 4), (BF, 40), (F32, 2), (F32, 30)])
def test_a_scale_that_is_nan_reaches_whoever_sees_it(sv, dtype, n):
    """However small the weight of its tokens: by the values' scale and by the keys'."""
    for which in range(2):
        c, q, rows = filled(n, dtype, [100, 70], n, 4, 2, 64, 16)
        if which == 0:
            c.k8.view(torch.uint8)[c.table[0, 2].long(), :, 0] = 0   # the page's keys: scores of 0, beside those of 1000 and more
            q[0, :, 0] = 100 * c.k[c.table[0, 0].long(), 3, 0]
        (c.vs, c.ks)[which][c.table[0, 2].long(), 0] = 255
        out, lse = sv.sv_kv_attend8(q, *c.args8, lse=True)
        bad = torch.isnan(out).cpu()
        want = torch.zeros_like(bad)
        want[0, :, :2] = True
        assert torch.equal(bad, want)
        assert torch.equal(torch.isnan(lse).cpu(), want[..., 0] if which else torch.zeros_like(want[..., 0]))


def test_rows_of_no_token_and_empty_blocks(sv):
    """Ragged: an empty block, a block without context."""
    c, q, _ = filled(2, BF, [0, 50, 9], 4, 4, 2, 64, 16)
    start = torch.tensor([0, 4, 4, 7], dtype=torch.int32).cuda()
    flat = torch.cat([q[0], q[2, :3]])
    out, lse = sv.sv_kv_attend8(flat, *c.args8, row_start=start, max_rows=4, lse=True)
    one, l1 = sv.sv_kv_attend8(q, *c.args8, lse=True)
    assert torch.equal(out[:4], one[0])
    check_attend8(c, flat, out, lse, 64 ** -0.5, [slice(0, 4), slice(4, 4), slice(4, 7)])


def test_long_contexts_split_over_blocks(sv):
    """Units that several blocks share, beside short ones; twice the same to the bit."""
    c, q, rows = filled(8, BF, [20000, 3, 9000, 17], 3, 8, 2, 128, 64, spread=4)
    a = check_both(sv, c, q, {}, rows)
    b = sv.sv_kv_attend8(q, *c.args8, lse=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def path_of(rng, n, acc):
    return np.sort(rng.choice(np.arange(1, n), acc, replace=False)).astype(np.int32)


@pytest.mark.parametrize("layers,page,kv,dim,n", [(1, 16, 2, 64, 9), (3, 4, 3, 48, 30), (2, 1, 1, 16, 12), (2, 100, 9, 128, 129), (5, 7, 8, 256, 20)])
def test_commit_is_the_oracles_to_the_bit(sv, layers, page, kv, dim, n):
    rng = np.random.default_rng(n)
    contexts = [0, 5, page - 1, 37, 64]
    B, each = len(contexts), (64 + n) // page + 2
    P = B * each + 2
    table = rng.permutation(P)[:B * each].reshape(B, each).astype(np.int32)
    acc = [0, n - 1, min(3, n - 1), n // 2, 1]
    path = np.full((B, n - 1), -1, np.int32)
    for b in range(B):
        path[b, :acc[b]] = path_of(rng, n, acc[b])
    tensors, want = [], []
    for _ in range(2):
        c, s = random_codes(rng, (layers, P, page, kv, dim), 0x7E), torch.tensor(rng.integers(110, 122, (layers, P, kv)).astype(np.uint8))
        codes, e = c.view(E4M3).double().numpy().copy(), s.numpy().astype(np.int64) - 127
        for b in range(B):
            okv.commit8(codes, e, contexts[b], table[b], acc[b], path[b])
        tensors.append((c.cuda().view(E4M3), s.cuda()))
        want.append((codes, e))
    (k, ks), (v, vs) = tensors
    ctx = sv.sv_kv_commit8(k, v, ks, vs, torch.tensor(contexts, dtype=torch.int32).cuda(), torch.tensor(table).cuda(),
                           torch.tensor(acc, dtype=torch.int32).cuda(), torch.tensor(path).cuda())
    assert ctx.tolist() == [c + 1 + a for c, a in zip(contexts, acc)]
    for (c, s), (codes, e) in zip(tensors, want):
        np.testing.assert_array_equal(exps(s), e)
        same_codes(c, codes)


def test_bad_device_arrays_are_reported(sv):
    """A page id outside the pool, contexts outside the table, a path that does not rise: an error in stats, nothing written elsewhere."""
    from speculative_decoding_verification_gb300 import _abi
    c = AppendCase(4, BF, [3, 9], 4, 2, 2, 32, 8)
    good = c.table.clone()
    was = [x.view(torch.uint8).clone() for x in (*c.caches, *c.scales)]
    for table, ctx in (((0, 0, 99), None), ((1, 1, -1), None), (None, [3, 8 * good.shape[1]]), (None, [-1, 9])):
        c.table = good.clone()
        if table:
            c.table[table[0], table[1]] = table[2]
        c.contexts = ctx or [3, 9]
        st = sv.new_stats("cuda")
        for x, y in zip((*c.caches, *c.scales), was):
            x.view(torch.uint8).copy_(y)
        c.run(sv, stats=st)
        assert sv.read_stats(st)["status"] == _abi.SV_ERR_INVALID_ARG
        sv.sv_kv_attend8(c.q.cuda(), *c.caches, *c.scales, torch.tensor(c.contexts, dtype=torch.int32).cuda(), c.table.cuda(), stats=st)
        assert sv.read_stats(st)["status"] == _abi.SV_ERR_INVALID_ARG
    free = [p for p in range(was[0].shape[0]) if p not in good.flatten().tolist()]
    for x, y in zip((*c.caches, *c.scales), was):
        assert torch.equal(x.view(torch.uint8)[free], y[free])
    k, v, ks, vs = (x[None].contiguous() for x in (*c.caches, *c.scales))
    for acc, path in (([2, 0], [[2, 1, -1]] * 2), ([4, 0], [[1, 2, 3]] * 2), ([1, 0], [[9, -1, -1]] * 2)):
        st = sv.new_stats("cuda")
        before = k.view(torch.uint8).clone()
        out = sv.sv_kv_commit8(k, v, ks, vs, torch.tensor([3, 9], dtype=torch.int32).cuda(), good.cuda(), torch.tensor(acc, dtype=torch.int32).cuda(),
                               torch.tensor(path, dtype=torch.int32).cuda(), stats=st)
        assert sv.read_stats(st)["status"] == _abi.SV_ERR_INVALID_ARG and out.tolist() == [3, 10]
        assert torch.equal(before, k.view(torch.uint8))


@pytest.mark.parametrize("n", [4, 60])
def test_in_a_graph_and_on_two_streams(sv, n):
    c, q, _ = filled(n, BF, [3000, 20, 777], n, 8, 2, 128, 16, spread=1)
    want = sv.sv_kv_attend8(q, *c.args8, lse=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = sv.sv_kv_attend8(q, *c.args8, lse=True)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        graph.replay()
        other = [sv.sv_kv_attend8(q, *c.args8, lse=True, stream=s) for s in streams]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for x in (got, *other) for a, b in zip(x, want))


def test_a_step_as_it_is_used(sv):
    """Rounds of append, attention and commit of drafted trees against the same rounds in float64 over unrounded keys and values: attention over
    the cache is the oracle's over what the codes stand for, and those are within half a step, and one more for each time a page's scale grew,
    of what was appended."""
    rng = np.random.default_rng(0)
    B, n, H, kv, D, page, rounds = 3, 13, 4, 2, 64, 8, 12
    P = B * 16
    table = rng.permutation(P).reshape(B, 16).astype(np.int32)
    k8, v8 = (torch.zeros((1, P, page, kv, D), dtype=torch.uint8).cuda().view(E4M3) for _ in range(2))
    ks, vs = (torch.zeros((1, P, kv), dtype=torch.uint8).cuda() for _ in range(2))
    true = [[np.zeros((0, kv, D)) for _ in range(B)] for _ in range(2)]
    ctx = torch.zeros(B, dtype=torch.int32).cuda()
    dev_table = torch.tensor(table).cuda()
    for r in range(rounds):
        par = random_tree(rng, B, n)
        q = torch.tensor(rng.normal(size=(B, n, H, D)), dtype=BF)
        k, v = (torch.tensor(rng.normal(size=(B, n, kv, D)) * 2.0 ** rng.integers(-2, 3), dtype=BF) for _ in range(2))
        sv.sv_kv_append8(k.cuda(), v.cuda(), k8[0], v8[0], ks[0], vs[0], ctx, dev_table, parents=par.cuda())
        out, lse = sv.sv_kv_attend8(q.cuda(), k8[0], v8[0], ks[0], vs[0], ctx, dev_table, parents=par.cuda(), lse=True)
        held = SimpleNamespace(contexts=ctx.tolist(), table=torch.tensor(table), k=values(k8[0], ks[0]), v=values(v8[0], vs[0]))
        check_attend8(held, q.flatten(0, 1), out.flatten(0, 1).cpu(), lse.flatten(0, 1).cpu(), D ** -0.5,
                     [slice(b * n, b * n + n) for b in range(B)], par)
        acc = rng.integers(0, n, B).astype(np.int32)
        path = np.full((B, n - 1), -1, np.int32)
        for b in range(B):
            path[b, :acc[b]] = path_of(rng, n, acc[b])
            keep = [0, *path[b, :acc[b]]]
            true[0][b] = np.concatenate([true[0][b], f64(k[b])[keep]])
            true[1][b] = np.concatenate([true[1][b], f64(v[b])[keep]])
        new = sv.sv_kv_commit8(k8, v8, ks, vs, ctx, dev_table, torch.tensor(acc).cuda(), torch.tensor(path).cuda())
        room = np.array([len(x) for x in true[0]]) + n <= 16 * page
        assert new.tolist() == [len(x) for x in true[0]]
        ctx = new
        if not room.all():
            break
    assert r > 1
    for codes, scale, want in ((k8, ks, true[0]), (v8, vs, true[1])):
        have = values(codes[0], scale[0]).double().numpy()
        for b in range(B):
            t = np.arange(len(want[b]))
            p, o = table[b][t // page], t % page
            # each rounding is off by half a step of the scale then, at most today's: 2^-4 of the number, or 2^-10 of the scale.  A number is
            # rounded when appended and where the scale grows, from 2^-2 to 2^2 here: a power of two changes the fraction's bits only for
            # numbers that become subnormal, so the first error counts once and the second up to three times
            tol = 2.0 ** -4 * np.abs(want[b]) + 4 * 2.0 ** -10 * np.exp2(exps(scale[0])[p])[..., None]
            assert (np.abs(have[p, o] - want[b]) <= tol).all()
