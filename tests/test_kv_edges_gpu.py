"""GPU tests of attention at the edges of its inputs: infinite values that rows see, scales of either sign and none, scores near the
ends of float32, blocks of all shapes in every kernel.  The kernels are named by what takes a call there: "few" for bf16 with up to 32
packed rows a sequence and key head, "tall" for bf16 with more, "few32" for float32 with up to 8, "small32" up to 16, "f32" for more."""
import numpy as np
import pytest
import torch

from kv_helpers import U32, Cache, check_attend, random_tree

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

# kernel, dtype, rows, heads, kv_heads, dim
KERNELS = [("few", BF, 5, 8, 2, 128), ("few", BF, 3, 4, 4, 64), ("tall", BF, 40, 8, 2, 128), ("tall", BF, 150, 4, 2, 64),
           ("few32", F32, 2, 8, 2, 64), ("few32", F32, 1, 4, 1, 128), ("small32", F32, 4, 8, 2, 80), ("f32", F32, 30, 8, 2, 64),
           ("wide", BF, 2, 4, 2, 256), ("wide", BF, 30, 4, 2, 136)]


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_gb300 as sv
    sv.load()
    return sv


def randn(seed, *shape, dtype=F32):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def block(c, seed, n, heads, kv, dim, dtype, size=2.0):
    """Queries [B, n, heads, dim]; the block's keys and values go to the slots after each context."""
    B = len(c.contexts)
    for b in range(B):
        c.put(b, c.contexts[b], randn(seed + 1 + b, n, kv, dim), randn(seed + 101 + b, n, kv, dim))
    return randn(seed, B, n, heads, dim, dtype=dtype) * size


def rows_of(B, n):
    return [slice(b * n, b * n + n) for b in range(B)]


@pytest.mark.parametrize("kernel,dtype,n,heads,kv,dim", KERNELS)
@pytest.mark.parametrize("pre", [0, 384])
def test_infinite_values_that_rows_see(sv, kernel, dtype, n, heads, kv, dim, pre):
    """An infinite value reaches every row that sees it as that infinity, wherever its token lies; infinities of both signs
    and NaN as NaN; the other elements stay those of the finite ones."""
    ctx = [pre + 700, pre + 130]
    c = Cache(n + dim, dtype, ctx, n, kv, dim, 16, groups=[(0, pre)] if pre else None)
    q = block(c, 30, n, heads, kv, dim, dtype)
    inf, page = float("inf"), 16
    tokens = [pre + 3, pre + 127, pre + 128, pre + 129] + ([5, 300] if pre else [])
    for b, cx in enumerate(ctx):
        for t in tokens + [cx]:   # the last one is the block's first row
            at = int(c.table[b, t // page]), t % page
            c.v[at][:, 3] = inf
            c.v[at][:, 4] = -inf
            c.v[at][:, 5] = inf if t % 2 else -inf
            c.v[at][:, 6] = float("nan")
    out, lse = sv.sv_kv_attend(q, c.k, c.v, lse=True, **c.args, **c.group_args)
    assert bool((out[..., 3] == inf).all()) and bool((out[..., 4] == -inf).all())
    assert bool(out[..., 5:7].isnan().all()) and bool(torch.isfinite(lse).all())
    keep = [d for d in range(dim) if d not in (3, 4, 5, 6)]
    assert bool(torch.isfinite(out[..., keep]).all())
    c.v[..., 3:7] = 0.0
    out[..., 3:7] = 0.0
    check_attend(c, q.flatten(0, 1), out.flatten(0, 1), lse.flatten(0, 1), dim ** -0.5, rows_of(2, n))


@pytest.mark.parametrize("kernel,dtype,n,heads,kv,dim", KERNELS)
@pytest.mark.parametrize("size,scale", [(1.0, 0.0), (1e16, 0.0), (1e16, 1e-33), (1e16, -1e-34)])
def test_small_scales_of_large_products(sv, kernel, dtype, n, heads, kv, dim, size, scale):
    """Scores are scale times q.k, however small the one and large the other."""
    ctx = [300, 40]
    c = Cache(dim, dtype, ctx, n, kv, dim, 16)
    q = block(c, 50, n, heads, kv, dim, dtype, size)
    c.k.mul_(size)
    out, lse = sv.sv_kv_attend(q, c.k, c.v, lse=True, scale=scale, **c.args)
    check_attend(c, q.flatten(0, 1), out.flatten(0, 1), lse.flatten(0, 1), scale, rows_of(2, n))


@pytest.mark.parametrize("kernel,dtype,n,heads,kv,dim", KERNELS)
@pytest.mark.parametrize("scale", [-0.11, 0.0, 0.37])
@pytest.mark.parametrize("pre", [0, 272])
def test_scales_of_either_sign(sv, kernel, dtype, n, heads, kv, dim, scale, pre):
    """Every kernel, alone and with a prefix (few rows then go beside the kernel that takes the prefix), chains and trees."""
    ctx = [pre + 410, pre + 3, pre + 128]
    c = Cache(n + kv, dtype, ctx, n, kv, dim, 16, groups=[(0, pre)] if pre else None)
    q = block(c, 60, n, heads, kv, dim, dtype)
    par = random_tree(c.rng, 3, n) if 1 < n <= 129 else None
    for parents in (None, par) if par is not None else (None,):
        kw = {} if parents is None else dict(parents=parents.cuda())
        out, lse = sv.sv_kv_attend(q, c.k, c.v, lse=True, scale=scale, **kw, **c.args, **c.group_args)
        check_attend(c, q.flatten(0, 1), out.flatten(0, 1), lse.flatten(0, 1), scale, rows_of(3, n), parents)


@pytest.mark.parametrize("kernel,dtype,n,heads,kv,dim", KERNELS)
@pytest.mark.parametrize("pre", [0, 256])
def test_ragged_in_every_kernel(sv, kernel, dtype, n, heads, kv, dim, pre):
    """Ragged blocks up to each kernel's rows, over contexts whose units several blocks share; with max_rows left out the number of
    all rows decides on the kernel."""
    lens = [n, 0, 1, (n + 1) // 2, n, 0, 1, n]
    ctx = [pre + x for x in (1900, 40, 700, 3, 128, 0, 2500, 1030)]
    starts = np.concatenate([[0], np.cumsum(lens)]).tolist()
    c = Cache(n + dim, dtype, ctx, n, kv, dim, 16, groups=[(0, pre), (5, pre)] if pre else None)
    q = randn(70, starts[-1], heads, dim, dtype=dtype) * 2
    for b, m in enumerate(lens):
        if m:
            c.put(b, ctx[b], randn(71 + b, m, kv, dim), randn(171 + b, m, kv, dim))
    rows = [slice(starts[b], starts[b + 1]) for b in range(len(lens))]
    kw = dict(row_start=torch.tensor(starts, dtype=torch.int32).cuda(), **c.args, **c.group_args)
    for most in (n, None):
        st = sv.new_stats("cuda")
        out, lse = sv.sv_kv_attend(q, c.k, c.v, max_rows=most, lse=True, stats=st, **kw)
        assert sv.read_stats(st)["status"] == 0
        check_attend(c, q, out, lse, dim ** -0.5, rows)
        assert torch.equal(out, sv.sv_kv_attend(q, c.k, c.v, max_rows=most, **kw)[0])


@pytest.mark.parametrize("dtype,dim,heads,kv", [(BF, 128, 4, 2), (BF, 64, 4, 1), (F32, 64, 4, 2), (BF, 160, 2, 2)])
@pytest.mark.parametrize("ctx", [[0, 0], [0, 900], [1111, 64]])
def test_long_prompts(sv, dtype, dim, heads, kv, ctx):
    """Prompts of 1,300 and 700 rows in one ragged call, each row over all rows before it; a sample of rows is checked, among them the
    first and last of row tiles."""
    lens = [1300, 700]
    c = Cache(dim, dtype, ctx, 1300, kv, dim, 32)
    q = randn(80, 2000, heads, dim, dtype=dtype) * 2
    for b, first in ((0, 0), (1, 1300)):
        c.put(b, ctx[b], randn(81 + b, lens[b], kv, dim), randn(91 + b, lens[b], kv, dim))
    out, lse = sv.sv_kv_attend(q, c.k, c.v, row_start=torch.tensor([0, 1300, 2000], dtype=torch.int32).cuda(), max_rows=1300, lse=True, **c.args)
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    for b, first in ((0, 0), (1, 1300)):
        for i in sorted({0, 1, 63, 64, 127, 128, 255, 256, 383, 511, 512, lens[b] // 2 + 1, lens[b] - 2, lens[b] - 1}):
            at = Cache.__new__(Cache)   # the same cache with the rows before i as its context
            at.k, at.v, at.table, at.contexts = c.k, c.v, c.table, list(ctx)
            at.contexts[b] += i
            r = [slice(0, 0)] * 2
            r[b] = slice(first + i, first + i + 1)
            check_attend(at, q, out, lse, dim ** -0.5, r)


def test_costs_past_30_bits(sv):
    """32,768 rows of two million cached tokens each, which all lie in one page: 1.07e9 key tiles.  32 repeats of a page weigh as the
    page itself, with log(32) more in the log-sum-exp.  A warp adds up to 2^18 weighted values in a row; roundings of alternating
    sign leave about sqrt(2^18) u32 = 2^-15 of the largest value, and a lane's 2^15 weights sqrt(2^15) u32 = 2^-16.5 of their sum.
    Eight times that is allowed."""
    B, H, page, reps, dim = 1024, 32, 1 << 16, 32, 4
    k, v = randn(1, 1, page, H, dim), randn(2, 1, page, H, dim)
    q = randn(3, B, 1, H, dim)
    ctx = torch.full((B,), reps * page, dtype=torch.int32).cuda()
    table = torch.zeros((B, reps + 1), dtype=torch.int32).cuda()
    st = sv.new_stats("cuda")
    k[0, 0], v[0, 0] = k[0, 1], v[0, 1]   # the rows' own token is the first slot of the page, once more
    out, lse = sv.sv_kv_attend(q, k, v, ctx, table, lse=True, stats=st)
    assert sv.read_stats(st)["status"] == 0
    for b in (0, 1, 511, 1022, 1023):
        s = torch.einsum("hd,thd->ht", q[b, 0].double(), k[0].double()) * dim ** -0.5
        w = s.exp() * reps
        w[:, 0] *= 1 + 1 / reps
        want = torch.einsum("ht,thd->hd", w, v[0].double()) / w.sum(1, keepdim=True)
        assert float((out[b, 0] - want).abs().max()) <= 2.0 ** -12 * float(v.abs().max())
        assert float((lse[b, 0] - w.sum(1).log()).abs().max()) <= 2.0 ** -13.5 + 16 * U32
