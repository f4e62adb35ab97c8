"""GPU tests of attention over codes where it can go wrong: the same calls in every kernel, against the oracle."""
import pytest
import torch

from kv8_helpers import Cache8, check_attend8
from test_kv8_gpu import filled

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

# type, rows, query heads, width: the kernel for few rows of either type, that for more, and that of wide heads
KERNELS = [(BF, 4, 4, 64), (BF, 5, 8, 128), (BF, 40, 4, 128), (BF, 3, 4, 192), (F32, 1, 4, 64), (F32, 3, 4, 128), (F32, 30, 4, 64)]


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_gb300 as sv
    sv.load()
    return sv


def spare_first_page(c):
    """Moves what page 0 holds elsewhere: (cache, numbers of two pages that no table names)."""
    free = sorted(set(range(c.k8.shape[0])) - set(c.table.flatten().tolist()))
    if 0 not in free:
        to = free.pop()
        for x in (c.k8, c.v8, c.ks, c.vs):
            x.view(torch.uint8)[to] = x.view(torch.uint8)[0]
        c.table[c.table == 0] = to
        c.args["page_table"] = c.table.cuda()
        free = [0] + free
    return free[0], free[1]


@pytest.mark.parametrize("dtype,n,H,dim", KERNELS)
@pytest.mark.parametrize("bad", [-1, -7, 1 << 20, 2 ** 31 - 1])
def test_a_page_outside_the_pool_reads_zeros_whatever_the_first_page_holds(sv, dtype, n, H, dim, bad):
    """It is reported; its tokens have keys and values of 0, and no other page's scale has to do with them."""
    from speculative_decoding_verification_gb300 import _abi
    c, q, rows = filled(n + dim, dtype, [300, 70, 130], n, H, 2, dim, 16, spread=2)
    first, zeros = spare_first_page(c)
    for s in (c.ks, c.vs):
        s[first] = 255
        s[zeros] = 127
    for x in (c.k8, c.v8):
        x.view(torch.uint8)[first] = 0x7F
        x.view(torch.uint8)[zeros] = 0
    table = c.table.clone()
    for b, entry in ((0, 3), (0, 17), (1, 0), (2, 4)):
        table[b, entry] = bad
        c.table[b, entry] = zeros
    c.refresh()
    stats = sv.new_stats("cuda")
    out, lse = sv.sv_kv_attend8(q, *c.args8[:5], table.cuda(), lse=True, stats=stats)
    assert sv.read_stats(stats)["status"] == _abi.SV_ERR_INVALID_ARG
    check_attend8(c, q.flatten(0, 1), out.flatten(0, 1), lse.flatten(0, 1), dim ** -0.5, rows)


@pytest.mark.parametrize("dtype,n,H,dim", KERNELS)
@pytest.mark.parametrize("prefix", [0, 1024])
def test_nan_reaches_every_row_from_a_part_of_the_context_without_weight(sv, dtype, n, H, dim, prefix):
    """A value of NaN, by its code and by its scale, among tokens that another block works on, or that the prefix holds, and whose weights underflow
    beside the largest."""
    ctx = [prefix + 2500, prefix + 40]
    for by_scale in (False, True):
        c = Cache8(n + dim, dtype, ctx, n, 2, dim, 16, groups=[(0, prefix)] if prefix else None)
        g = torch.Generator().manual_seed(7)
        for b in range(2):
            c.put(b, ctx[b], torch.randn((n, 2, dim), generator=g), torch.randn((n, 2, dim), generator=g))
        c.refresh()
        q = torch.randn((2, n, H, dim), generator=g).to(dtype).cuda()
        k8, v8 = c.k8.view(torch.uint8), c.v8.view(torch.uint8)
        for b, at, best in ((0, 100, ctx[0] - 200), (1, 100 if prefix else 3, ctx[1] - 3)):
            page, place = c.table[b, at // 16].long(), at % 16
            k8[page, :, 0] = 0   # scores of 0 beside those of 1000 and more
            q[b, :, : H // 2] = 1000.0 * c.k[c.table[b, best // 16].long(), best % 16, 0]
            if by_scale:
                c.vs[page, 0] = 255
            else:
                v8[page, place, 0, 3] = 0x7F
        out, lse = sv.sv_kv_attend8(q, *c.args8, lse=True, **c.group_args)
        want = torch.zeros(out.shape, dtype=torch.bool)
        want[:, :, : H // 2, slice(None) if by_scale else slice(3, 4)] = True
        assert (torch.isnan(out).cpu() == want).all(), by_scale
        assert not torch.isnan(lse).any()


@pytest.mark.parametrize("dtype,n,H,dim", KERNELS)
@pytest.mark.parametrize("ctx", [37, 133, 6, 200])
@pytest.mark.parametrize("tree", [False, True])
def test_nan_reaches_whoever_sees_it_however_small_its_weight(sv, dtype, n, H, dim, ctx, tree):
    """A value's NaN code or NaN scale at a token whose weight underflows to 0, among tokens that not all rows see: a cached one near the block, and
    one of the block's own."""
    if tree and n < 3:
        pytest.skip("no tree")
    for at, by_scale in ((ctx - 1, False), (ctx - 1, True), (ctx + n // 2, False)):
        c, q, _ = filled(n + dim, dtype, [ctx, 20], n, H, 2, dim, 8)
        k8, v8 = c.k8.view(torch.uint8), c.v8.view(torch.uint8)
        page, place = c.table[0, at // 8].long(), at % 8
        k8[page, place, 0] = 0                               # a score of 0 beside those of 1000 and more
        q[0, :, : H // 2] = 1000.0 * c.k[c.table[0, 0].long(), 1, 0]
        if by_scale:
            c.vs[page, 0] = 255
            seen_from, elements = at - at % 8, slice(None)
        else:
            v8[page, place, 0, 3] = 0x7F
            seen_from, elements = at, slice(3, 4)
        par = torch.tensor([[0] * (n - 1)] * 2, dtype=torch.int32) if tree else None   # all of them children of row 0
        out, lse = sv.sv_kv_attend8(q, *c.args8, lse=True, parents=None if par is None else par.cuda())
        want = torch.zeros(out.shape, dtype=torch.bool)
        for i in range(n):
            seen = seen_from <= ctx or i == seen_from - ctx if tree else seen_from <= ctx + i
            want[0, i, : H // 2, elements] = seen
        assert (torch.isnan(out).cpu() == want).all(), (at, by_scale)
        assert not torch.isnan(lse).any()
