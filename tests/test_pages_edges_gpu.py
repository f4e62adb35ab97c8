"""GPU tests of a cache's pages where counts and tables do not fit, and of ends of batches."""
import numpy as np
import pytest
import torch

from test_pages_gpu import BF, E4M3, Pool

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_gb300 as sv
    sv.load()
    return sv


@pytest.mark.parametrize("src", [(0, 1, 2, 3), (0, 0, 1, 1, 3), (3, 3, 3, 0, 0, 0)])
@pytest.mark.parametrize("lacking", [0, 1, 2, 8, 13])
def test_counts_below_the_holders_are_reported_and_give_no_page_away(sv, src, lacking):
    """A page that the old table names more often than refs says: reported with its number, also where as many sequences come to it as leave
    it, and it is nobody else's afterwards."""
    from speculative_decoding_verification_gb300 import _abi
    p = Pool(4, 2, 4, 2, 16, E4M3, 4, 30, extra=40)
    p.ctx[:] = [8, 9, 13, 6]
    p.table[:] = -1
    for b, pages in enumerate(([0, 1, 9], [0, 2, 3], [4, 5, 6, 8], [0, 13])):   # page 0 is three sequences' first, 9 a page without tokens
        p.table[b, :len(pages)] = pages
    p.refs[:] = 0
    np.add.at(p.refs, p.table[p.table >= 0], 1)
    stats = sv.new_stats("cuda")
    p.fork(sv, src, 6, stats=stats)
    assert sv.read_stats(stats)["status"] == 0
    p.refs[lacking] -= 1
    table, ctx, refs = p.fork(sv, src, 6, stats=stats)
    st = sv.read_stats(stats)
    assert (st["status"], st["error_index"]) == (_abi.SV_ERR_INVALID_ARG, lacking)
    table, refs, ctx = table.cpu().numpy(), refs.cpu().numpy(), ctx.tolist()
    assert ctx == [p.ctx[b] for b in src] and (refs >= 0).all()
    for j, b in enumerate(src):
        full = ctx[j] // 4
        np.testing.assert_array_equal(table[j, :full], p.table[b, :full])   # shared pages
        new = table[j, full:][table[j, full:] >= 0]
        assert len(new) == -(-(ctx[j] + 6) // 4) - full
        others = np.concatenate([table[i] for i in range(len(src)) if i != j] + [table[j, :full]])
        assert not set(new.tolist()) & set(others.tolist())   # what a sequence will write is its own
        assert (refs[new] == 1).all()
    named = np.bincount(table[table >= 0], minlength=p.pages)
    assert (refs >= named).all()


@pytest.mark.parametrize("dtype", [torch.uint8, torch.int8, torch.float8_e5m2])
def test_one_byte_caches_without_scales_of_their_pages(sv, dtype):
    """Their bytes move as those of a cache held in 8 bits do; that one is refused without its scales."""
    p = Pool(5, 2, 4, 2, 32, E4M3, 6, 40)
    src = np.array([0, 0, 1, 3, 3, 5])
    plain = [c.clone().view(dtype) for c in p.caches]
    table, ctx, refs = p.fork(sv, src, 3)
    got = sv.sv_kv_fork(*plain, p.dev(p.refs), p.dev(p.ctx), p.dev(p.table), p.dev(src), reserve=3)
    assert all(torch.equal(a, b) for a, b in zip(got, (table, ctx, refs)))
    want = sv.sv_kv_compact(*p.caches, refs, table, **p.kw)
    got = sv.sv_kv_compact(*plain, refs, table)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for a, b in zip(plain, p.caches):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    with pytest.raises(ValueError, match="scales"):
        sv.sv_kv_fork(*p.caches, p.dev(p.refs), p.dev(p.ctx), p.dev(p.table), p.dev(src))


def test_a_batch_that_ends_whole(sv):
    """No new sequences: every page goes that nobody else holds."""
    p = Pool(6, 2, 4, 2, 16, BF, 5, 30)
    for refs_out in (None, p.dev(p.refs)):
        table, ctx, refs = p.fork(sv, np.zeros(0), 4, refs_out=refs_out)
        left = p.refs.copy()
        np.subtract.at(left, p.table[p.table >= 0], 1)
        assert table.shape == (0, p.width) and ctx.shape == (0,) and refs.tolist() == left.tolist()
        assert refs_out is None or refs is refs_out
    p.check_bytes([])
