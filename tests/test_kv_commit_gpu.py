"""GPU tests of the commit after ragged blocks, and at the end of a page table."""
import numpy as np
import pytest
import torch

from kv_helpers import f64
from oracle import kv as okv

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_gb300 as sv
    sv.load()
    return sv


def i32(*x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def caches(dtype, layers=2, pages=20, page=4, kv=2, dim=64, seed=0):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn((layers, pages, page, kv, dim), generator=g).to(dtype).cuda() for _ in range(2)]


TABLE = [[3, 17, 5], [0, 9, 12], [7, 1, 19], [2, 11, 4]]   # 12 slots a sequence


@pytest.mark.parametrize("dtype", [BF, F32])
def test_commit_ragged(sv, dtype):
    """A block of three rows that ends where its pages do, an empty one at the end of its pages, a full one, a single row."""
    k, v = caches(dtype)
    ctx, lens, acc = [9, 12, 2, 11], [3, 0, 5, 1], [1, 0, 3, 0]
    path = [[2, -1, -1, -1], [-1] * 4, [1, 3, 4, -1], [-1] * 4]
    k64, v64 = f64(k), f64(v)
    want = [okv.commit(k64, v64, c, np.array(t), a, p) if n else c for c, t, a, p, n in zip(ctx, TABLE, acc, path, lens)]
    starts = np.concatenate([[0], np.cumsum(lens)])
    st = sv.new_stats("cuda")
    got = sv.sv_kv_commit(k, v, i32(*ctx), i32(*TABLE), i32(*acc), i32(*path), row_start=i32(*starts.tolist()), stats=st)
    assert sv.read_stats(st)["status"] == 0
    assert got.tolist() == want == [11, 12, 6, 12]
    assert np.array_equal(f64(k), k64) and np.array_equal(f64(v), v64)


def test_commit_looks_at_touched_slots_only(sv):
    """Blocks of one size: rows past the pages' end that the path leaves out do not matter."""
    k, v = caches(BF)
    ctx, acc, path = [9, 11, 2, 8], [1, 0, 2, 3], [[2, -1, -1, -1], [-1] * 4, [2, 4, -1, -1], [1, 2, 3, -1]]
    k64, v64 = f64(k), f64(v)
    want = [okv.commit(k64, v64, c, np.array(t), a, p) for c, t, a, p in zip(ctx, TABLE, acc, path)]
    st = sv.new_stats("cuda")
    got = sv.sv_kv_commit(k, v, i32(*ctx), i32(*TABLE), i32(*acc), i32(*path), stats=st)
    assert sv.read_stats(st)["status"] == 0 and got.tolist() == want
    assert np.array_equal(f64(k), k64) and np.array_equal(f64(v), v64)
    k, v = caches(BF)
    k0, v0 = k.clone(), v.clone()
    for c, a, p in ((9, 1, 3), (12, 0, 1), (2**31 - 3, 1, 4)):   # the path's slot, row 0's, and one past 32 bits
        st = sv.new_stats("cuda")
        got = sv.sv_kv_commit(k, v, i32(c, 0, 0, 0), i32(*TABLE), i32(a, 0, 0, 0), i32([p, -1, -1, -1], *[[-1] * 4] * 3), stats=st)
        assert sv.read_stats(st)["status"] == 1 and got.tolist() == [c, 1, 1, 1]
        assert torch.equal(k, k0) and torch.equal(v, v0)


def test_commit_ragged_reports(sv):
    """Paths and counts that do not fit the sequence's own block, and row starts that fall."""
    k, v = caches(BF)
    k0, v0 = k.clone(), v.clone()
    ctx = [3, 3, 3, 3]
    cases = [([0, 3, 3, 8, 9], [3, 0, 0, 0], [1, 2, 3, 4], 0),    # three rows hold two drafted tokens
             ([0, 3, 3, 8, 9], [1, 0, 0, 0], [3, -1, -1, -1], 0),   # node 3 of three rows
             ([0, 3, 3, 8, 9], [0, 1, 0, 0], [1, -1, -1, -1], 1),   # an empty block accepts nothing
             ([0, 5, 3, 8, 9], [0, 0, 0, 0], [-1] * 4, 1)]          # row starts that fall
    for starts, acc, path, who in cases:
        st = sv.new_stats("cuda")
        got = sv.sv_kv_commit(k, v, i32(*ctx), i32(*TABLE), i32(*acc), i32(*[path] * 4), row_start=i32(*starts), stats=st)
        s = sv.read_stats(st)
        assert s["status"] == 1 and s["error_index"] == who
        assert got.tolist()[who] == 3
        assert torch.equal(k, k0) and torch.equal(v, v0)
