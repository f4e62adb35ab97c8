"""CPU tests of the sizes that the cache calls refuse.  An accepted call without a workspace answers SV_ERR_WORKSPACE before any device
is looked for, so the two are told apart without one."""
import pytest

from test_kv_abi import FAKE, structs

INVALID, WORKSPACE = 1, 5


@pytest.fixture(scope="module")
def sv():
    from speculative_decoding_verification_gb300 import build
    build.build()
    import speculative_decoding_verification_gb300 as sv
    sv.load()
    return sv


def attend(sv, q_heads=4, groups=0, **kw):
    c, b = structs(sv, **kw)
    return sv.load().sv_kv_attend(c, b, FAKE, 256, 64, q_heads, 0.1, FAKE, FAKE, groups, FAKE, 256, 64, None, None, None, 0, None)


@pytest.mark.parametrize("page", [1, 16, 1000])
def test_slots_of_a_page_table(sv, page):
    """Places a few tiles past a table's last slot still fit 32 bits; tables with more are refused."""
    most = (2**31 - 1 - 1024) // page
    assert attend(sv, size=page, mp=most, pitch=most) == WORKSPACE
    assert attend(sv, size=page, mp=most + 1, pitch=most + 1) == INVALID


def test_rows_that_meet_the_same_tokens(sv):
    """A key head's cost within a block or a prefix is kept below 2^31: rows times tokens past that are refused, whole batches are not."""
    big = dict(size=1 << 16, B=1, n=1 << 20, rows=1 << 20, kv=1)
    assert attend(sv, 8, mp=32, pitch=32, **big) == WORKSPACE            # a million rows of 8 heads over two million tokens
    assert attend(sv, 8, mp=64, pitch=64, **big) == INVALID
    many = dict(size=1 << 16, mp=64, pitch=64, B=1 << 14, n=64, rows=1 << 20, kv=1)
    assert attend(sv, 8, **many) == WORKSPACE                            # the same rows in blocks of 64
    assert attend(sv, 8, groups=1, **many) == INVALID                    # but not over one prefix
    few = dict(size=1 << 16, mp=30000, pitch=30000, B=1 << 14, n=4, rows=1 << 16, kv=1)
    assert attend(sv, 8, **few) == WORKSPACE
    assert attend(sv, 1 << 15, n=2, rows=1 << 15, B=1 << 14, kv=1) == WORKSPACE   # rows * q_heads = 2^30
    assert attend(sv, 1 << 15, n=3, rows=3 << 14, B=1 << 14, kv=1) == INVALID


def test_parents_of_another_block_size(sv):
    """parents [B, m] of trees with other numbers of rows than the block's would be read with the wrong row length."""
    import types

    import torch
    host, i32 = types.SimpleNamespace(index=-1), dict(dtype=torch.int32)
    ctx, table = torch.zeros(3, **i32), torch.zeros(3, 5, **i32)

    def batch(*shape):
        return sv._kv_batch(host, ctx, table, (3, 4, 8, 64), None, torch.zeros(shape, **i32), None)
    for shape in ((3, 3), (5, 3), (9,), (20,)):   # as many trees or more; flat arrays hold at least the elements
        assert batch(*shape)[:2] == (3, 12)
    for shape in ((3, 4), (3, 2), (9, 1), (12, 4)):
        with pytest.raises(ValueError, match="parents must be"):
            batch(*shape)


def test_packed_structures(sv):
    """The bytes that the binding passes are those of the structures."""
    import ctypes

    from speculative_decoding_verification_gb300._abi import KV_BATCH, KV_CACHE, SvKvBatch, SvKvCache
    cache = (1 << 40, 3 << 41, 5 << 33, 7 << 32, -9, 11, 13, 17, 19, 1)
    batch = (1 << 40, 3 << 41, 5 << 42, 7 << 43, 9 << 33, 11, 13, 17, 2**31 - 1)
    for packed, cls, values in ((KV_CACHE, SvKvCache, cache), (KV_BATCH, SvKvBatch, batch)):
        assert packed.size == ctypes.sizeof(cls)
        assert packed.pack(*values) == bytes(cls(*values))
