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
