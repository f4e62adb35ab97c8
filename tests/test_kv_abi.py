"""CPU tests of the target's side of a step: the host-only frequencies against the oracle, argument errors of every entry
point before any launch, and the binding's refusals."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import kv as okv


@pytest.fixture(scope="module")
def sv():
    from speculative_decoding_verification_gb300 import build
    build.build()
    import speculative_decoding_verification_gb300 as sv
    sv.load()
    return sv


@pytest.mark.parametrize("rotary", [2, 26, 64, 128, 256])
@pytest.mark.parametrize("scaling,kw", [("none", {}), ("linear", dict(factor=4.0)), ("base", dict(factor=8.0)),
                                        ("turns", dict(factor=8.0, low=1.0, high=4.0, original_len=8192)),
                                        ("dims", dict(factor=16.0, low=1.0, high=32.0, original_len=4096))])
def test_frequencies_match_the_oracle(sv, rotary, scaling, kw):
    if scaling == "base" and rotary < 4:
        with pytest.raises(sv.SvError):
            sv.sv_rope_frequencies(rotary, 10000.0, scaling, **kw)
        return
    f, mag = sv.sv_rope_frequencies(rotary, 500000.0, scaling, **kw)
    want, wmag = okv.rope_frequencies(rotary, 500000.0, scaling, **kw)
    np.testing.assert_allclose(f, want, rtol=2.0 ** -24 + 1e-13)
    assert mag == pytest.approx(wmag, rel=2.0 ** -23)


def test_scaled_frequencies_limits():
    """Fast pairs keep their frequency and slow ones are divided by the factor, in both blended forms."""
    plain, _ = okv.rope_frequencies(128)
    for scaling in ("turns", "dims"):
        f, _ = okv.rope_frequencies(128, 10000.0, scaling, 8.0, 1.0, 32.0, 4096)
        assert f[0] == plain[0] and f[-1] == pytest.approx(plain[-1] / 8.0, rel=1e-12)
        assert np.all(np.diff(f) < 0)


def test_frequencies_refuse(sv):
    for args in ((3,), (0,), (258,), (64, 1.0), (64, 0.5), (64, 1e4, "linear", 0.5), (64, 1e4, "linear", float("nan")),
                 (64, 1e4, "turns", 4.0, 4.0, 1.0, 100), (64, 1e4, "turns", 4.0, 1.0, 4.0, 0), (64, 1e4, "dims", 4.0, 0.0, 4.0, 100)):
        with pytest.raises(sv.SvError, match="invalid"):
            sv.sv_rope_frequencies(*args)
    with pytest.raises(ValueError, match="scaling"):
        sv.sv_rope_frequencies(64, scaling="cubic")


def test_rope_is_orthogonal_in_the_oracle():
    """The oracle's own check: the backward undoes the forward, and scores depend on position differences only."""
    rng = np.random.default_rng(0)
    f, _ = okv.rope_frequencies(8)
    x, y = rng.normal(size=(5, 1, 10)), rng.normal(size=(5, 1, 10))
    for style in ("half", "interleaved"):
        pos = np.arange(5)
        np.testing.assert_allclose(okv.rope(okv.rope(x, pos, f, style), pos, f, style, backward=True), x, atol=1e-14)
        a = (okv.rope(x, pos, f, style) * okv.rope(y, pos + 3, f, style)).sum(-1)
        b = (okv.rope(x, pos + 70, f, style) * okv.rope(y, pos + 73, f, style)).sum(-1)
        np.testing.assert_allclose(a, b, atol=1e-12)


FAKE = 1 << 20   # a 16-byte aligned non-null address, never dereferenced


def structs(sv, **kw):
    from speculative_decoding_verification_gb300._abi import SvKvBatch, SvKvCache
    d = dict(k=FAKE, v=FAKE, ps=16 * 2 * 64, ss=2 * 64, hs=64, pages=10, size=16, kv=2, dim=64, dtype=1, ctx=FAKE, table=FAKE, rs=None,
             par=None, pitch=5, mp=5, B=3, n=4, rows=12)
    d.update(kw)
    return (SvKvCache(d["k"], d["v"], d["ps"], d["ss"], d["hs"], d["pages"], d["size"], d["kv"], d["dim"], d["dtype"]),
            SvKvBatch(d["ctx"], d["table"], d["rs"], d["par"], d["pitch"], d["mp"], d["B"], d["n"], d["rows"]))


BAD_SHARED = [dict(k=None), dict(v=None), dict(k=FAKE + 8), dict(ps=4), dict(ss=3), dict(hs=1), dict(pages=0), dict(size=0), dict(kv=0),
              dict(dim=0), dict(dim=264), dict(dim=12), dict(dtype=7), dict(ctx=None), dict(table=None), dict(B=0), dict(n=0), dict(mp=0),
              dict(pitch=4), dict(mp=2**30, pitch=2**30, size=16)]
BAD_BLOCK = [dict(rows=11), dict(rows=-1), dict(rs=FAKE, par=FAKE), dict(par=FAKE, n=130, rows=390)]


def test_append_rejects_bad_arguments(sv):
    lib = sv.load()

    def call(q=FAKE, qo=FAKE, qh=4, k=FAKE, v=FAKE, qs=(256, 64), ks=(128, 64), inv=FAKE, rot=64, style=0, **kw):
        c, b = structs(sv, **kw)
        return lib.sv_kv_append(c, b, q, qs[0], qs[1], qo, 256, 64, qh, k, ks[0], ks[1], v, 128, 64, inv, rot, style, 1.0, None, None)
    for kw in BAD_SHARED + BAD_BLOCK + [dict(q=None), dict(qo=None), dict(qh=0), dict(k=None), dict(v=None), dict(k=FAKE + 2),
                                        dict(qs=(255, 64)), dict(ks=(128, 4)), dict(inv=None), dict(rot=63), dict(rot=66), dict(style=2)]:
        assert call(**kw) == 1, kw
    c, b = structs(sv)
    assert lib.sv_kv_append(None, b, None, 0, 0, None, 0, 0, 0, FAKE, 128, 64, FAKE, 128, 64, None, 0, 0, 1.0, None, None) == 1
    assert lib.sv_kv_append(c, None, None, 0, 0, None, 0, 0, 0, FAKE, 128, 64, FAKE, 128, 64, None, 0, 0, 1.0, None, None) == 1


def test_attend_rejects_bad_arguments(sv):
    lib = sv.load()
    ws = lib.sv_kv_attend_workspace_size(12, 4, 64, 3, 1)
    assert ws > 0 and lib.sv_kv_attend_workspace_size(-1, 4, 64, 3, 0) == 0 and lib.sv_kv_attend_workspace_size(12, 4, 300, 3, 0) == 0

    def call(q=FAKE, qh=4, scale=0.1, gs=FAKE, pl=FAKE, ng=1, out=FAKE, qs=(256, 64), ws_p=FAKE, wsb=ws, **kw):
        c, b = structs(sv, **kw)
        return lib.sv_kv_attend(c, b, q, qs[0], qs[1], qh, scale, gs, pl, ng, out, 256, 64, None, None, ws_p, wsb, None)
    for kw in BAD_SHARED + BAD_BLOCK + [dict(q=None), dict(out=None), dict(q=FAKE + 4), dict(qh=3), dict(qh=0), dict(scale=float("inf")),
                                        dict(scale=float("nan")), dict(gs=None), dict(pl=None), dict(ng=4), dict(ng=-1), dict(qs=(250, 64))]:
        assert call(**kw) == 1, kw
    assert call(ws_p=None) == 5 and call(wsb=ws - 1) == 5 and call(ws_p=FAKE + 16) == 5


def test_commit_and_rope_reject_bad_arguments(sv):
    lib = sv.load()

    def commit(layers=2, stride=64, acc=FAKE, path=FAKE, out=FAKE + 64, **kw):
        c, b = structs(sv, **kw)
        return lib.sv_kv_commit(c, b, layers, stride, acc, path, out, None, None)
    for kw in BAD_SHARED + [dict(layers=0), dict(stride=3), dict(acc=None), dict(path=None), dict(out=FAKE), dict(n=130)]:
        assert commit(**kw) == 1, kw

    def rope(x=FAKE, out=FAKE, dtype=1, rows=4, heads=2, dim=64, pos=FAKE, inv=FAKE, rot=64, style=0):
        return lib.sv_rope(x, 128, 64, out, 128, 64, dtype, rows, heads, dim, pos, inv, rot, style, 1.0, 0, None)
    for kw in (dict(x=None), dict(out=None), dict(dtype=5), dict(rows=-1), dict(heads=0), dict(dim=0), dict(pos=None), dict(inv=None),
               dict(rot=0), dict(rot=63), dict(rot=66), dict(style=-1), dict(dim=512, rot=258)):
        assert rope(**kw) == 1, kw
    assert rope(rows=0, x=None, out=None) == 0


def test_binding_refuses(sv):
    """Host tensors and mismatched shapes, dtypes and strides are refused before the library is called."""
    i32 = dict(dtype=torch.int32)
    x, cache, one = torch.zeros(2, 3, 4, 64), torch.zeros(5, 16, 2, 64), torch.zeros(2, **i32)
    table = torch.zeros(2, 3, **i32)
    for call in (lambda: sv.sv_rope(x, one, torch.ones(4)), lambda: sv.sv_kv_append(x, x, cache, cache, one, table),
                 lambda: sv.sv_kv_attend(x, cache, cache, one, table),
                 lambda: sv.sv_kv_commit(cache[None], cache[None], one, table, one, table)):
        with pytest.raises(TypeError, match="CUDA tensor"):
            call()
    with pytest.raises(ValueError, match="last axis"):
        sv._heads(x.transpose(2, 3), "q")
    with pytest.raises(ValueError, match="one stride"):
        sv._heads(torch.zeros(3, 4, 2, 64)[:, :3], "q")
    with pytest.raises(ValueError, match="expected"):
        sv._heads(x[0, 0], "q")
    assert sv._heads(torch.zeros(2, 3, 9, 64)[:, :, 2:6], "q") == (9 * 64, 64)
    assert sv._heads(torch.zeros(2, 1, 9, 64), "q") == (9 * 64, 64)
    with pytest.raises(ValueError, match="style"):
        sv._style("pairs")


def test_structs_match_the_header():
    """The binding's structures have the header's layout (sizes and the offset of every field)."""
    import os
    import subprocess
    import tempfile
    from speculative_decoding_verification_gb300._abi import SvKvBatch, SvKvCache
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    lines = ['#include <stdio.h>', '#include "specverify.h"', 'int main(void) {']
    want = []
    for cls, name in ((SvKvCache, "sv_kv_cache"), (SvKvBatch, "sv_kv_batch")):
        lines.append(f'printf("%zu ", sizeof({name}));')
        want.append(ctypes.sizeof(cls))
        for f, _ in cls._fields_:
            lines.append(f'printf("%zu ", offsetof({name}, {f}));')
            want.append(getattr(cls, f).offset)
    lines.append('return 0; }')
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "t.c"), os.path.join(d, "t")
        open(src, "w").write("\n".join(lines))
        subprocess.run(["gcc", "-I", os.path.join(root, "include"), src, "-o", exe], check=True)
        got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert got == want
