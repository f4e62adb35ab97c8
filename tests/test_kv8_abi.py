"""CPU tests of the cache held in 8 bits and of a cache's pages: the oracle's own checks, argument errors of every entry point before any
launch, and the binding's refusals."""
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


def test_the_oracles_grid_is_torchs():
    x = np.concatenate([np.linspace(-448, 448, 20001), 2.0 ** np.arange(-14, 9), [2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -10 * 1.001, 0.0]])
    want = torch.tensor(x, dtype=torch.float32).to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(okv.e4m3_grid(x.astype(np.float32)), want)
    assert np.isnan(okv.e4m3_grid([np.inf, -np.inf, np.nan])).all()


def test_the_oracles_scale_is_the_smallest():
    m = np.concatenate([448.0 * 2.0 ** np.arange(-60.0, 60), 448.0 * 2.0 ** np.arange(-60.0, 60) * (1 + 1e-9), np.geomspace(1e-30, 1e30, 999)])
    e = okv.scale_exponent(m)
    assert (m <= 448 * np.exp2(e)).all() and (m > 448 * np.exp2(e - 1)).all()
    assert okv.scale_exponent(0.0) == -120 and okv.scale_exponent(1e-60) == -120


def test_the_oracles_fork_counts_every_holder():
    rng = np.random.default_rng(0)
    for trial in range(200):
        size, B, N = int(rng.integers(1, 6)), int(rng.integers(1, 6)), int(rng.integers(1, 9))
        ctx = rng.integers(0, 20, B)
        width = 40 // size + 4
        table, ids = np.full((B, width), -1), list(rng.permutation(400))
        for b in range(B):
            took = -(-int(ctx[b]) // size)
            table[b, :took] = [ids.pop() for _ in range(took)]
        refs = np.zeros(400, int)
        np.add.at(refs, table[table >= 0], 1)
        src, reserve = rng.integers(-1, B, N), int(rng.integers(0, 9))
        rows, c, after, copies = okv.fork(refs, ctx, table, src, reserve, size)
        rows = np.array(rows)
        count = np.zeros(400, int)
        np.add.at(count, rows[rows >= 0], 1)
        assert (count == after).all()
        part = {(j, rows[j][c[j] // size]) for j in range(N) if src[j] >= 0 and c[j] % size}
        assert len({p for _, p in part}) == len(part)   # nobody shares the page it will write
        assert len({t for _, t, _ in copies}) == len(copies)


FAKE = 1 << 20   # a 16-byte aligned non-null address, never dereferenced


def structs(**kw):
    from speculative_decoding_verification_gb300._abi import SvKvBatch, SvKvCache8
    d = dict(k=FAKE, v=FAKE, ks=FAKE + 1, vs=FAKE + 3, ps=16 * 2 * 64, ss=2 * 64, hs=64, sps=3, shs=1, pages=10, size=16, kv=2, dim=64, ctx=FAKE,
             table=FAKE, rs=None, par=None, pitch=5, mp=5, B=3, n=4, rows=12)
    d.update(kw)
    return (SvKvCache8(d["k"], d["v"], d["ks"], d["vs"], d["ps"], d["ss"], d["hs"], d["sps"], d["shs"], d["pages"], d["size"], d["kv"], d["dim"]),
            SvKvBatch(d["ctx"], d["table"], d["rs"], d["par"], d["pitch"], d["mp"], d["B"], d["n"], d["rows"]))


BAD_SHARED = [dict(k=None), dict(v=None), dict(ks=None), dict(vs=None), dict(k=FAKE + 8), dict(ps=4), dict(ss=24), dict(hs=8), dict(pages=0),
              dict(size=0), dict(kv=0), dict(dim=0), dict(dim=272), dict(dim=24), dict(ctx=None), dict(table=None), dict(B=0), dict(n=0),
              dict(mp=0), dict(pitch=4), dict(mp=2**30, pitch=2**30, size=16)]
BAD_BLOCK = [dict(rows=11), dict(rows=-1), dict(rs=FAKE, par=FAKE), dict(par=FAKE, n=130, rows=390)]


def test_append8_rejects_bad_arguments(sv):
    lib = sv.load()

    def call(dt=1, q=FAKE, qo=FAKE, qh=4, k=FAKE, v=FAKE, qs=(256, 64), ks_=(128, 64), inv=FAKE, rot=64, style=0, **kw):
        c, b = structs(**kw)
        return lib.sv_kv_append8(c, b, dt, q, qs[0], qs[1], qo, 256, 64, qh, k, ks_[0], ks_[1], v, 128, 64, inv, rot, style, 1.0, None, None)
    for kw in BAD_SHARED + BAD_BLOCK + [dict(q=None), dict(qo=None), dict(qh=0), dict(k=None), dict(v=None), dict(dt=2), dict(dt=7), dict(inv=None),
                                        dict(rot=63), dict(rot=66), dict(rot=-2), dict(style=2), dict(qs=(257, 64)), dict(ks_=(128, 9)),
                                        dict(q=FAKE + 4), dict(k=FAKE + 2), dict(qo=FAKE + 16)]:
        assert call(**kw) == 1, kw
    assert lib.sv_kv_append8(None, None, 1, None, 0, 0, None, 0, 0, 0, None, 0, 0, None, 0, 0, None, 0, 0, 1.0, None, None) == 1


def test_attend8_rejects_bad_arguments(sv):
    lib = sv.load()
    ws = lib.sv_kv_attend_workspace_size(12, 4, 64, 3, 0)

    def call(dt=1, q=FAKE, out=2 * FAKE, qh=4, qs=(256, 64), os=(256, 64), scale=0.1, gs=None, pl=None, g=0, w=FAKE, wb=ws, **kw):
        c, b = structs(**kw)
        return lib.sv_kv_attend8(c, b, dt, q, qs[0], qs[1], qh, scale, gs, pl, g, out, os[0], os[1], None, None, w, wb, None)
    for kw in BAD_SHARED + BAD_BLOCK + [dict(q=None), dict(out=None), dict(qh=3), dict(qh=0), dict(dt=2), dict(dt=-1), dict(scale=float("nan")),
                                        dict(scale=float("inf")), dict(g=1), dict(g=4, gs=FAKE, pl=FAKE), dict(g=-1), dict(qs=(4, 64)),
                                        dict(os=(256, 3)), dict(out=FAKE), dict(out=FAKE + 128)]:
        assert call(**kw) == 1, kw
    assert call(w=None) == 5 and call(w=FAKE + 16) == 5 and call(wb=ws - 1) == 5


def test_commit8_rejects_bad_arguments(sv):
    lib = sv.load()

    def call(layers=2, ls=4096, sls=7, acc=FAKE, path=FAKE, out=None, **kw):
        c, b = structs(**kw)
        return lib.sv_kv_commit8(c, b, layers, ls, sls, acc, path, out, None, None)
    for kw in BAD_SHARED + [dict(layers=0), dict(ls=8), dict(acc=None), dict(path=None), dict(out=FAKE), dict(n=130), dict(layers=2**31 - 1)]:
        assert call(**kw) == 1, kw


def pool(**kw):
    from speculative_decoding_verification_gb300._abi import SvKvPool
    d = dict(k=FAKE, v=2 * FAKE, ks=None, vs=None, ls=1 << 16, ps=4096, ss=256, hs=128, hb=128, sls=0, sps=0, shs=0, layers=2, pages=10, size=16, kv=2)
    d.update(kw)
    return SvKvPool(*(d[x] for x in ("k", "v", "ks", "vs", "ls", "ps", "ss", "hs", "hb", "sls", "sps", "shs", "layers", "pages", "size", "kv")))


BAD_POOL = [dict(k=None), dict(v=None), dict(ks=FAKE), dict(vs=FAKE), dict(k=FAKE + 4), dict(ls=8), dict(ps=24), dict(ss=4), dict(hs=2), dict(hb=0),
            dict(hb=24), dict(hb=2048), dict(layers=0), dict(pages=0), dict(size=0), dict(kv=0), dict(size=2**20, kv=2**12), dict(pages=2**30 + 1)]


def test_fork_rejects_bad_arguments(sv):
    lib = sv.load()
    R, C, T, S, RO, TO, CO = (FAKE * i for i in range(1, 8))

    def call(refs=R, ctx=C, table=T, pitch=5, mp=5, B=3, src=S, N=4, reserve=2, ro=RO, to=TO, top=5, co=CO, w=FAKE, wb=None, **kw):
        wb = lib.sv_kv_fork_workspace_size(10, min(max(N, 1), 2**30)) if wb is None else wb
        return lib.sv_kv_fork(pool(**kw), refs, ctx, table, pitch, mp, B, src, N, reserve, ro, to, top, co, None, w, wb, None)
    for kw in BAD_POOL + [dict(refs=None), dict(ctx=None), dict(table=None), dict(src=None), dict(ro=None), dict(to=None), dict(co=None), dict(B=0),
                          dict(N=0), dict(mp=0), dict(pitch=4), dict(top=4), dict(reserve=-1), dict(mp=2**29, pitch=2**29, top=2**29),
                          dict(to=T), dict(to=T + 8), dict(co=C), dict(co=S + 4), dict(ro=R + 4), dict(to=RO), dict(ro=T), dict(co=TO + 16),
                          dict(N=2**30), dict(to=R), dict(N=2**30 + 1, mp=1, B=1, layers=1)]:
        assert call(**kw) == 1, kw
    assert call(w=None) == 5 and call(w=FAKE + 16) == 5 and call(wb=100) == 5
    assert lib.sv_kv_fork_workspace_size(0, 4) == 0 and lib.sv_kv_fork_workspace_size(4, 0) == 0


def test_compact_rejects_bad_arguments(sv):
    lib = sv.load()
    R, T, RO, TO, M, L = (FAKE * i for i in range(1, 7))

    def call(refs=R, table=T, pitch=5, mp=5, B=3, ro=RO, to=TO, top=5, moved=M, live=L, w=FAKE, wb=None, **kw):
        wb = lib.sv_kv_compact_workspace_size(10) if wb is None else wb
        return lib.sv_kv_compact(pool(**kw), refs, table, pitch, mp, B, ro, to, top, moved, live, None, w, wb, None)
    for kw in BAD_POOL + [dict(refs=None), dict(ro=None), dict(live=None), dict(table=None), dict(to=None), dict(B=-1), dict(mp=0), dict(pitch=4),
                          dict(top=4), dict(ro=R + 4), dict(to=T + 4), dict(to=T, top=6), dict(moved=R), dict(moved=RO), dict(live=T + 4),
                          dict(live=M + 8), dict(to=R)]:
        assert call(**kw) == 1, kw
    assert call(w=None) == 5 and call(wb=100) == 5 and lib.sv_kv_compact_workspace_size(0) == 0


def test_structure_layouts(sv):
    from speculative_decoding_verification_gb300 import _abi
    assert _abi.KV_CACHE8.size == ctypes.sizeof(_abi.SvKvCache8) and _abi.KV_POOL.size == ctypes.sizeof(_abi.SvKvPool)
    args = list(range(1, 14))
    assert _abi.KV_CACHE8.pack(*args) == bytes(_abi.SvKvCache8(*args))
    args = list(range(1, 17))
    assert _abi.KV_POOL.pack(*args) == bytes(_abi.SvKvPool(*args))
    assert sv.status_string(_abi.SV_ERR_NO_PAGE) == "no free page left in the pool"


def test_binding_refuses_host_tensors(sv):
    x = torch.zeros((1, 2, 2, 64))
    c, s, i = torch.zeros((4, 16, 2, 64)).to(torch.float8_e4m3fn), torch.zeros((4, 2), dtype=torch.uint8), torch.zeros(1, dtype=torch.int32)
    t = i.view(1, 1)
    for call in (lambda: sv.sv_kv_append8(x, x, c, c, s, s, i, t), lambda: sv.sv_kv_attend8(x, c, c, s, s, i, t),
                 lambda: sv.sv_kv_commit8(c[None], c[None], s[None], s[None], i, t, i, t), lambda: sv.sv_kv_fork(c[None], c[None], i, i, t, i),
                 lambda: sv.sv_kv_compact(c[None], c[None], i, t)):
        with pytest.raises(TypeError, match="CUDA"):
            call()


@pytest.mark.gpu
def test_binding_refuses(sv):
    """Wrong types, shapes and places, before any work is queued."""
    F8 = torch.float8_e4m3fn
    c, s = torch.zeros((4, 16, 2, 64), dtype=torch.uint8).cuda().view(F8), torch.zeros((4, 2), dtype=torch.uint8).cuda()
    x, i = torch.zeros((1, 2, 2, 64)).cuda(), torch.zeros(1, dtype=torch.int32).cuda()
    t = i.view(1, 1)
    bad = [(TypeError, (x, x, c.view(torch.uint8), c.view(torch.uint8), s, s, i, t)), (TypeError, (x, x, c, c, s.float(), s.float(), i, t)),
           (TypeError, (x, x, c, c, s, s.view(torch.float8_e8m0fnu), i, t)), (ValueError, (x, x, c, c, s[:3], s[:3], i, t)),
           (ValueError, (x, x, c, c, s, s.t().contiguous().t(), i, t)), (ValueError, (x, x, c, c, s.cpu(), s, i, t)),
           (ValueError, (x, x.transpose(2, 3), c, c, s, s, i, t)), (TypeError, (x, x.bfloat16(), c, c, s, s, i, t)),
           (TypeError, (x.half(), x.half(), c, c, s, s, i, t)), (ValueError, (x.cpu(), x.cpu(), c, c, s, s, i, t))]
    for err, args in bad:
        with pytest.raises(err):
            sv.sv_kv_append8(*args)
        with pytest.raises((TypeError, ValueError)):
            sv.sv_kv_attend8(*args[1:]) if args[1].dtype is not torch.bfloat16 else sv.sv_kv_attend8(x.half(), *args[2:])
    r = torch.zeros(4, dtype=torch.int32).cuda()
    with pytest.raises(ValueError, match="scales"):
        sv.sv_kv_fork(c[None], c[None], r, i, t, i)
    with pytest.raises(ValueError, match="together"):
        sv.sv_kv_fork(c[None], c[None], r, i, t, i, k_scale=s[None])
    with pytest.raises(ValueError, match="holds"):
        sv.sv_kv_fork(c[None], c[None], r[:3], i, t, i, k_scale=s[None], v_scale=s[None])
    with pytest.raises(ValueError, match="table_out"):
        sv.sv_kv_fork(c[None], c[None], r, i, t, i, k_scale=s[None], v_scale=s[None], table_out=torch.zeros((1, 2), dtype=torch.int32).cuda())
    with pytest.raises(sv.SvError, match="invalid"):
        sv.sv_kv_fork(c[None], c[None], r, i, t, i, k_scale=s[None], v_scale=s[None], table_out=t)
    with pytest.raises(ValueError, match="table_out"):
        sv.sv_kv_compact(c[None], c[None], r, k_scale=s[None], v_scale=s[None], table_out=t)
