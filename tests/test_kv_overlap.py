"""Outputs that overlap inputs are refused, those that only interleave with them are not."""
import itertools
import os
import subprocess

import numpy as np
import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def sv():
    from speculative_decoding_verification_gb300 import build
    build.build()
    import speculative_decoding_verification_gb300 as sv
    sv.load()
    return sv


def places(at, row, head, rows, heads, width):
    """Byte addresses of [rows][heads][width], in steps of 16."""
    return set((at + np.arange(rows)[:, None, None] * row + np.arange(heads)[:, None] * head + np.arange(0, width, 16)).ravel().tolist())


def test_overlap_is_exact(tmp_path):
    """The library's answer, compiled for the host, against the sets of bytes: bases, strides, orders of the axes, single rows and heads."""
    from speculative_decoding_verification_gb300 import build
    src, exe = tmp_path / "t.cu", tmp_path / "t"
    src.write_text('''#include <stdio.h>
#include "sv_kv.cuh"
int main() {
    long long a[11];
    while (scanf("%lld %lld %lld %lld %lld %lld %lld %lld %lld %lld", a, a + 1, a + 2, a + 3, a + 4, a + 5, a + 6, a + 7, a + 8, a + 9) == 10) {
        const sv::RowsView x{(const void *)(intptr_t)1048576, a[0], a[1], a[2], a[3], a[4]};
        const sv::RowsView y{(const void *)(intptr_t)(1048576 + a[5]), a[6], a[7], a[8], a[9], a[4]};
        putchar(sv::overlap(x, y) ? '1' : '0');
    }
}
''')
    r = subprocess.run([build._nvcc(), *build.ARCH, "-std=c++17", "-I", build.INCLUDE, "-I", build.CSRC, str(src), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    heads, width = 4, 32
    layouts = [(heads * width, width), (2 * heads * width, width), (width, 64 * width), (6 * width, width), (0, width), (48, 32), (-128, 32),
               (heads * 2 * width, 2 * width), (16, 16), (1000 * width, 16)]
    lines, want = [], []
    for (ra, rb), ha, (ar, ah), (br, bh) in itertools.product([(1, 1), (3, 3), (1, 3), (5, 2)], (1, heads), layouts, layouts):
        if min(ra, rb) > 1 and ar != br:   # of these only those with one base are told
            continue
        for off in (-640, -400, -272, -128, -32, -16, 0, 16, 32, 64, 112, 128, 256, 272, 400, 512, 8192):
            lines.append(f"{ar} {ah} {ra} {ha} {width} {off} {br} {bh} {rb} {heads}")
            want.append(bool(places(0, ar, ah, ra, ha, width) & places(off, br, bh, rb, heads, width)))
    lines += ["128 32 3 4 32 0 256 32 3 4", "128 32 0 4 32 0 128 32 0 4"]
    want += [True, False]
    many = 1 << 28   # heads: the answer may not take long
    lines += [f"0 32 1 {many} 32 {32 * many - 32} 0 32 1 {many}", f"0 32 1 {many} 32 {32 * many} 0 32 1 {many}",
              f"0 64 1 {many} 32 32 0 64 1 {many}", f"0 64 1 {many} 32 64 0 32 1 {many}"]
    want += [True, False, False, False]
    got = subprocess.run([str(exe)], input="\n".join(lines), capture_output=True, text=True).stdout
    assert len(got) == len(want)
    wrong = [(x, w) for x, g, w in zip(lines, got, want) if (g == "1") != w]
    assert not wrong, (len(wrong), wrong[:5])
    assert 0.1 < sum(want) / len(want) < 0.9


@pytest.mark.gpu
def test_binding_refuses_overlap(sv):
    q = torch.randn(2, 3, 4, 64, device="cuda")
    wide = torch.randn(2, 3, 8, 64, device="cuda")
    k = torch.randn(9, 16, 2, 64, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    args = (k, k.clone(), torch.tensor([5, 9], **i32), torch.arange(4, **i32).reshape(2, 2))
    for out in (q, wide[:, :, 1:5]):
        x = q if out is q else wide[:, :, :4]
        with pytest.raises(sv.SvError, match="invalid"):
            sv.sv_kv_attend(x, *args, out=out)
    beside, _ = sv.sv_kv_attend(wide[:, :, :4], *args, out=wide[:, :, 4:])
    alone, _ = sv.sv_kv_attend(wide[:, :, :4].contiguous(), *args)
    assert torch.equal(beside, alone)
    # rotations: in place is fine, onto rows that are still read is not
    inv, pos = torch.ones(16, device="cuda"), torch.arange(6, **i32)
    with pytest.raises(sv.SvError, match="invalid"):
        sv.sv_rope(wide[:, :, :4], pos, inv, out=wide[:, :, 1:5])
    flat = torch.randn(7, 4, 64, device="cuda")
    with pytest.raises(sv.SvError, match="invalid"):
        sv.sv_rope(flat[:6], pos, inv, out=flat[1:])
    want = sv.sv_rope(wide[:, :, :4].contiguous(), pos, inv)
    assert torch.equal(sv.sv_rope(wide[:, :, :4], pos, inv, out=wide[:, :, 4:]), want)
    assert torch.equal(sv.sv_rope(wide[:, :, :4], pos, inv, out=wide[:, :, :4]), want)
    kv = torch.randn(2, 3, 2, 64, device="cuda")
    with pytest.raises(sv.SvError, match="invalid"):
        sv.sv_kv_append(kv, kv, k, k.clone(), *args[2:], q=wide[:, :, :4], q_out=wide[:, :, 2:6])
    sv.sv_kv_append(kv, kv, k, k.clone(), *args[2:], q=wide[:, :, :4], q_out=wide[:, :, :4])
