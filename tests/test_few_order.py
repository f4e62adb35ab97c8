"""CPU test of the order of products in the few-row attention kernel over codes, with the kernel's own rule compiled for the host."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_no_scores_over_ones_still_read(tmp_path):
    from speculative_decoding_verification_gb300 import build
    exe = str(tmp_path / "few_order")
    cmd = [build._nvcc(), *build.ARCH, "-std=c++17", "-O1", "-I", build.INCLUDE, "-I", build.CSRC,
           os.path.join(ROOT, "tests", "few_order.cu"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    out = subprocess.run([exe], capture_output=True, text=True).stdout.split()
    assert out[:1] == ["ok"] and int(out[2]) > 1000000, out
