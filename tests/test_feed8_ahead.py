"""CPU test of the look-ahead of attention over codes in page tables whose slots end near 2^31, with the kernel's own function."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_places_ahead_stay_within_the_table(tmp_path):
    from speculative_decoding_verification_gb300 import build
    exe = str(tmp_path / "feed8_ahead")
    cmd = [build._nvcc(), *build.ARCH, "-std=c++17", "-O1", "-I", build.INCLUDE, "-I", build.CSRC,
           os.path.join(ROOT, "tests", "feed8_ahead.cu"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    out = subprocess.run([exe], capture_output=True, text=True).stdout.split()
    assert out[:1] == ["ok"] and int(out[1]) > 1000000, out
    assert int(out[2]) > 0   # lanes whose own offset passes 32 bits were among them
