"""CPU test of how attention's work is cut into ranges of blocks: the functions that the kernels walk with, compiled for the host, over
random batches and over contexts whose costs pass 32 bits."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_ranges_cover_every_tile_once(tmp_path):
    from speculative_decoding_verification_gb300 import build
    exe = str(tmp_path / "kv_ranges")
    cmd = [build._nvcc(), *build.ARCH, "-std=c++17", "-O1", "-I", build.INCLUDE, "-I", build.CSRC,
           os.path.join(ROOT, "tests", "kv_ranges.cu"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    out = subprocess.run([exe, "400"], capture_output=True, text=True).stdout.split()
    assert out[:2] == ["ok", "400"], out
    assert int(out[2]) > 1 << 32   # costs past 32 bits were among them
