"""CPU check of the grouped products' grid and tile numbering (no GPU):
tests/host/grouped_ranges.cpp, built with g++ under AddressSanitizer and
UndefinedBehaviorSanitizer against the header that the kernels use."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_grid_and_tiles(tmp_path):
    exe = str(tmp_path / "grouped_ranges")
    cmd = ["g++", "-std=c++17", "-O2", "-g", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-I" + ROOT,
           os.path.join(ROOT, "tests", "host", "grouped_ranges.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:verify_asan_link_order=0")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=280, env=env)
    assert r.returncode == 0, (r.stdout + r.stderr)[-3000:]
    assert "grouped ranges ok" in r.stdout
