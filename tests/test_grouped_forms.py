"""CPU check of the grouped products' plan at the limits of the entry point
(tests/host/grouped_limits.cpp, built with g++ under AddressSanitizer and
UndefinedBehaviorSanitizer against the header that the kernels use), and that the sizes
which the GPU tests run reach every tile."""
import os
import shutil
import subprocess

import pytest

import grouped_cases as C

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("grouped") / "grouped_limits")
    cmd = ["g++", "-std=c++17", "-O2", "-g", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-I" + ROOT,
           os.path.join(ROOT, "tests", "host", "grouped_limits.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    return exe


def run(*cmd, text=None):
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:verify_asan_link_order=0")
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=280, env=env, input=text)
    assert r.returncode == 0, (r.stdout + r.stderr)[-3000:]
    return r.stdout


def test_limits(program):
    assert "grouped limits ok" in run(program)


def test_the_gpu_tests_reach_every_tile(program):
    cases, lines = list(C.all_cases()), ""
    for kind, tile, K, gated, _ in cases:
        sizes, N, Ng = C.TILES[tile]
        code = ["bf16", "fp16", "row", "mx"].index(kind)
        lines += f"{sum(sizes)} {len(sizes)} {Ng if gated else N} {K * (2 if code < 2 else 1)} {code} {int(gated)}\n"
    for case, tile in zip(cases, run(program, "plan", text=lines).split()):
        assert int(tile) == case[1], f"{case}: the plan takes tiles of {tile} rows"
    for tile, (sizes, _, _) in C.TILES.items():
        last = {(n - 1) % tile + 1 for n in sizes if n}
        assert tile in last and 1 in last and any(tile // 2 < n < tile for n in last)
        assert tile == 64 or any(n <= tile // 4 for n in last) and any(tile // 4 < n <= tile // 2 for n in last)
