"""CPU check of the linear operator with 4-bit weights: its plans, work split and
addresses (tests/host/linear4_ranges.cpp, built with g++ under AddressSanitizer and
UndefinedBehaviorSanitizer against the header that the kernels use), and that the sizes
which the GPU tests run reach every kernel."""
import os
import shutil
import subprocess

import pytest

import linear4_cases as C

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("linear4") / "linear4_ranges")
    cmd = ["g++", "-std=c++17", "-O2", "-g", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-I" + ROOT,
           os.path.join(ROOT, "tests", "host", "linear4_ranges.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    return exe


def run(*cmd, text=None):
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:verify_asan_link_order=0")
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=280, env=env, input=text)
    assert r.returncode == 0, (r.stdout + r.stderr)[-3000:]
    return r.stdout


def test_work_split_and_addresses(program):
    assert "linear4 ranges ok" in run(program)


def test_the_gpu_tests_reach_every_kernel(program):
    cases = list(C.all_cases())
    lines = "".join(f"{M} {N} {K} {int(dtype == 'fp16')} {int(scales == 'mx')} {int(gated)}\n"
                    for scales, dtype, _, _, _, M, N, K, gated in cases)
    plans = run(program, "plan", text=lines).splitlines()
    assert len(plans) == len(cases)
    seen = set()
    for c, line in zip(cases, plans):
        form, fm, whole, left = line.split()
        whole, left = int(whole), int(left)
        how = "" if form != "tile" else "both" if whole and left else "whole" if whole else "cut"
        assert (form, int(fm), how) == c[2:5], f"{c}: the plan takes {line}"
        seen.add((c[:2], form, int(fm), how, c[8]))
    for pair in C.PAIRS:
        for gated in (False, True):
            want = {("tile", fm, how) for fm in (1, 2, 4, 8) for how in ("whole", "cut", "both")} | {("wide", 0, ""), ("few", 0, "")}
            assert want <= {s[1:4] for s in seen if s[0] == pair and s[4] == gated}
