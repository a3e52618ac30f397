"""A group's rows of partial column sums, counted on the CPU by the code that the kernel counts them with: where offsets
are in order against the definition, and inside the workspace where they are in no order at all."""

import os
import random
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "dense_fp32_gemm_sm_gb300", "csrc")
LOWEST, MOST_ROWS = -(2**31), 2**31 - 256


@pytest.fixture(scope="module")
def ranges(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("slices") / "gemm16_slices")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-fsanitize=signed-integer-overflow",
                        "-fsanitize-undefined-trap-on-error", "-I", CSRC, os.path.join(ROOT, "tests", "gemm16_slices.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(M, height, most, offsets):
        text = "%d %d %d %d\n%s\n" % (M, height, most, len(offsets) - 1, " ".join(map(str, offsets)))
        r = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=60)
        assert r.returncode == 0, r.stderr
        return [tuple(map(int, line.split())) for line in r.stdout.splitlines()]

    return run


@pytest.mark.parametrize("seed", range(6))
def test_in_order(ranges, seed):
    rng = random.Random(seed)
    groups, M, height = rng.choice([1, 7, 33, 1024]), rng.choice([1, 500, 100000, MOST_ROWS]), rng.choice([16, 24, 64])
    offsets = sorted(rng.randint(0, M) for _ in range(groups + 1))
    most, at = M // height + min(groups, M), 0
    got = ranges(M, height, most, offsets)
    assert len(got) == groups
    for e, (i, j) in enumerate(zip(offsets, offsets[1:])):
        end = at + -(-(j - i) // height)
        assert got[e] == (at, end) and end <= most
        at = end


@pytest.mark.parametrize("M", [1, 1000, (1 << 28) + 64, MOST_ROWS])
@pytest.mark.parametrize("pattern", ["alternating", "falling", "lowest and highest"])
def test_out_of_order(ranges, M, pattern):
    """1024 groups; with M in every other one, their slices come to 2^31 and more."""
    groups, height = 1024, 64
    offsets = {"alternating": [0, M] * 512 + [0], "falling": list(range(groups, -1, -1)),
               "lowest and highest": [LOWEST, 2**31 - 1] * 512 + [LOWEST]}[pattern]
    most = M // height + min(groups, M)
    for start, end in ranges(M, height, most, offsets):
        assert 0 <= start <= most and end <= most


def test_the_kernel_counts_with_this_code():
    with open(os.path.join(CSRC, "gemm16_rows.cu")) as f:
        code = f.read()
    kernel = code[code.index("sums_kernel(const float"):code.index("bool vectors(")]
    assert re.search(r"long long before = slices_before\(offsets, lane, 32, e, M, height\)", kernel)
    assert "rows = inside(before, before + slices_of(offsets, e, M, height), most)" in kernel
    assert "rows = inside(start[e], start[e + 1], most)" in kernel and "rows.from + warp; r < rows.to" in kernel
