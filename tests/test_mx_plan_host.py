"""Which kernel the sizes of test_gpu_mxfp4_tiles.py reach, by the library's own rule: a
rule that changes must not leave a kernel without its tests (no GPU)."""
import os
import shutil
import subprocess

import pytest

from test_gpu_mxfp4_tiles import LARGE, PIECES, SMALL

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_sizes_reach_the_kernels_they_are_for(tmp_path):
    exe = str(tmp_path / "mx_plan_print")
    subprocess.run(["g++", "-std=c++17", "-o", exe, os.path.join(HERE, "csrc", "mx_plan_print.cpp")], check=True)

    def plans(sizes):
        out = subprocess.run([exe] + [str(n) for s in sizes for n in s], capture_output=True, text=True, check=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]
    assert plans(LARGE) == [(256, 1)] * len(LARGE)
    assert plans(SMALL) == [(128, 1)] * len(SMALL)
    assert all(tile == 128 and pieces > 1 for tile, pieces in plans(PIECES))
    # rows and columns past the last whole tile, one group of 1024 k and more, rows of
    # scales that have to be padded and that have not
    for sizes in (LARGE, SMALL, PIECES):
        assert all(any(f(*s) for s in sizes) for f in (
            lambda m, n, k: m % 256 and n % 256, lambda m, n, k: k > 1024 * (1 + (sizes is not SMALL)), lambda m, n, k: k % 1024 and k % 128,
            lambda m, n, k: k % 128 == 0))
