"""The shapes of the tests of many tokens reach every tile, by the library's own rule (no
GPU is needed)."""
import os
import re
import shutil
import subprocess

import pytest

from mxfp4_block_amax_amd import build as fp4_build
from tests import _w4_tiles

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not found")
def test_shapes(tmp_path):
    exe = str(tmp_path / "linear_tiles")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror",
                    os.path.join(ROOT, "tests", "native", "linear_tiles.cpp"), "-o", exe], check=True)
    shapes = [str(v) for _, m, n in _w4_tiles.CASES for v in (m, n)]
    out = subprocess.run([exe, *shapes], check=True, capture_output=True, text=True).stdout
    assert [tuple(map(int, line.split())) for line in out.splitlines()] == \
        [tile for tile, _, _ in _w4_tiles.CASES]


def test_no_tile_is_missing():
    """Every tile that the rule may choose has shapes, and is launched."""
    def braces(name, pattern):
        with open(os.path.join(fp4_build.CSRC, name)) as f:
            return {tuple(map(int, t)) for t in re.findall(pattern, f.read())}
    rule = braces("fp4_linear.h", r"\{(\d+), (\d+), (?!8\})\d+\}")
    assert len(rule) == 5 and rule == set(_w4_tiles.TILES)
    assert braces("fp4_linear.hip", r"launch_wide<FMT, PACKED, (\d+), (\d+)>\(A, s\)") == rule
