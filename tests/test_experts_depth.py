"""How many loads the decode kernel of the routed rows has on their way, asked
on the host."""

import ctypes
import os
import subprocess

import pytest

from bitlinear_w1_a8_amd import build

# rows of every depth (2, 4, 6, 8, 10 chunks of 256; longer ones take 10), with
# K a multiple of 64 and not, and one shorter than 64
ROWS = [48, 448, 400, 960, 1008, 1216, 1264, 1472, 1520, 1984, 1840, 2240, 2480, 2816, 2704, 5184, 5200]


@pytest.fixture(scope="module")
def depth(tmp_path_factory):
    folder = str(tmp_path_factory.mktemp("depth"))
    src, lib = os.path.join(folder, "depth.cpp"), os.path.join(folder, "depth.so")
    with open(src, "w") as f:
        f.write('#include "experts_plan.h"\nextern "C" int depth(int64_t k) { return bl::few_depth(k); }\n')
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", build.CSRC, src, "-o", lib], check=True)
    fn = ctypes.CDLL(lib).depth
    fn.argtypes = [ctypes.c_int64]
    return fn


def test_depth_follows_the_row(depth):
    """No row loads more than one chunk that it does not have, and none of up to
    ten chunks waits for a later load."""
    for k in range(16, 131072 + 1, 16):
        chunks = -(-k // 256)
        assert min(chunks, 10) <= depth(k) <= min(chunks + 1, 10) and depth(k) % 2 == 0


def test_rows_of_every_depth(depth):
    for whole in (True, False):
        assert {depth(k) for k in ROWS if (k % 64 == 0) == whole and k > 64} == {2, 4, 6, 8, 10}
