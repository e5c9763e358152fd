"""Where the join of shared prefixes looks for parts (csrc/ops/mk_ops_parts.h),
on the host: inside the workspace whatever numbers it finds there."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
OPS = os.path.join(HERE, "..", "moe_decode_megakernel_gb300", "csrc", "ops")

SHIM = """
#include "mk_ops_parts.h"
extern "C" int parts(int32_t first, int32_t last, int grid) { return mk::ops::parts_of({first, last}, grid); }
extern "C" int64_t slot(int32_t first, int32_t last, int k) { return mk::ops::part_slot({first, last}, k); }
"""


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    where = tmp_path_factory.mktemp("parts")
    src, lib = where / "shim.cpp", where / "shim.so"
    src.write_text(SHIM)
    subprocess.run([gxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", OPS, str(src), "-o", str(lib)], check=True)
    L = ctypes.CDLL(str(lib))
    L.parts.argtypes, L.parts.restype = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int], ctypes.c_int
    L.slot.argtypes, L.slot.restype = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int], ctypes.c_int64
    return L


@pytest.mark.parametrize("grid", [1, 2, 148, 152, 160])
def test_places_of_ctas_are_all_there(shim, grid):
    for first in range(grid):
        for last in range(first, grid):
            n = shim.parts(first, last, grid)
            assert n == last - first + 1
            slots = [shim.slot(first, last, k) for k in range(n)]
            # the first CTA's last slot, the others' first ones: each its own
            assert slots == [2 * first + 1] + [2 * c for c in range(first + 1, last + 1)]


EDGE = [0, 1, -1, 147, 148, 149, 151, 152, 160, 1 << 16, (1 << 31) - 1, -(1 << 31), 0x7fc00000 - (1 << 31), 0x3f800000]


@pytest.mark.parametrize("grid", [1, 148, 152, 160])
def test_places_that_were_never_written_lie_inside(shim, grid):
    r = random.Random(grid)
    pairs = [(a, b) for a in EDGE for b in EDGE]
    pairs += [(r.randrange(-(1 << 31), 1 << 31), r.randrange(-(1 << 31), 1 << 31)) for _ in range(2000)]
    pairs += [(r.randrange(-3, grid + 3), r.randrange(-3, grid + 3)) for _ in range(2000)]
    for first, last in pairs:
        n = shim.parts(first, last, grid)
        assert 0 <= n <= grid
        assert (n > 0) == (0 <= first <= last < grid)
        assert all(0 <= shim.slot(first, last, k) < 2 * grid for k in range(n))


def test_the_join_asks_for_no_slot_otherwise():
    """The joining kernel's places go through parts_of and part_slot alone."""
    with open(os.path.join(OPS, "mk_tree_attn.cu")) as f:
        src = f.read()
    body = src[src.index("merge_kernel(const __grid_constant__ AttnArgs"):src.index("size_t part_bytes")]
    assert ".first" not in body and ".last" not in body
    assert body.count("parts_of(") == 2 and body.count("part_slot(") == 2
