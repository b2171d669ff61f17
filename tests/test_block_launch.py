"""Launch shapes of the 16-bit block's kernels (csrc/block_launch.cuh), compiled for this host."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "serving_route_count_gb300", "csrc")
SHIM = """
#include "block_launch.cuh"
extern "C" void group_shape(int S, int widest, int* o) {
  const moe::GroupShape g = moe::group_shape(S, widest);
  o[0] = g.ctas; o[1] = g.per_cta; o[2] = g.per_warp; o[3] = g.warps;
}
extern "C" void grouped_simt_grid(int S, int E, int cols, unsigned* o) {
  const moe::GsGrid g = moe::grouped_simt_grid(S, E, cols);
  o[0] = g.x; o[1] = g.y;
}
"""


@pytest.fixture(scope="module")
def shapes(tmp_path_factory):
    d = tmp_path_factory.mktemp("shapes")
    (d / "shim.cpp").write_text(SHIM)
    so = str(d / "shim.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-fPIC", "-shared", "-I", CSRC, str(d / "shim.cpp"), "-o", so], check=True)
    return ctypes.CDLL(so)


@pytest.mark.parametrize("widest", [8, 16])
@pytest.mark.parametrize("S", [0, 1, 31, 32, 33, 255, 256, 257, 1024, 1025, 8192, 8193, 65536, 99991, 1 << 20, (1 << 30) - 1, 1 << 30])
def test_group_shape(shapes, S, widest):
    o = (ctypes.c_int * 4)()
    shapes.group_shape(S, widest, o)
    ctas, per_cta, per_warp, warps = o
    assert 1 <= ctas <= widest and 1 <= warps <= 32
    assert per_cta > 0 and per_cta % 32 == 0 and per_warp > 0 and per_warp % 32 == 0
    assert ctas * per_cta >= S and warps * per_warp >= per_cta > (warps - 1) * per_warp     # every slot has one owner
    assert ctas * per_cta + 32 * per_warp < 1 << 31                                         # a warp's first slot is an int


@pytest.mark.parametrize("cols", [1, 64, 65, 4194240, 4194241, 1 << 22])
@pytest.mark.parametrize("S,E", [(1, 1), (63, 4), (65, 1024), (1 << 20, 3), (1 << 30, 1024)])
def test_grouped_simt_grid(shapes, S, E, cols):
    """Every size that a plan takes launches: x up to 2^31 - 1, y up to 65535, and enough of both."""
    o = (ctypes.c_uint * 2)()
    shapes.grouped_simt_grid(S, E, cols, o)
    x, y = o
    assert -(-S // 64) <= x < 1 << 31 and 1 <= y <= 65535 and y == min(65535, -(-cols // 64))
    # the most tiles: E - 1 experts of one position, the rest in the last one
    rest = S - (E - 1)
    assert x >= ((E - 1) + -(-rest // 64) if rest > 0 else S)
