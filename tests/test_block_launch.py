"""Launch shapes of the 16-bit block's kernels (csrc/block_launch.cuh), compiled for this host."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "serving_route_count_gb300", "csrc")
SHIM = """
#include "block_launch.cuh"
#include <thread>
#include <vector>
// 16 threads ask for devices 0 .. 3, over and over; o[d]: how often device d was asked.  Its first two answers are errors.
extern "C" int per_device(int* o) {
  moe::PerDevice<int> per;
  std::atomic<int> asked[4] = {}, errors{0}, wrong{0};
  std::vector<std::thread> threads;
  for (int i = 0; i < 16; ++i)
    threads.emplace_back([&, i] {
      for (int j = 0; j < 2000; ++j) {
        const int dev = (unsigned)(i + j) % 4u;
        int v = -1;
        if (per.get(dev, &v, [&](int* p) { *p = 100 + dev; return asked[dev]++ < 2 ? 7 : 0; }) != 0)
          ++errors;
        else if (v != 100 + dev)
          ++wrong;
      }
    });
  for (auto& t : threads) t.join();
  for (int d = 0; d < 4; ++d) o[d] = asked[d];
  o[4] = errors;
  int past = 0;
  for (int j = 0; j < 3; ++j) per.get(j < 2 ? 64 : -1, &o[5], [&](int* p) { *p = 5; ++past; return 0; });
  o[6] = past;
  return wrong;
}
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
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-fPIC", "-shared", "-pthread", "-I", CSRC, str(d / "shim.cpp"), "-o", so], check=True)
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


def test_facts_of_each_device(shapes):
    """A kernel's attributes are set once on every device that launches it, whichever thread comes first; errors are not kept."""
    o = (ctypes.c_int * 7)()
    assert shapes.per_device(o) == 0
    assert list(o) == [3, 3, 3, 3, 8, 5, 3]
