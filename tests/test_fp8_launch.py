"""Which of its two kernels an 8-bit product of a few positions takes (csrc/block_launch.cuh, compiled for this host): the one that
was measured to be faster, and launches that cover all columns and positions.  Widths of the tensor cores' tiles."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "serving_route_count_gb300", "csrc")
SHIM = """
#include "block_launch.cuh"
extern "C" int takes(int S, int E, int offsets, int act, int N, int K) {
  return moe::fp8_few_takes(S, E, offsets, act, N, K, 152);
}
extern "C" void plan(int S, int E, int KT, int RB, int* o) {
  const moe::F8Plan p = moe::fp8_tc_plan(S, E, KT, RB, 76), most = moe::fp8_tc_by_rows(S, E);
  o[0] = p.bn; o[1] = p.fix_steps; o[2] = most.bn; o[3] = most.fix_steps;
}
extern "C" void shape(int S, int offsets, int cols, int K, int* o) {
  const moe::F8vShape f = moe::fp8_few_shape(S, offsets, cols, K, 152);
  o[0] = f.nc; o[1] = f.warps; o[2] = f.x; o[3] = f.y;
}
"""


@pytest.fixture(scope="module")
def few(tmp_path_factory):
    folder = tmp_path_factory.mktemp("few")
    src, so = folder / "shim.cpp", folder / "shim.so"
    src.write_text(SHIM)
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-fPIC", "-shared", "-I", CSRC, str(src), "-o", str(so)], check=True)
    return ctypes.CDLL(str(so))


# (positions, experts, offsets, SwiGLU, N, K), us on the CUDA cores and on the tensor cores, weights from HBM
MEASURED = [
    ((1, 384, 1, 0, 7168, 576), 7.1, 7.8), ((2, 384, 1, 0, 7168, 576), 11.7, 8.8), ((6, 384, 1, 0, 7168, 576), 31.2, 14.2),
    ((8, 384, 1, 0, 7168, 576), 40.9, 15.2), ((8, 256, 1, 0, 6144, 512), 34.4, 12.7), ((8, 256, 1, 1, 1024, 6144), 19.2, 23.0),
    ((6, 384, 1, 1, 1152, 7168), 22.1, 23.3), ((8, 384, 1, 1, 1152, 7168), 22.9, 26.0), ((4, 64, 1, 1, 2304, 7168), 22.8, 26.0),
    ((8, 64, 1, 1, 2304, 7168), 42.2, 28.4), ((8, 64, 1, 1, 4096, 7168), 75.0, 48.3), ((8, 64, 1, 0, 7168, 7168), 117.7, 68.3),
    ((2, 64, 1, 0, 4096, 4096), 13.0, 19.4), ((8, 64, 1, 0, 4096, 4096), 42.0, 34.4), ((4, 64, 1, 0, 2560, 4096), 15.6, 21.3),
    ((8, 64, 1, 0, 512, 7168), 13.0, 19.8), ((8, 64, 1, 0, 512, 512), 4.7, 6.9), ((1, 64, 1, 0, 16384, 576), 13.2, 9.0),
    ((2, 1, 1, 0, 7168, 576), 10.9, 7.2), ((4, 1, 1, 0, 7168, 7168), 59.2, 21.9), ((2, 1, 1, 1, 2304, 7168), 11.8, 18.4),
    ((1, 1, 0, 1, 2304, 7168), 7.8, 18.2), ((2, 1, 0, 1, 2304, 7168), 9.1, 18.3), ((4, 1, 0, 1, 2304, 7168), 15.1, 18.3),
    ((8, 1, 0, 1, 2304, 7168), 24.1, 18.4), ((1, 1, 0, 0, 7168, 7168), 17.6, 21.8), ((2, 1, 0, 0, 7168, 7168), 27.4, 21.9),
    ((4, 1, 0, 0, 7168, 7168), 43.2, 21.7), ((4, 1, 0, 0, 4096, 4096), 20.9, 16.6), ((2, 1, 0, 0, 4096, 4096), 10.7, 16.5),
    ((1, 1, 0, 0, 16384, 4096), 21.5, 17.9), ((1, 1, 0, 1, 12288, 7168), 36.7, 28.1), ((2, 1, 0, 0, 6144, 512), 7.1, 6.2),
    ((4, 1, 0, 0, 2560, 4096), 12.0, 15.4),
]


@pytest.mark.parametrize("call,cores,tensor", MEASURED)
def test_the_faster_kernel(few, call, cores, tensor):
    assert few.takes(*call) == (cores < tensor)


def test_what_is_not_taken(few):
    assert not any(few.takes(1, 8, 1, 0, 64, K) for K in (1, 8, 17, 100))            # no whole vectors
    assert not few.takes(9, 1024, 1, 0, 16, 16) and not few.takes(3, 1, 0, 0, 512, 4080) and not few.takes(5, 1, 0, 0, 512, 4096)
    assert not few.takes(1, 1, 0, 0, 1 << 22, 1 << 18) and not few.takes(1, 1024, 1, 1, 1 << 21, 16)


@pytest.mark.parametrize("offsets", [0, 1])
def test_every_column_and_position_has_a_cta(few, offsets):
    o = (ctypes.c_int * 4)()
    for S in (1, 2, 3, 4, 8):
        for cols in (1, 7, 512, 1152, 7168, 1 << 22):
            for K in (16, 512, 528, 6144, 1 << 24):
                few.shape(S, offsets, cols, K, o)
                nc, warps, x, y = o
                assert nc in (1, 2, 4) and warps in (1, 2, 4, 8) and nc * y >= S > nc * (y - 1)
                assert x * (8 // warps) >= cols > (x - 1) * (8 // warps) and y <= 8


def tiles(few, S, E, N, K, act):
    o = (ctypes.c_int * 4)()
    few.plan(S, E, -(-K // 128), -(-(N // 2) // 128) if act else -(-N // 256), o)
    return list(o)


# E, rows of each, N, K, SwiGLU; the fastest width measured, and whether whole units were faster than cut ones
@pytest.mark.parametrize("E,mean,N,K,act,bn,whole", [
    (4, 120, 1024, 4096, 0, 32, 1), (4, 60, 1024, 4096, 0, 32, 1), (4, 250, 1024, 4096, 0, 64, 1), (8, 60, 1024, 4096, 0, 32, 1),
    (8, 120, 1024, 4096, 0, 64, 1), (2, 120, 2304, 7168, 1, 32, 1), (4, 60, 2304, 7168, 1, 32, 1), (4, 120, 2304, 7168, 1, 64, 1),
    (8, 120, 1024, 6144, 1, 64, 1), (4, 250, 1024, 6144, 1, 64, 1), (8, 120, 512, 7168, 0, 32, 1), (8, 250, 512, 7168, 0, 64, 1),
    (16, 120, 512, 7168, 0, 64, 1), (2, 16, 4096, 2048, 0, 32, 1), (2, 100, 512, 7168, 0, 32, 0), (2, 120, 512, 7168, 0, 32, 0)])
def test_few_experts_take_the_fastest_width(few, E, mean, N, K, act, bn, whole):
    got = tiles(few, E * mean, E, N, K, act)
    assert got[:2] == [bn, 0x7FFFFFFF if whole else 0]


def test_widths_over_many_experts_go_by_rows(few):
    for S, bn in ((64, 32), (24 * 256, 32), (24 * 256 + 1, 64), (56 * 256, 64), (56 * 256 + 1, 128), (104 * 256, 128), (104 * 256 + 1, 256)):
        got = tiles(few, S, 256, 1024, 6144, 1)
        assert got[0] == bn and got[:2] == got[2:]


def test_no_width_is_wider_than_the_scratch_buffer(few):
    """The buffer is sized by the most positions of a plan; a call of fewer gets at most the width by rows, which grows with them."""
    for E in (2, 3, 8, 40, 1024):
        for N, K, act in ((16, 16, 0), (1024, 4096, 0), (2304, 7168, 1)):
            last = 0
            for S in sorted({*range(1, 300, 7), *range(E, 300 * E, max(1, 11 * E // 2)), 1 << 30}):
                bn, _, most, _ = tiles(few, S, E, N, K, act)
                assert bn in (32, 64, 128, 256) and bn <= most and most >= last
                last = most
    for S in (1, 32, 33, 64, 65, 128, 129, 5000, 1 << 30):                        # one matrix: the tile that holds all positions
        assert tiles(few, S, 1, 4096, 7168, 0)[0] <= max(32, 1 << (min(S, 256) - 1).bit_length())
