"""Launch shapes of the 16-bit block's kernels: every call that is taken fits its launch."""
import ctypes

import pytest

import block_shapes


@pytest.fixture(scope="module")
def shapes(tmp_path_factory):
    return block_shapes.build(tmp_path_factory.mktemp("shapes"))


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


@pytest.mark.parametrize("res", [2, 4])
@pytest.mark.parametrize("combine", [0, 1])
def test_norm_shape(shapes, combine, res):
    o = (ctypes.c_int * 3)()
    rings = set()
    for H in [*range(1, 1100, 3), *range(1096, 32769, 8), 32767, 32768]:
        for M in (1, 152, 153, 1000, 2000, 40000):
            for vec in (0, 1) if H % 8 == 0 else (0,):
                ring = shapes.norm_shape(M, H, res, vec, combine, 152, o)
                nch, threads, slots = o
                assert threads % 32 == 0 and nch * threads * 8 >= H                         # every channel has a thread
                if ring:
                    assert vec and nch in (2, 4) and threads <= 480 and 2 <= slots <= 16
                    assert slots * H * res <= shapes.norm_rings()
                    rings.add(nch)
                else:
                    assert nch in (1, 2, 4) and threads <= 1024 and slots == 0
    assert rings == ({2, 4} if res == 2 else {2})


@pytest.mark.parametrize("M,H,res,combine,ring", [(4096, 7168, 2, 1, 1), (8192, 6144, 4, 0, 1), (1, 7168, 2, 1, 0), (152, 7168, 2, 1, 0), (153, 7168, 2, 1, 1),
                                                  (8192, 2048, 2, 1, 1), (16384, 1024, 2, 1, 1), (32768, 1024, 2, 0, 0), (32768, 512, 2, 1, 0)])
def test_norm_kernel_of_a_size(shapes, M, H, res, combine, ring):
    """The sizes whose times decide between the two kernels, on 152 SMs."""
    assert shapes.norm_shape(M, H, res, 1, combine, 152, (ctypes.c_int * 3)()) == ring
