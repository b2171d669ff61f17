"""Launch shapes of the 16-bit block's kernels (csrc/block_launch.cuh), compiled for this host."""
import ctypes
import os
import subprocess

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
extern "C" int norm_shape(int M, int H, int res_bytes, int vec, int combine, int sms, int* o) {
  const moe::NormShape n = moe::norm_shape(M, H, res_bytes, vec, combine, sms);
  o[0] = n.nch; o[1] = n.threads; o[2] = n.slots;
  return n.ring;
}
extern "C" int norm_rings() { return moe::kNormRings; }
"""


def build(folder):
    """The shapes as a library, built in `folder`."""
    src, so = os.path.join(str(folder), "shim.cpp"), os.path.join(str(folder), "shim.so")
    with open(src, "w") as f:
        f.write(SHIM)
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-fPIC", "-shared", "-pthread", "-I", CSRC, src, "-o", so], check=True)
    return ctypes.CDLL(so)
