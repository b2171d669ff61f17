// block_launch.cuh - launch shapes of the 16-bit block's kernels: host arithmetic alone, without
// CUDA, so that it can be checked on any host.
#pragma once

#include <algorithm>
#include <atomic>
#include <mutex>

namespace moe {

// What a kernel's first launch on a device sets or finds out there (its attributes, how many CTAs
// fit): one value per device, from any thread.  init(&value) returns 0 or an error, which is not
// kept; a device number past the table is asked anew every time.
template <typename V>
class PerDevice {
 public:
  template <typename Init>
  int get(int dev, V* out, Init init) {
    if (dev < 0 || dev >= kDevices) return init(out);
    if (!ready_[dev].load(std::memory_order_acquire)) {
      std::lock_guard<std::mutex> lock(mutex_);
      if (!ready_[dev].load(std::memory_order_relaxed)) {
        const int e = init(&value_[dev]);
        if (e != 0) return e;
        ready_[dev].store(true, std::memory_order_release);
      }
    }
    *out = value_[dev];
    return 0;
  }

 private:
  static constexpr int kDevices = 64;
  std::atomic<bool> ready_[kDevices] = {};
  V value_[kDevices] = {};
  std::mutex mutex_;
};

inline int ceil_to(int v, int a) { return (v + a - 1) / a * a; }

// ---------------------------------------------------------------------------------- group
constexpr int kGroupThreads = 1024;
constexpr int kGroupWarps = kGroupThreads / 32;

// CTAs of the cluster, slots of each CTA and of each warp (multiples of 32), warps that own slots
// (at least one, also of a call without slots, which still writes the offsets).
struct GroupShape {
  int ctas, per_cta, per_warp, warps;
};

// widest: the largest cluster the device can hold (8 or 16).
// Few slots: the cluster's barriers cost more than they share out (1 / 4 / 8 / 16 CTAs at 256
// experts: 96 slots 3.0 / 3.1 / 3.6 us; 512: 3.8 / 3.5 / 3.7; 2048: 6.6 / 4.1 / 4.1 / 4.4; 8192:
// 12.7 / 6.8 / 5.5 / 5.1; 16384: 21.9 / 8.5 / 7.1 / 6.3).
inline GroupShape group_shape(int S, int widest) {
  GroupShape g;
  g.ctas = S <= 256 ? 1 : (S <= 1024 ? 4 : (S <= 8192 ? 8 : widest));
  g.per_cta = std::max(32, ceil_to((S + g.ctas - 1) / g.ctas, 32));
  g.per_warp = ceil_to((g.per_cta + kGroupWarps - 1) / kGroupWarps, 32);
  g.warps = (g.per_cta + g.per_warp - 1) / g.per_warp;
  return g;
}

// ---------------------------------------------------------------------------------- products
// On the CUDA cores: tiles of 64 positions of one expert (at most one partial one per expert that
// has a position) in x, tiles of 64 output columns in y, as far as a launch counts there: a CTA
// takes every y-th of them.
constexpr int kGsTile = 64;

struct GsGrid {
  unsigned x, y;
};

inline GsGrid grouped_simt_grid(int S, int E, int cols) {
  return {(unsigned)((S + kGsTile - 1) / kGsTile) + (unsigned)std::min(E, S),
          (unsigned)std::min((cols + kGsTile - 1) / kGsTile, 65535)};
}

// ---------------------------------------------------------------------------------- norms
constexpr int kNormSlots = 16;          // most ring buffers of a CTA

// Ring buffers of all of an SM's CTAs; what is left of its shared memory serves as L1 for the weights
// (4096 x 7168 top-6, us with 100 / 132 / 170 / 200 KB: 94 / 91 / 100 / 105).
constexpr int kNormRings = 132 * 1024;

// The row ring (chunks of eight channels a thread, summing threads, buffers of a CTA) or plain
// loads (no slots).
struct NormShape {
  bool ring;
  int nch, threads, slots;
};

// vec: rows of whole vectors (H % 8 == 0 among it); res_bytes: of a residual element; combine: rows
// come by slots.
inline NormShape norm_shape(int M, int H, int res_bytes, bool vec, bool combine, int sms) {
  const int chunks = (H + 7) / 8;
  if (vec) {
    // The ring, but for short rows, where the copying warp costs more than it hides.  us with the ring
    // and with plain loads: 4096 x 7168 top-6 91 / 193, 8192 x 2048 top-6 56 / 70, 16384 x 1024 top-6
    // 62 / 68; without a combine 8192 x 6144 (fp32 residual) 102 / 118, 16384 x 2048 67 / 73, 32768 x
    // 1024 74 / 70, 32768 x 512 52 / 38.  ctas: what an SM's registers hold at the two-chunk kernel's 64
    // a thread; of the four-chunk kernel (126 a thread, H > 7680) it holds one, whose ring is then half
    // of what the SM could give or less (4096 x 8192 top-6 163 us, 54 % of the copy bandwidth).
    const int nch = chunks <= 960 ? 2 : 4, threads = ceil_to((chunks + nch - 1) / nch, 32);
    const int ctas = std::max(1, 65536 / 64 / (threads + 32));
    const int slots = std::min(kNormSlots, kNormRings / ctas / (H * res_bytes));
    // And for few tokens, a CTA each and all of them at once or nearly: 1 x 7168 top-6 4.8 us with
    // plain loads, 5.7 with the ring; 152: 5.2 / 5.9; 304: 9.5 / 7.7; 912 x 4096: 11.1 / 12.2; 1216:
    // 18.1 / 17.6.
    const int at_once = std::max(1, 65536 / 40 / ceil_to(chunks, 32));
    const bool few = M <= sms * (2 * at_once - 1);
    if (!few && chunks >= (combine ? 128 : 192) && threads <= 480 && slots >= 2)
      return {true, nch, threads, slots};
  }
  const int nch = chunks <= 1024 ? 1 : (chunks <= 2048 ? 2 : 4);
  return {false, nch, ceil_to((chunks + nch - 1) / nch, 32), 0};
}

}  // namespace moe
