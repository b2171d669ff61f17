// block_launch.cuh - launch shapes of the kernels of the 16-bit block and of the 8-bit products: host arithmetic alone, without CUDA, so that it can be checked on any host.
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

// ---------------------------------------------------------------------------------- 8-bit products of a few positions
constexpr int kF8vThreads = 256, kF8vWarps = kF8vThreads / 32;

// CUDA-core kernel: positions that share a CTA's rows, warps of an output column, CTAs over the columns and over
// the positions.
struct F8vShape {
  int nc, warps, x, y;
};

inline F8vShape fp8_few_shape(int S, bool offsets, int cols, int K, int sms) {
  F8vShape f;
  f.nc = offsets ? 1 : (S > 2 ? 4 : S);
  f.y = (S + f.nc - 1) / f.nc;
  f.warps = 1;
  // warps enough for every SM to have 16, as far as each still has a vector of every lane
  while (f.warps < kF8vWarps && (long long)cols * f.y * f.warps < 16LL * sms && K > f.warps * 512) f.warps *= 2;
  const int per = kF8vWarps / f.warps;
  f.x = (cols + per - 1) / per;
  return f;
}

// Whether a call takes that kernel or the tensor cores', whose units stream a matrix once for all positions of it, after
// a start of 6 us and more with K.  The CUDA cores win as long as their CTAs run at once or nearly: an SM holds four
// (a SwiGLU's hold twice the loads), and of those without a SwiGLU a second wave pays still.  us on the CUDA cores /
// on the tensor cores, weights from HBM:
//   one position to a CTA (offsets), by CTAs: SwiGLU K = 6144, N = 1024, 8 positions of as many experts, 512 CTAs: 19.2 /
//   23.0;  K = 7168, N = 2304, 4 (576): 22.8 / 26.0, 6 (864): 39.2 / 30.2;  K = 2048, N = 8192, 1 (512): 8.4 / 16.6, 2
//   (1024): 15.1 / 13.4;  none: K = 7168, N = 9216, 1 (1152): 23.4 / 25.5;  K = 4096, N = 2560, 4 (1280): 15.6 / 21.3;
//   K = 576, N = 7168, 1 (896): 7.1 / 7.8, 2 (1792): 11.7 / 8.8, 8 (7168): 40.9 / 15.2;  K = 576, N = 16384, 1 (2048): 13.2 / 9.0.
//   Positions of one expert read its rows once each, where the tensor cores read them once: K = 7168, N = 2304, 4: 19.0 / 19.0.
//   two of one matrix: SwiGLU K = 7168, N = 2304 (576): 9.1 / 18.3;  none: K = 4096, N = 4096 (512): 10.7 / 16.5;  K = 512,
//   N = 6144 (768): 7.1 / 6.2;  K = 7168, N = 7168 (896): 27.4 / 21.9.
//   three or four: K = 7168, N = 2304 SwiGLU 15.1 / 18.3;  K = 4096, N = 2560 12.0 / 15.4;  K = 7168, N = 2816 22.2 / 17.8;
//   K = 4096, N = 4096 20.9 / 16.6;  K = 2048, N = 4096 12.5 / 9.9.
inline bool fp8_few_takes(int S, int E, bool offsets, bool act, int N, int K, int sms) {
  if (K % 16 != 0 || S < 1 || S > (E > 1 ? 8 : (K >= 4096 ? 4 : 2))) return false;
  const F8vShape f = fp8_few_shape(S, offsets, act ? N / 2 : N, K, sms);
  const long long ctas = (long long)f.x * f.y;
  if (f.nc == 4) return ctas <= 4LL * sms && N <= 2560;
  return ctas <= (f.nc == 1 && !act ? 17LL * sms / 2 : 4LL * sms);
}

// ---------------------------------------------------------------------------------- 8-bit products, tensor cores
// Token-tile width, and the K steps that cutting the units which whole waves leave over has to save (none: 0; as many
// as there are: never).
struct F8Plan {
  int bn, fix_steps;
};

// Over experts, whose rows are known on the device only, by the mean positions per expert (of S, dropped
// slots among them): an expert should be one tile while HBM is the bound, and up to 64 tokens a step's
// epilogue stays under its loads.  E = 256, K = 6144, N = 1024, SwiGLU, gathered, us at widths 32 / 64 /
// 128 / 256: mean 16: 254 / 253 / 349 / 421;  24: 248 / 258 / 352 / 429;  32: 302 / 262 / 359 / 435;  48:
// 395 / 270 / 368 / 443;  64: 504 / 389 / 373 / 450;  96: 690 / 496 / 387 / 460;  128: 890 / 625 / 576 / 472.
// The crossings are of that layer, where units are many: E = 64, K = 7168, N = 2304, mean 60 takes 128 (246 us; 64:
// 175), E = 64, K = 576, N = 7168, mean 120 takes 256 (147; 128: 106).
inline F8Plan fp8_tc_by_rows(int S, int E) {
  const long long e = E;
  if (S <= 24 * e) return {32, 8};
  if (S <= 56 * e) return {64, 12};
  return S <= 104 * e ? F8Plan{128, 24} : F8Plan{256, 40};
}

// The least of the estimated times at widths up to `widest`, for S positions spread evenly over E experts (one
// matrix: E = 1): a unit's K step, and joining its pieces by rows and pieces.  One matrix, K = 7168, N = 4096, us at
// widths 32 / 64 / 128 / 256: 32 rows 18 / 19 / 22 / 34;  128: 23 / 25 / 33 / 39;  200: 39 / 26 / 33 / 40;  300: 54 /
// 46 / 34 / 40;  1000: 119 / 87 / 62 / 43.
inline F8Plan fp8_tc_by_time(int S, int E, int KT, int RB, int pairs, int widest) {
  const long long touched = std::min(S, E), per = (S + touched - 1) / touched;
  F8Plan best{widest, 0x7FFFFFFF};
  double least = 1e300;
  for (int bn = 32; bn <= widest; bn *= 2) {
    const long long tiles = touched * ((per + bn - 1) / bn);
    const double step = bn == 32 ? 320 : (bn == 64 ? 385 : (bn == 128 ? 560 : 740));     // ns
    const long long units = tiles * RB, waves = units / pairs, left = units % pairs;
    const double base = (double)waves * KT * step;
    const double whole = base + (left ? KT * step : 0);
    if (whole <= least) {
      least = whole;
      best = {bn, 0x7FFFFFFF};
    }
    if (left) {
      const double pieces = (double)pairs / left + 1, rows = (double)((S + tiles - 1) / tiles);
      const double cut = base + (double)left * KT / pairs * step + 4000 + rows * (100 + 6 * pieces);
      if (cut < least) {
        least = cut;
        best = {bn, 0};
      }
    }
    if (bn >= per) break;              // one tile holds an expert's
  }
  return best;
}

// One matrix goes by estimated time.  Experts go by rows, but where the units of that width leave half of the pairs or
// more idle (few experts, a small N): there too the estimate decides, at widths up to that one, which the scratch
// buffer is sized for.  us by rows / here, E = 4, K = 4096, N = 1024 without a SwiGLU: mean 120: 26 / 17;  60: 27 / 16;
// E = 8, K = 7168, N = 512, mean 120: 36 / 24;  E = 4, K = 7168, N = 2304 SwiGLU, mean 120: 40 / 28.  With half of all rows at
// one expert, which the mean does not tell, narrow tiles lose once more pairs are busy (E = 16, K = 6144, N = 1024, mean
// 120: 41 by rows, 63 by the estimate), hence the half.
inline F8Plan fp8_tc_plan(int S, int E, int KT, int RB, int pairs) {
  if (E == 1) return fp8_tc_by_time(S, 1, KT, RB, pairs, 256);
  const F8Plan p = fp8_tc_by_rows(S, E);
  const long long touched = std::min(S, E), per = (S + touched - 1) / touched;
  const long long units = touched * ((per + p.bn - 1) / p.bn) * RB;
  return 2 * units <= pairs ? fp8_tc_by_time(S, E, KT, RB, pairs, p.bn) : p;
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
