// tc_units.cuh - how the pair kernels of the 16- and 8-bit products (grouped by expert or dense) share
// out their work: units of a token tile and a weight row block, whole or cut along K.
#pragma once

#include "block_ops.cuh"
#include "grouped.cuh"
#include "../../include/moe_gb300.h"

namespace moe {

constexpr int kGtMinSteps = 4;           // K steps below which a piece is not cut further

// Units of one pair: first its range of the leftover units' K steps, then its whole units, round
// robin (sorted: to and fro).  A unit is a token tile and a weight row block of it.  Numbers: the blocks of a tile
// adjacent (they share its tokens), and where the last block has only one of two accumulators
// (half the work) those of all tiles at the end, so that the last wave consists of them.
struct GtWork {
  int KT, RB, G, Gs, D, first;     // RB: blocks with all accumulators; first: units before it are whole
  uint32_t W, x, x1;               // leftover steps, this pair's range of them
  int full, w;                     // units of whole blocks; next wave
  int at, back;                    // this pair's place in even and in odd waves
  __device__ __forceinline__ void init(int tiles, int kt, int rbs, int half, int g, int cta,
                                       int fix_steps, bool sorted) {
    KT = kt; RB = rbs; G = g;
    full = tiles * rbs;
    const int units = full + (half ? tiles : 0);
    D = units / g;
    w = 0;
    at = cta;
    back = sorted ? g - 1 - cta : cta;
    first = D * g;
    const uint32_t R = (uint32_t)(units - first);
    W = R * (uint32_t)kt;
    // cut the leftover units when that shortens the longest pair's work by more than the join
    // costs (both in K steps)
    if (kt - (int)(W / (uint32_t)g) <= fix_steps) {
      first = units;
      D += ((D & 1) ? back : at) < (int)R;
      W = 0;
    }
    // pairs that share the leftover steps: all of them, unless the pieces got too short
    const uint32_t most = W / kGtMinSteps > R ? W / kGtMinSteps : R;
    Gs = most < (uint32_t)g ? (int)most : g;
    x = W && cta < Gs ? begin_of(cta) : 0u;
    x1 = W && cta < Gs ? begin_of(cta + 1) : 0u;
  }
  __device__ __forceinline__ uint32_t begin_of(int cta) const {
    return (uint32_t)cta * W / (uint32_t)Gs;
  }
  __device__ __forceinline__ void place(int unit, int& t, int& r) const {
    if (unit < full) {
      t = unit / RB;
      r = unit - t * RB;
    } else {
      t = unit - full;
      r = RB;
    }
  }
  __device__ __forceinline__ bool next(int& unit, int& t, int& r, int& k0, int& len) {
    if (x < x1) {
      const uint32_t kt = (uint32_t)KT;
      unit = first + (int)(x / kt);
      k0 = (int)(x % kt);
      len = (int)min(kt - (uint32_t)k0, x1 - x);
      x += (uint32_t)len;
    } else if (D > 0) {
      --D;
      unit = w * G + ((w & 1) ? back : at);
      ++w;
      k0 = 0;
      len = KT;
    } else {
      return false;
    }
    place(unit, t, r);
    return true;
  }
  // The pairs that hold unit u's steps are a run of them; [c0, c1] bounds it.
  __device__ __forceinline__ void owners(int u, int& c0, int& c1) const {
    const uint32_t xs = (uint32_t)(u - first) * (uint32_t)KT, xe = xs + (uint32_t)KT;
    c0 = (int)((uint64_t)xs * (uint32_t)Gs / W);
    while (c0 > 0 && begin_of(c0) > xs) --c0;
    while (begin_of(c0 + 1) <= xs) ++c0;
    c1 = c0;
    while (c1 + 1 < Gs && begin_of(c1 + 1) < xe) ++c1;
  }
  __device__ __forceinline__ int slot_of(int cta, int u) const {
    return 2 * cta + (first + (int)(begin_of(cta) / (uint32_t)KT) == u ? 0 : 1);
  }
};

// A token tile: its expert, first position, positions, and how many of them (padded) a CTA of the pair
// loads, a multiple of 8.
struct GtTile {
  int e, p0, n, nhalf;
};
// An expert's tokens go in tiles of one size, a multiple of 16 (256 + 24 rows would cost a tile of
// 24 that streams as many weights as one of 256).
template <int BN>
__device__ __forceinline__ int gt_size(int cnt, int tiles) {
  return tiles > 1 ? 16 * cdiv(cdiv(cnt, tiles), 16) : BN;
}
// Rows of the experts, by all threads of a CTA: thread t owns experts 4 t .. 4 t + 3 (cnt), the tables
// s_off and s_cnt get all of them, s_tile what lies past E.  Offsets that are out of order or range make
// the call empty (every CTA sees the same ones; the result is true), so that no tile is ever out of
// its bounds.  offsets NULL: one expert, all S rows.
__device__ __forceinline__ int gt_counts(const int32_t* offsets, int E, int S, int (&cnt)[4], int* s_off,
                                         int* s_cnt, int* s_tile) {
  int bad = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = 4 * (int)threadIdx.x + i;
    cnt[i] = 0;
    if (e < E) {
      const int a = offsets != nullptr ? offsets[e] : 0, b = offsets != nullptr ? offsets[e + 1] : S;
      if (a < 0 || b < a || b > S)
        bad = 1;
      else
        cnt[i] = b - a;
      s_off[e] = a;
      s_cnt[e] = cnt[i];
    }
    if (e >= E && e < 1024) s_tile[e] = 0x7FFFFFFF;
  }
  return __syncthreads_or(bad);
}
// Numbers the experts' tiles in the tables' order (s_tile); their total.  s_warp: an int for each warp.
template <int BN, int THREADS>
__device__ __forceinline__ int gt_number(const int (&cnt)[4], int E, int* s_tile, int* s_warp) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int tiles = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) tiles += cdiv(cnt[i], BN);
  int incl = tiles;
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  int before = incl - tiles, total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += s_warp[w];
    total += s_warp[w];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (4 * tid + i < E) s_tile[4 * tid + i] = before;
    before += cdiv(cnt[i], BN);
  }
  return total;
}

// A tile's expert and token range (by a whole warp).  s_tile[i]: tiles before the
// tables' expert i, 1024 entries; the tile's is the last one with s_tile[i] <= tile, found by two
// 32-way comparisons.  s_expert: the experts' numbers, NULL where the tables are in their order.
template <int BN>
__device__ __forceinline__ GtTile gt_tile(int tile, const int* s_tile, const int* s_off,
                                          const int* s_cnt, const int* s_expert, int lane) {
  const int hi = __popc(__ballot_sync(0xffffffffu, s_tile[32 * lane] <= tile)) - 1;
  const int lo = __popc(__ballot_sync(0xffffffffu, s_tile[32 * hi + lane] <= tile)) - 1;
  GtTile r;
  const int i = 32 * hi + lo;
  r.e = s_expert != nullptr ? s_expert[i] : i;
  const int t = tile - s_tile[i], cnt = s_cnt[i], size = gt_size<BN>(cnt, cdiv(cnt, BN));
  r.p0 = s_off[i] + t * size;
  r.n = min(size, cnt - t * size);
  r.nhalf = 8 * cdiv(r.n, 16);
  return r;
}

// Stores 32 accumulator columns (tokens c0 .. c0 + 31 of the unit, n of them valid) of this
// lane's row; col0: output column of the CTA's first row.  A lane and its neighbour exchange every
// other token, so that each store writes two adjacent output columns; where the output's rows do
// not start on 4 bytes (odd widths or strides) each lane stores its column.  One pointer that
// advances and one bound serve all tokens: an address formed anew for each under its own bound
// took 37 us where this takes 23 (14 experts, 31864 rows, 336 -> 387 columns; 386 columns: 21).
template <typename T, bool ACT, typename Params>
__device__ __forceinline__ void gt_store(const Params& p, float (&v)[32], const GtTile& un,
                                         int col0, int c0, int q, int lane) {
  T* out = static_cast<T*>(p.c.out);
  const int odd = lane & 1;
  if constexpr (ACT) {
    // lanes 0-15: half 0 of outputs i .. i + 15, lanes 16-31: half 1; after the exchange lanes
    // 0-15 hold tokens c0 .. c0 + 15 of both halves, lanes 16-31 tokens c0 + 16 .. c0 + 31
    const bool hi = lane >= 16;
    const bool up_first = p.d.layout == MOE_W13_UP_GATE;
    float h[16];
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      const float got = __shfl_xor_sync(0xffffffffu, hi ? v[c] : v[c + 16], 16);
      const float a = hi ? got : v[c], b = hi ? v[c + 16] : got;
      h[c] = swiglu_f32(up_first ? a : b, up_first ? b : a, p.d.limit, p.d.alpha, p.d.beta);
    }
    const int col = col0 + q * 16 + (lane & 15);
    const int t0 = c0 + (hi ? 16 : 0);
    if (p.packed) {
      T* o = out + (size_t)(un.p0 + t0 + odd) * p.c.ldo + (col & ~1);
      const int n = col < p.cols ? un.n - t0 - odd : 0;
#pragma unroll
      for (int c = 0; c < 16; c += 2) {
        const float got = __shfl_xor_sync(0xffffffffu, odd ? h[c] : h[c + 1], 1);
        const T pair[2] = {from_f32<T>(odd ? got : h[c]), from_f32<T>(odd ? h[c + 1] : got)};
        uint32_t w;
        memcpy(&w, pair, 4);
        if (c < n) *reinterpret_cast<uint32_t*>(o) = w;
        o += 2 * p.c.ldo;
      }
    } else {
      T* o = out + (size_t)(un.p0 + t0) * p.c.ldo + col;
      const int n = col < p.cols ? un.n - t0 : 0;
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        if (c < n) *o = from_f32<T>(h[c]);
        o += p.c.ldo;
      }
    }
  } else {
    const int col = col0 + q * 32 + lane;
    if (p.packed) {
      T* o = out + (size_t)(un.p0 + c0 + odd) * p.c.ldo + (col & ~1);
      const int n = col < p.cols ? un.n - c0 - odd : 0;
#pragma unroll
      for (int c = 0; c < 32; c += 2) {
        const float got = __shfl_xor_sync(0xffffffffu, odd ? v[c] : v[c + 1], 1);
        const T pair[2] = {from_f32<T>(odd ? got : v[c]), from_f32<T>(odd ? v[c + 1] : got)};
        uint32_t w;
        memcpy(&w, pair, 4);
        if (c < n) *reinterpret_cast<uint32_t*>(o) = w;
        o += 2 * p.c.ldo;
      }
    } else {
      T* o = out + (size_t)(un.p0 + c0) * p.c.ldo + col;
      const int n = col < p.cols ? un.n - c0 : 0;
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        if (c < n) *o = from_f32<T>(v[c]);
        o += p.c.ldo;
      }
    }
  }
}

}  // namespace moe
