// gemm_grouped_tc.cu - products grouped by expert with ragged sizes on the tensor cores
// (moe_grouped_run): out[p] = act(W[e] . x[row(p)]).
//
// The weight rows are the MMA's M operand and the tile's tokens its N operand, so an expert with
// one row still streams its weights once, through full-size MMAs.  A pair of CTAs (one MMA of 256
// weight rows, tcgen05 cta_group::2) owns a unit: 256 weight rows of one expert (for a SwiGLU 128
// up and 128 gate rows, interleaved 16 by 16, so that a warp's 32 accumulator lanes hold both
// halves of 16 outputs) x up to BN of the expert's tokens.  Each CTA loads its 128 weight rows and
// half of the tokens per K step of 64; the accumulators are double-buffered in tensor memory, so
// a unit's epilogue runs under the next unit's loads and MMAs.  At BN = 256, where the tensor cores
// are the bound, a unit has 512 weight rows in two accumulators instead: the tokens are loaded
// once for both, a quarter less L2 traffic and half the row gathers per MMA.
//
// The grid is persistent, one pair per two SMs.  The number of units is known on the device only
// (offsets); every CTA builds the table of the experts' tiles in shared memory.  Whole waves of
// units go round robin; where it shortens the longest pair's work, the units left over are cut evenly
// by K steps: every piece's fp32 sums go to the scratch buffer, and the piece that arrives last adds
// them in K order (bit-stable, nobody waits).
//
// Bounds and measurements (GB300, weights read once at the measured 6791 GB/s, bf16 unless stated):
//   fc1 + SwiGLU of 8 tokens top-8, E = 256, K = 6144, N = 1024: 107-117 us, HBM floor 106; of one
//   token 21.8, floor 14.8;
//   fc2 of 16 tokens top-6, E = 384, K = 576, N = 7168: 112-117 us, floor 104 - what is left is the
//   start (tables 2 us, first loads 2.5 us) and the last units;
//   fc1 of 2048 tokens top-8: 495-508 us, floor 480; fc2 (K = 512, N = 6144): 275 us, floor 269;
//   4096 tokens top-6 over 16 experts, K = 7168, N = 2304 (f16): 473-485 us (1.7 PFLOP/s) in short
//   runs, 552-574 (1.41-1.47 PFLOP/s) in runs of seconds, where the power limit takes the clocks to 1.5
//   GHz: bound by the tensor cores and their power (floor 422 burst, 473 sustained; 8192 x 8192 x 8192
//   in bf16: 568 us, 1.94 PFLOP/s; cuBLAS 538-552).
//   A call with dropped slots writes their rows as zeros before the first weight copy: 4096 tokens top-8,
//   one of eight ranks (4,027 of 32,768 rows its own, N = 7168, K = 512) 144 us, its rows alone 53.
//
// Roles: warp 0 weight copies, warp 1 MMA issue (leader CTA), warps 2-7 token copies (tiles, or
// gathers of four rows by index, whose issue takes ~70 cycles each: six warps share it; warp 3
// also allocates the tensor memory), warps 8-15 epilogue.
#include <type_traits>

#include "block_ops.cuh"
#include "grouped.cuh"
#include "tc_pair.cuh"
#include "tc_tile.cuh"
#include "tc_units.cuh"
#include "../../include/moe_gb300.h"

namespace moe {
using namespace tc;

constexpr int kGtThreads = 512;
constexpr int kGtTokenWarps = 6;         // warps 2-7
constexpr int kGtK = 64;                 // K step: one 128-byte swizzled row per operand row
constexpr int kGtSortSteps = 56;         // K steps from which tiles are ordered by size (below)

template <int BN, int ACC>
struct GtCfg {
  static constexpr int kAcc = ACC;                           // accumulators of a unit
  static constexpr int kHalf = BN / 2;                       // tokens a CTA loads
  static constexpr int kChunk = kHalf < 32 ? kHalf : 32;     // tokens per tile copy
  static constexpr int kBytesW = 128 * 128;                  // weight rows of one accumulator
  static constexpr int kBytesA = kAcc * kBytesW, kBytesB = kHalf * 128, kStage = kBytesA + kBytesB;
  static constexpr bool kSorts = BN == 256;                  // tiles ordered by size
  static constexpr int kTables = (kSorts ? 4 : 3) * 1028 * 4 + 512;   // expert tables, barriers
  static constexpr int kStages = (227 * 1024 - 1024 - kTables) / kStage > 12
                                     ? 12 : (227 * 1024 - 1024 - kTables) / kStage;
  static constexpr int kSmem = 1024 + kStages * kStage + kTables;
  static constexpr int kCols = 2 * BN;                       // tensor-memory columns: two buffers
  // K steps that joining the pieces of a unit costs (its sums through the scratch buffer; 8192 x
  // 8192 x 1024 with every leftover unit cut: 134 us, with this rule 100; lower bounds for narrow
  // tiles under many units cost fc2 of 16 tokens 2 us)
  static constexpr int kFixSteps = BN <= 32 ? 8 : (BN <= 64 ? 12 : (BN <= 128 ? 24 : 40));
};

struct GtParams {
  CUtensorMap tm_w, tm_x;
  GroupedDims d;
  GroupedCall c;
  float* part;          // [pairs][2][2 CTAs][accumulators][BN][128]
  int32_t* tickets;     // [pairs][2 CTAs][2 accumulators]
  int KT, RB, half, cols, packed;   // RB: row blocks with all accumulators; half: one more with one
  int whole16;          // SwiGLU weights by whole 16-row groups: one 5-d copy per K step
};

template <typename T, bool ACT, int BN, int ACC>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGtThreads, 1)
grouped_tc_kernel(const __grid_constant__ GtParams p) {
  using Cfg = GtCfg<BN, ACC>;
  constexpr int S = Cfg::kStages;
  extern __shared__ uint8_t raw[];
  uint8_t* st = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(st + S * Cfg::kStage);   // [S] (leader's are used)
  uint64_t* empty = full + S;          // [S]
  uint64_t* tfull = empty + S;         // [2] accumulators ready
  uint64_t* tempty = tfull + 2;        // [2] accumulators read (leader's are used)
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(tempty + 2);
  int* s_flag = reinterpret_cast<int*>(s_tmem + 1);   // [2]
  int* s_warp = s_flag + 2;            // [warps]
  int* s_fills = s_warp + kGtThreads / 32;   // fills whose stage the weight warp has found empty
  int* s_off = reinterpret_cast<int*>(st + S * Cfg::kStage + 512);
  int* s_cnt = s_off + 1028;
  int* s_tile = s_cnt + 1028;
  int* s_expert = s_tile + 1028;       // where tiles are ordered by size
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, G = gridDim.x >> 1;
  const int E = p.d.E;
  int32_t* err = p.c.err;

  if (warp == 3) {
    tmem2_alloc(s_tmem, Cfg::kCols);
    tmem2_relinquish();
  }
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 8);        // four epilogue warps of each CTA
    }
    fence_barrier_init();
    *s_fills = 0;
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  // the next launch may start now that this CTA's tensor memory is allocated
  pdl_wait_prev();
  pdl_launch_next();

  // the experts' tiles
  int cnt[4];
  const int bad = gt_counts(p.c.offsets, E, p.c.S, cnt, s_off, s_cnt, s_tile);
  if constexpr (Cfg::kSorts) {
    for (int e = tid; e < E; e += kGtThreads) s_expert[e] = e;
  }
  const auto number = [&]() { return gt_number<BN, kGtThreads>(cnt, E, s_tile, s_warp); };
  int total = number();
  bool sorted = false;
  if constexpr (Cfg::kSorts) {
    // More units than pairs, and long ones: the experts in descending order of their tiles' size, and
    // every other wave in reverse, so that a wave's units are alike, the pairs' sums of them too, and
    // the last ones the smallest.  us without / with: 100 experts of 164 rows, K = 5120 436 / 384;
    // 384 of 128, skewed, K = 7168 1348 / 1255; 8 of 1500, K = 4096 280 / 270, 3584 243 / 238; 16 of
    // 1536, K = 7168 485 / 473; 256 of 128 alike, K = 6144 536 / 543.  At K = 2560 and less the
    // epilogues weigh more, and pairs out of step overlap them better: 32 of 768, K = 2560 235 / 237;
    // 16 of 1536, K = 2048 466 / 475, 1152 284 / 288.
    if (!bad && E > 1 && E <= kGtThreads && p.KT >= kGtSortSteps && total * (p.RB + p.half) > G) {
      int n = 0, off = 0, key = 0, at = 0;
      if (tid < E) {
        n = s_cnt[tid];
        off = s_off[tid];
        const int tiles = cdiv(n, BN);
        key = tiles > 1 ? gt_size<BN>(n, tiles) : n;
        s_expert[tid] = key;
      }
      __syncthreads();
      if (tid < E)
        for (int j = 0; j < E; ++j) at += s_expert[j] > key || (s_expert[j] == key && j < tid);
      __syncthreads();
      if (tid < E) {
        s_cnt[at] = n;
        s_off[at] = off;
        s_expert[at] = tid;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i) cnt[i] = 4 * tid + i < E ? s_cnt[4 * tid + i] : 0;
      total = number();
      sorted = true;
    }
  }
  if (bad) {
    total = 0;
    if (tid == 0) set_error(err, kErrRouteBounds);
  }
  // rows past the last group
  {
    const int end = max(0, min(p.c.S, p.c.offsets[E]));
    T* out = static_cast<T*>(p.c.out);
    for (long long r = end + (long long)blockIdx.x; r < p.c.S; r += gridDim.x)
      for (int c = tid; c < p.cols; c += kGtThreads) out[r * p.c.ldo + c] = from_f32<T>(0.f);
  }
  __syncthreads();

  // Every loop below is taken by whole warps; one lane issues.
  constexpr int kRows = ACT ? 64 : 128;      // output columns of one CTA and accumulator
  GtWork work;
  work.init(total, p.KT, p.RB, p.half, G, pair, Cfg::kFixSteps, sorted);
  int u, tile, rb, k0, len;
  int s = 0, issued = 0;             // ring stage, stages filled
  uint32_t phase = 0;
  bool ok = true;
  const auto advance = [&]() {
    if (++s == S) {
      s = 0;
      phase ^= 1;
    }
  };
  // first output column of a unit, and how many of its accumulators lie within the matrix
  const auto unit_col = [&](int rb) { return rb * (2 * kRows * Cfg::kAcc); };
  const auto accs_of = [&](int rb) { return Cfg::kAcc == 2 && rb < p.RB ? 2 : 1; };
  if (warp == 0) {
    const uint32_t bar0 = map_rank(&full[0], 0);
    while (ok && work.next(u, tile, rb, k0, len)) {
      const GtTile un = gt_tile<BN>(tile, s_tile, s_off, s_cnt, Cfg::kSorts ? s_expert : nullptr, lane);
      const int accs = accs_of(rb);
      const int rows = p.c.perm != nullptr ? un.nhalf : cdiv(un.nhalf, Cfg::kChunk) * Cfg::kChunk;
      const uint32_t bytes = 2u * (accs * Cfg::kBytesW + rows * 128);
      const int r0 = unit_col(rb) + (int)rank * kRows;
      for (int x = k0 * kGtK; x < (k0 + len) * kGtK; x += kGtK, ++issued) {
        if (!mbar_wait_warp(&empty[s], phase ^ 1, err)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          publish_count(s_fills, issued + 1);
          const uint32_t bar = bar0 + 8 * s;
          if (rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
          for (int c = 0; c < accs; ++c) {
            uint8_t* a = st + s * Cfg::kStage + c * Cfg::kBytesW;
            const int r = r0 + c * 2 * kRows;
            if constexpr (!ACT) {
              tma2_load_3d(a, &p.tm_w, x, r, un.e, bar);
            } else if (p.whole16) {
              tma2_load_5d(a, &p.tm_w, x, 0, 0, r >> 4, un.e, bar);
            } else {
#pragma unroll
              for (int b = 0; b < 4; ++b)
                tma2_load_4d(a + b * 4096, &p.tm_w, x, r + 16 * b, 0, un.e, bar);
            }
          }
        }
        advance();
      }
    }
    if (lane == 0) {
      // the last fills have been multiplied: nothing arrives at this CTA's barriers any more
      for (int j = max(0, issued - S); ok && j < issued; ++j)
        ok = mbar_wait(&empty[j % S], (j / S) & 1, err);
      if (!ok && rank == 0) drain_stage_loads<S>(full, issued, err);
    }
  } else if (warp == 1) {
    // operand descriptors: only the address changes from stage to stage and from K block to K block
    const uint64_t desc0 = desc_sw128(st);
    const uint32_t hi = (uint32_t)(desc0 >> 32), lo0 = (uint32_t)desc0;
    uint32_t uses[2] = {0, 0};       // units that each accumulator buffer has held
    int seg = 0;
    // nothing commits to this phase before the first unit's MMAs
    if (p.d.probe_ns != 0 && blockIdx.x == 0)
      ok = __all_sync(0xffffffffu, mbar_wait(&tfull[0], 0, err, p.d.probe_ns));
    while (rank == 0 && ok && work.next(u, tile, rb, k0, len)) {
      const GtTile un = gt_tile<BN>(tile, s_tile, s_off, s_cnt, Cfg::kSorts ? s_expert : nullptr, lane);
      const int accs = accs_of(rb);
      const int b0 = Cfg::kAcc == 2 ? 0 : seg & 1;
      for (int c = 0; ok && c < accs; ++c)
        ok = mbar_wait_warp(&tempty[b0 + c], (uses[b0 + c] & 1) ^ 1, err);
      if (!ok) break;
      tc_fence_after();
      const uint32_t idesc = idesc_pair16(std::is_same<T, __nv_bfloat16>::value, 2 * un.nhalf);
      uint32_t accumulate = 0;
      for (int i = 0; i < len; ++i) {
        if (!mbar_wait_warp(&full[s], phase, err)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (lane == 0) {
          const uint32_t lo = lo0 + s * (Cfg::kStage >> 4);
#pragma unroll
          for (int c = 0; c < Cfg::kAcc; ++c) {
            if (c < accs) {
#pragma unroll
              for (int kb = 0; kb < 4; ++kb) {
                const uint64_t da = ((uint64_t)hi << 32) | (lo + c * (Cfg::kBytesW >> 4) + 2 * kb);
                const uint64_t db = ((uint64_t)hi << 32) | (lo + (Cfg::kBytesA >> 4) + 2 * kb);
                mma2_f16(tmem + (b0 + c) * BN, da, db, idesc, kb == 0 ? accumulate : 1u);
              }
            }
          }
          tc2_commit(&empty[s]);
        }
        accumulate = 1;
        advance();
      }
      for (int c = 0; c < accs; ++c) {
        if (lane == 0) tc2_commit(&tfull[b0 + c]);
        ++uses[b0 + c];
      }
      ++seg;
    }
  } else if (warp < 2 + kGtTokenWarps) {
    const int tl = lane * kGtTokenWarps + (warp - 2);
    const uint32_t bar0 = map_rank(&full[0], 0);
    // rows 4 tl .. 4 tl + 3 of this CTA's tokens by permutation (past the tile its last row again);
    // a unit's entries are loaded under the copies of the one before it
    int f[4] = {0, 0, 0, 0};
    GtTile un = {};
    const auto look_up = [&](int tile) {
      un = gt_tile<BN>(tile, s_tile, s_off, s_cnt, Cfg::kSorts ? s_expert : nullptr, lane);
      if (p.c.perm != nullptr) {
        const int first = un.p0 + (int)rank * un.nhalf + 4 * tl;
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = p.c.perm[min(first + i, un.p0 + un.n - 1)];
      }
    };
    // A warp may have no copy in a unit, and then nothing waits for it: it goes by the weight warp's
    // count of empty stages, which the copies of every fill follow, and not by the barriers' parities
    // (a warp two phases behind or ahead would take the wrong one).
    int fill = 0;                    // fills before this unit
    bool more = work.next(u, tile, rb, k0, len);
    if (more) look_up(tile);
    while (ok && more) {
      int4 rows = make_int4(0, 0, 0, 0);
      const bool gathers = p.c.perm != nullptr && 4 * tl < un.nhalf;
      const bool copies = p.c.perm == nullptr && tl * Cfg::kChunk < un.nhalf;
      if (gathers) {
        int r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          r[i] = f[i] < 0 ? -1 : f[i] / p.c.topk;
          if (r[i] < 0 || r[i] >= p.c.x_rows) {
            set_error(err, kErrRouteBounds);
            r[i] = 0;
          }
        }
        rows = make_int4(r[0], r[1], r[2], r[3]);
      }
      const int first = un.p0 + (int)rank * un.nhalf + tl * Cfg::kChunk;
      const bool active = __any_sync(0xffffffffu, gathers || copies);
      const int x0 = k0 * kGtK, steps = len;
      more = work.next(u, tile, rb, k0, len);
      if (more) look_up(tile);
      if (active) {
        s = fill % S;
        for (int i = 0; i < steps; ++i) {
          if (!wait_count_warp(s_fills, fill + i + 1, err)) {
            ok = false;
            break;
          }
          uint8_t* bs = st + s * Cfg::kStage + Cfg::kBytesA;
          const int x = x0 + i * kGtK;
          if (gathers) tma2_gather4(bs + tl * 512, &p.tm_x, x, rows, bar0 + 8 * s);
          if (copies) tma2_load_2d(bs + tl * Cfg::kChunk * 128, &p.tm_x, x, first, bar0 + 8 * s);
          if (++s == S) s = 0;
        }
      }
      fill += steps;
    }
  } else {
    // two groups of four warps, one per accumulator buffer
    const int q = warp & 3, g = (warp - 2 - kGtTokenWarps) >> 2;
    const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16) + g * BN;
    const uint32_t bempty = map_rank(&tempty[g], 0);
    uint32_t uses = 0;
    const auto sync_group = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(1 + g) : "memory"); };
    for (int seg = 0; ok && work.next(u, tile, rb, k0, len); ++seg) {
      if (Cfg::kAcc == 2 ? g >= accs_of(rb) : (seg & 1) != g) continue;
      const GtTile un = gt_tile<BN>(tile, s_tile, s_off, s_cnt, Cfg::kSorts ? s_expert : nullptr, lane);
      const int acc = Cfg::kAcc == 2 ? g : 0;
      const int col0 = unit_col(rb) + acc * 2 * kRows + (int)rank * kRows;
      ok = mbar_wait_warp(&tfull[g], uses & 1, err);
      ++uses;
      float v[32];
      if (len == p.KT) {               // no named barrier from here on: pieces come first
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int c0 = 0; c0 < un.n; c0 += 32) {
          tmem_ld32(trow + c0, v);
          gt_store<T, ACT>(p, v, un, col0, c0, q, lane);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(bempty);
      } else {
        // one verdict for the four warps: all of them reach the named barriers below, or none
        if (lane == 0) s_warp[4 * g + q] = ok;
        sync_group();
        ok = s_warp[4 * g] && s_warp[4 * g + 1] && s_warp[4 * g + 2] && s_warp[4 * g + 3];
        if (!ok) break;
        tc_fence_after();
        const size_t stride = (size_t)2 * Cfg::kAcc * BN * 128;     // floats of one slot
        const size_t at = (size_t)(rank * Cfg::kAcc + acc) * BN * 128 + q * 32 + lane;
        float* mine = p.part + (size_t)work.slot_of(pair, u) * stride + at;
#pragma unroll 1
        for (int c0 = 0; c0 < un.n; c0 += 32) {
          tmem_ld32(trow + c0, v);
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (c0 + j < un.n) __stcg(mine + (size_t)(c0 + j) * 128, v[j]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(bempty);
        sync_group();
        int c_lo, c_hi;
        work.owners(u, c_lo, c_hi);
        if (q == 0 && lane == 0) {
          __threadfence();                              // the group's sums, ordered by its barrier
          int32_t* ticket = p.tickets + 4 * (u - work.first) + 2 * rank + acc;
          const int last = atomicAdd(ticket, 1) == c_hi - c_lo;
          if (last) *ticket = 0;                        // ready for the next call
          __threadfence();
          s_flag[g] = last;
        }
        sync_group();
        if (s_flag[g]) {
          if (un.n <= 8) {
            // few tokens: the sums of four pieces in flight at a time (one token top-8, fc1 of the
            // E = 256 layer: 24.8 -> 21.8 us, most of it here, the rest by writing n columns only)
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = 0.f;
            for (int c = c_lo; c <= c_hi; c += 4) {
              float t[4][8];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float* src = p.part + (size_t)work.slot_of(min(c + i, c_hi), u) * stride + at;
#pragma unroll
                for (int j = 0; j < 8; ++j) t[i][j] = __ldcg(src + (size_t)min(j, un.n - 1) * 128);
              }
#pragma unroll
              for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] += c + i <= c_hi ? t[i][j] : 0.f;
            }
            gt_store<T, ACT>(p, v, un, col0, 0, q, lane);
          } else {
#pragma unroll 1
            for (int c0 = 0; c0 < un.n; c0 += 32) {
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = 0.f;
#pragma unroll 2
              for (int c = c_lo; c <= c_hi; ++c) {
                const float* src = p.part + (size_t)work.slot_of(c, u) * stride + at;
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] += __ldcg(src + (size_t)(c0 + j) * 128);
              }
              gt_store<T, ACT>(p, v, un, col0, c0, q, lane);
            }
          }
        }
        sync_group();                                   // s_flag and s_warp read by all
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();        // no CTA leaves while the other may still signal it
  tc_fence_after();
  if (warp == 3) tmem2_dealloc(tmem, Cfg::kCols);
}

// ---------------------------------------------------------------------------------- host side

// Token-tile width by the mean positions per expert (of S, dropped slots among them: the rows that
// belong here are known on the device only; a rank of eight may get a tile up to eight times as wide
// as its rows ask for, 2-4 % by the table): an expert should be one tile while HBM is the
// bound (its weights pass an SM pair once per tile), and a narrower tile leaves more of the shared
// memory to weights in flight.  E = 256, K = 6144, N = 1024, SwiGLU, us at widths 32 / 64 / 128 /
// 256: mean 8: 469 / 471 / 481 / 488;  24: 484 / 478 / 488 / 495;  48: 778 / 493 / 500 / 503;  64:
// 968 / 591 / 508 / 509;  96: 1346 / 780 / 522 / 521;  128: 1722 / 971 / 696 / 534.
int grouped_tc_bn(int S, int E) {
  if ((long long)S <= 8LL * E) return 32;
  if ((long long)S <= 24LL * E) return 64;
  if ((long long)S <= 64LL * E) return 128;
  return 256;
}

size_t grouped_tc_part_bytes(int S, int E) {
  const int bn = grouped_tc_bn(S, E);
  return (size_t)kGtMaxPairs * 2 * 2 * (bn > 128 ? 2 : 1) * bn * 128 * sizeof(float);
}

static bool gt_tmap(CUtensorMap* tm, bool bf16, int rank, const void* base, const cuuint64_t* dims,
                    const cuuint64_t* strides, const cuuint32_t* box) {
  EncodeTiledFn enc = tc_encode_fn();
  if (!enc) return false;
  const cuuint32_t es[5] = {1, 1, 1, 1, 1};
  return enc(tm, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
             (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, bool ACT, int BN, int ACC = 1>
static cudaError_t launch_gt(GtParams& p, cudaStream_t st) {
  using Cfg = GtCfg<BN, ACC>;
  auto kernel = grouped_tc_kernel<T, ACT, BN, ACC>;
  static PerDevice<int> per;
  int pairs = 0;
  cudaError_t err = on_device(per, &pairs, [&](int* v) {
    cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t q = {};
    q.gridDim = dim3(2 * kGtMaxPairs);
    q.blockDim = dim3(kGtThreads);
    q.dynamicSmemBytes = Cfg::kSmem;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, kernel, &q);
    *v = n < 1 ? 1 : (n < kGtMaxPairs ? n : kGtMaxPairs);
    return e;
  });
  if (err != cudaSuccess) return err;
  const bool bf16 = std::is_same<T, __nv_bfloat16>::value;
  const GroupedDims& d = p.d;
  const GroupedCall& c = p.c;
  bool ok;
  p.whole16 = ACT && (d.N / 2) % 16 == 0;
  if (p.whole16) {
    // [E][I / 16 groups][2 halves][16 rows][K]
    const cuuint64_t dims[5] = {(cuuint64_t)d.K, 16, 2, (cuuint64_t)(d.N / 32), (cuuint64_t)d.E};
    const cuuint64_t row = (cuuint64_t)c.ldw * 2;
    const cuuint64_t str[4] = {row, row * (d.N / 2), row * 16, row * d.N};
    const cuuint32_t box[5] = {kGtK, 16, 2, 4, 1};
    ok = gt_tmap(&p.tm_w, bf16, 5, c.w, dims, str, box);
  } else if (ACT) {
    const cuuint64_t dims[4] = {(cuuint64_t)d.K, (cuuint64_t)(d.N / 2), 2, (cuuint64_t)d.E};
    const cuuint64_t str[3] = {(cuuint64_t)c.ldw * 2, (cuuint64_t)c.ldw * d.N, (cuuint64_t)c.ldw * d.N * 2};
    const cuuint32_t box[4] = {kGtK, 16, 2, 1};
    ok = gt_tmap(&p.tm_w, bf16, 4, c.w, dims, str, box);
  } else {
    const cuuint64_t dims[3] = {(cuuint64_t)d.K, (cuuint64_t)d.N, (cuuint64_t)d.E};
    const cuuint64_t str[2] = {(cuuint64_t)c.ldw * 2, (cuuint64_t)c.ldw * d.N * 2};
    const cuuint32_t box[3] = {kGtK, 128, 1};
    ok = gt_tmap(&p.tm_w, bf16, 3, c.w, dims, str, box);
  }
  const cuuint64_t xdims[2] = {(cuuint64_t)d.K, (cuuint64_t)(c.perm ? c.x_rows : c.S)};
  const cuuint64_t xstr[1] = {(cuuint64_t)c.ldx * 2};
  const cuuint32_t xbox[2] = {kGtK, c.perm ? 1u : (cuuint32_t)Cfg::kChunk};
  ok = ok && gt_tmap(&p.tm_x, bf16, 2, c.x, xdims, xstr, xbox);
  if (!ok) return cudaErrorInvalidValue;
  const int blocks = cdiv(p.cols, ACT ? 128 : 256);
  p.RB = blocks / Cfg::kAcc;
  p.half = blocks % Cfg::kAcc;
  // no more pairs than K steps can keep busy
  const long long units = ((long long)cdiv(c.S, BN) + (d.E < c.S ? d.E : c.S)) * (p.RB + p.half);
  const long long useful = units * (p.KT < kGtMinSteps ? 1 : cdiv(p.KT, kGtMinSteps));
  const int G = useful < pairs ? (int)useful : pairs;
  return launch_kernel(kernel, dim3(2 * G), dim3(kGtThreads), Cfg::kSmem, st, true, p);
}

template <typename T, bool ACT>
static cudaError_t launch_gt_bn(GtParams& p, cudaStream_t st) {
  // expected units of two accumulators, against the pairs of a whole GPU
  const long long tiles = cdiv(p.c.S, 256) + (p.d.E < p.c.S ? p.d.E : p.c.S) / 2;
  const bool few = tiles * cdiv(p.cols, ACT ? 256 : 512) < 60;
  switch (grouped_tc_bn(p.c.S, p.d.E)) {
    case 32: return launch_gt<T, ACT, 32>(p, st);
    case 64: return launch_gt<T, ACT, 64>(p, st);
    case 128: return launch_gt<T, ACT, 128>(p, st);
    // 256 tokens.  One accumulator, double-buffered, where units of two would leave pairs idle (256
    // rows over 2 experts, K = N = 4096: 27 us against 49; 4000 over 16, K = N = 512: 11.6 against
    // 14.7), and where the tokens are in place and K is short: the exposed epilogue of two weighs
    // more than the traffic it saves (24,576 rows over 16 experts, f16: K = 512 147 -> 135 us, 3584
    // 481 -> 454, but 7168 487 -> 501).  Two accumulators otherwise: with one, the row gathers are
    // the bound (K = 1152 318 against 385 us, 7168 480 against 627).
    default:
      return few || (p.c.perm == nullptr && p.KT <= 64) ? launch_gt<T, ACT, 256, 1>(p, st)
                                                        : launch_gt<T, ACT, 256, 2>(p, st);
  }
}

// Whether the tile copies can address the operands: 16-byte bases and strides.
bool grouped_tc_addressable(const GroupedDims& d, const GroupedCall& c) {
  const auto on16 = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0; };
  return on16(c.x) && on16(c.w) && c.ldx % 8 == 0 && c.ldw % 8 == 0 && c.ldx < (1LL << 38) &&
         c.ldw * d.N < (1LL << 38);
}

cudaError_t launch_grouped_tc(const GroupedDims& d, const GroupedCall& c, float* part,
                              int32_t* tickets, cudaStream_t st) {
  GtParams p;
  p.d = d;
  p.c = c;
  p.part = part;
  p.tickets = tickets;
  p.KT = cdiv(d.K, kGtK);
  p.cols = grouped_cols(d);
  p.packed = p.cols % 2 == 0 && c.ldo % 2 == 0 && (reinterpret_cast<uintptr_t>(c.out) & 3) == 0;
  if (d.dtype == MOE_DTYPE_F16)
    return d.act ? launch_gt_bn<__half, true>(p, st) : launch_gt_bn<__half, false>(p, st);
  return d.act ? launch_gt_bn<__nv_bfloat16, true>(p, st) : launch_gt_bn<__nv_bfloat16, false>(p, st);
}

}  // namespace moe
