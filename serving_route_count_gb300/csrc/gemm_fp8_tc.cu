// gemm_fp8_tc.cu - 8-bit products with block scales on the tensor cores (moe_fp8_run), dense or grouped
// by expert: out[p] = act(sum over blocks b of 128 of x_scale * w_scale * (W[e] . x[row(p)])_b).
//
// The schedule, the loads and the roles are the 16-bit grouped products' (gemm_grouped_tc.cu): a pair of
// CTAs (tcgen05 cta_group::2) owns a unit of 256 weight rows x up to BN tokens of one expert.  The scales
// are fp32, so they cannot ride in the MMA: a K step is one block of 128 values (one 128-byte swizzled row),
// its product goes to a tensor-memory buffer of its own, and the epilogue warps take it out and add it,
// times both scales, to sums in registers, under the MMAs of the next steps.
//
// Two forms, by the tile's tokens:
//   up to 128: weight rows are the MMA's M operand and tokens its N operand, so one token still streams its
//     weights through full-size MMAs.  A lane holds one weight row; the tokens' scales (times the
//     row's) pass through shared memory, four steps at a time, from two warps of their own.
//   256: tokens are M and weight rows N.  A lane holds one token and 128 weight rows, all of one scale (two for
//     a SwiGLU), so a step costs it one factor and 64 packed FMAs; with the scales read from shared
//     memory, as above, those reads and the MMA's operands would share its bandwidth at par.
// The sums of an epilogue thread (up to 128) and what it has in flight need 184 or 208 registers: the other
// warps give theirs up (setmaxnreg).  The compiler, which shares out 128 for all roles, spills a few words of the widths
// 128 and 256 (4 to 32 bytes stored, 12 to 36 loaded); whether inside a step is not known.
//
// Bounds and measurements (GB300, HBM at the measured 6784 GB/s, e4m3 at twice the measured bf16 rate):
//   up projections + SwiGLU of 8 tokens top-8, E = 256, K = 6144, N = 1024: 63 to 70 us, HBM floor 53; down projections
//   of 16 tokens top-6, E = 384, K = 576, N = 7168: 81 to 88 us, floor 52 - the start (tables 2 us, first loads 2.5),
//   units of five steps, their stores (76 us without) and 128-byte copies of 576-byte rows;
//   2048 tokens top-8, skewed: 395 us, floor 241: bound by the epilogue's handling of a step at 128 tokens (272
//   with the MMAs and copies alone), which takes the tile's whole width however few rows it holds;
//   8192 x 7168 x 7168: 453 us, 1.86 PFLOP/s (floor 220; 277 with the MMAs and copies alone, 342 with the loads
//   from tensor memory, the rest the FMAs that do not hide under them).
// What cost most on the way, us of up decode / dense prefill: an arrival with cluster-scope release after the
// tensor-memory loads waited for the scales' global loads, 145 / 883; its CTA-scope form 91 / 575; scales
// from warps of their own and 64 columns in flight 78 / 443.
//
// Roles: warp 0 weight copies, warp 1 MMA issue (leader CTA), warps 2-5 or 2-6 token copies (tiles, or
// gathers of four rows by index; warp 3 also allocates the tensor memory, warp 2 asks for the next
// unit's weight scales), the others up to warp 7 scales and units, warps 8-15 epilogue.
#include <type_traits>

#include "block_ops.cuh"
#include "fp8.cuh"
#include "tc_pair.cuh"
#include "tc_tile.cuh"
#include "tc_units.cuh"
#include "../../include/moe_gb300.h"

namespace moe {
using namespace tc;

constexpr int kF8Threads = 512;
constexpr int kF8K = kFp8Block;          // K step: one block of scales, one 128-byte swizzled row
constexpr int kF8RegsLaunch = 128;       // of a thread, as ptxas reports and the host checks

// What a slot of scales says of its steps: how many (0: the work is over), whether the unit ends with them,
// and the unit: first position, positions, positions of a CTA, weight row block, number, whether it is a piece,
// expert, first step.
enum { kF8Steps, kF8Last, kF8P0, kF8N, kF8Half, kF8Rb, kF8Unit, kF8Piece, kF8Expert, kF8K0, kF8Head };

template <int BN, bool ACT>
struct F8Cfg {
  static constexpr bool kTokenRows = BN == 256;              // tokens are the MMA's M operand
  // registers shared out anew by role: a thread's of the epilogue warps and of the others
  static constexpr int kRegsMore = BN == 256 ? 208 : 184, kRegsLess = 256 - kRegsMore;
  static_assert(256 * (kRegsMore + kRegsLess) <= kF8Threads * kF8RegsLaunch, "register split");
  static constexpr int kHalf = BN / 2;                       // tokens a CTA loads
  static constexpr int kChunk = kHalf < 32 ? kHalf : 32;     // tokens per tile copy
  static constexpr int kBytesW = 128 * 128, kBytesB = kHalf * 128, kStage = kBytesW + kBytesB;
  static constexpr int kBuffers = BN == 256 ? 2 : 4;         // tensor-memory buffers of a step
  static constexpr int kTurn = kTokenRows ? 1 : 2;           // steps that change hands together
  static constexpr int kTurns = kBuffers / kTurn;
  static constexpr int kCols = kBuffers * BN;                // tensor-memory columns
  static constexpr int kGroups = BN == 32 ? 1 : 2;           // groups of four epilogue warps
  static constexpr int kWide = BN == 32 ? 32 : BN / 2;       // accumulator columns of a group
  static constexpr int kSets = ACT ? 2 : 1;                  // scales of a lane's column: up and gate
  static constexpr int kTokenWarps = kTokenRows ? 5 : 4;     // from warp 2 on
  static constexpr int kScaleWarps = 6 - kTokenWarps;        // the ones after them
  // ring of scales: slots of four steps, each [sets][kPad] of the tokens' columns (times the rows'; both
  // sets' words in other banks), and what they belong to; tokens as M: that alone, a slot for each unit
  static constexpr int kPad = BN + 4, kStep = kTokenRows ? 0 : kSets * kPad;
  static constexpr int kSlots = 3, kSlot = 4 * kStep, kScales = kSlots * (kSlot + kF8Head) * 4;
  static constexpr int kTables = 3 * 1028 * 4 + 512 + kScales;
  static constexpr int kStages = (227 * 1024 - 1024 - kTables) / kStage > 12
                                     ? 12 : (227 * 1024 - 1024 - kTables) / kStage;
  static constexpr int kSmem = 1024 + kStages * kStage + kTables;
};

struct F8Params {
  CUtensorMap tm_w, tm_x;
  GroupedDims d;
  GroupedCall c;
  const float* xs;
  const float* ws;
  long long ldxs;
  float* part;          // [pairs][2][2 CTAs][BN / 4][128][4]
  int32_t* tickets;     // [pairs][2 CTAs][2 groups]
  int KT, RB, cols, tall;
  int fix_steps;        // K steps that cutting the leftover units has to save (GtWork)
  int packed, vec;      // output rows on 4 bytes, on 16
  int whole16;          // SwiGLU weights by whole 16-row groups: one 5-d copy per K step
};

// Asks for the scales of the next unit's weight rows (up to four rows of KT) in L2: from DRAM under load
// they would take longer than the steps that a fetch is ahead.
__device__ __forceinline__ void f8_prefetch(const float* row, int n, int line) {
  const char* at = reinterpret_cast<const char*>(reinterpret_cast<uintptr_t>(row) & ~(uintptr_t)127) + 128 * line;
  if (at < reinterpret_cast<const char*>(row + n)) asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
}

// Stores a lane's outputs of 32 accumulator columns, tokens in lanes: columns col0 .. of row `row`.
template <typename T, bool ACT>
__device__ __forceinline__ void f8_store_row(const F8Params& p, const float (&x)[32], long long row, int col0) {
  T* o = static_cast<T*>(p.c.out) + row * p.c.ldo + col0;
  const bool up_first = p.d.layout == MOE_W13_UP_GATE;
#pragma unroll
  for (int c = 0; c < (ACT ? 16 : 32); c += 8) {
    T v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (ACT) {             // half 0 in the first 16 columns, half 1 in the others
        const float a = x[c + j], b = x[16 + c + j];
        v[j] = from_f32<T>(swiglu_f32(up_first ? a : b, up_first ? b : a, p.d.limit, p.d.alpha, p.d.beta));
      } else {
        v[j] = from_f32<T>(x[c + j]);
      }
    }
    const int left = p.cols - col0 - c;
    if (p.vec) {
      if (left > 0) {
        uint4 w;
        memcpy(&w, v, 16);
        *reinterpret_cast<uint4*>(o + c) = w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < left) o[c + j] = v[j];
    }
  }
}

template <typename T, bool ACT, int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kF8Threads, 1)
fp8_tc_kernel(const __grid_constant__ F8Params p) {
  using Cfg = F8Cfg<BN, ACT>;
  constexpr int S = Cfg::kStages, TURNS = Cfg::kTurns;
  static_assert(S > Cfg::kBuffers, "phases");
  extern __shared__ uint8_t raw[];
  uint8_t* st = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(st + S * Cfg::kStage);   // [S] (leader's are used)
  // [S] a step has been multiplied: its stage may be filled again, and its product is ready.  The MMAs are at
  // most kBuffers < S steps ahead of the epilogue, so no phase passes that it has not waited for.
  uint64_t* done = full + S;
  uint64_t* tempty = done + S;         // [TURNS] a turn's products have been read (leader's are used)
  uint64_t* sfull = tempty + TURNS;       // [slots] scales of four steps are there
  uint64_t* sempty = sfull + Cfg::kSlots;   // [slots] and have been read
  uint64_t* gbar = sempty + Cfg::kSlots;    // [2] the four warps of an epilogue group
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(gbar + 2);
  int* s_flag = reinterpret_cast<int*>(s_tmem + 1);   // [2]
  int* s_total = s_flag + 2;           // tiles of the call
  int* s_warp = s_total + 1;           // [warps]
  int* s_fills = s_warp + kF8Threads / 32;   // fills whose stage the weight warp has found empty
  int* s_off = reinterpret_cast<int*>(st + S * Cfg::kStage + 512);
  int* s_cnt = s_off + 1028;
  int* s_tile = s_cnt + 1028;
  float* s_scale = reinterpret_cast<float*>(s_tile + 1028);   // [slots][4][kStep]
  int* s_head = reinterpret_cast<int*>(s_scale + Cfg::kSlots * Cfg::kSlot);   // [slots][kF8Head]
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
      mbar_init(&done[s], 1);
    }
    for (int b = 0; b < TURNS; ++b) {
      mbar_init(&tempty[b], 8 * Cfg::kGroups);        // the epilogue warps of both CTAs
    }
    for (int b = 0; b < Cfg::kSlots; ++b) {
      mbar_init(&sfull[b], Cfg::kScaleWarps);
      mbar_init(&sempty[b], 4 * Cfg::kGroups);
    }
    for (int g = 0; g < 2; ++g) mbar_init(&gbar[g], 4);
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
  int total = gt_number<BN, kF8Threads>(cnt, E, s_tile, s_warp);
  if (bad) {
    total = 0;
    if (tid == 0) set_error(err, kErrRouteBounds);
  }
  if (tid == 0) *s_total = total;
  // rows past the last group
  if (p.c.offsets != nullptr) {
    const int end = max(0, min(p.c.S, p.c.offsets[E]));
    T* out = static_cast<T*>(p.c.out);
    for (long long r = end + (long long)blockIdx.x; r < p.c.S; r += gridDim.x)
      for (int c = tid; c < p.cols; c += kF8Threads) out[r * p.c.ldo + c] = from_f32<T>(0.f);
  }
  __syncthreads();

  // Every loop below is taken by whole warps; one lane issues.
  constexpr int kRows = ACT ? 64 : 128;      // output columns of one CTA's weight rows
  GtWork work;
  work.init(total, p.KT, p.RB, 0, G, pair, p.fix_steps, false);
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
  const auto tile_at = [&](int tile) { return gt_tile<BN>(tile, s_tile, s_off, s_cnt, nullptr, lane); };
  // row of x at position pos; a bad entry sets the error word where its row is copied
  const auto row_of = [&](int pos) {
    if (p.c.perm == nullptr) return pos;
    const int f = p.c.perm[pos], r = f < 0 ? 0 : f / p.c.topk;
    return r < p.c.x_rows ? r : 0;
  };
  // scales of set h of weight rows r .. of one tile row (a row past the matrix takes its last tile's)
  const auto scales_of = [&](int e, int h, int r) {
    const int half = p.tall / Cfg::kSets;
    return p.ws + ((size_t)e * p.tall + h * half + min(r / kFp8Block, half - 1)) * p.KT;
  };
  // the ring of scales, by the warps that fill it
  int slot = 0;
  uint32_t turn = 0;
  const auto head = [&](const GtTile& un, int steps, bool last) {
    int* h = s_head + slot * kF8Head;
    h[kF8Steps] = steps;
    h[kF8Last] = last;
    h[kF8P0] = un.p0;
    h[kF8N] = un.n;
    h[kF8Half] = un.nhalf;
    h[kF8Rb] = rb;
    h[kF8Unit] = u;
    h[kF8Piece] = len != p.KT;
    h[kF8Expert] = un.e;
    h[kF8K0] = k0;
  };
  const auto publish = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sfull[slot]);
    if (++slot == Cfg::kSlots) {
      slot = 0;
      ++turn;
    }
  };
  if (warp < 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::kRegsLess));
    if (warp == 0) {
      const uint32_t bar0 = map_rank(&full[0], 0);
      while (ok && work.next(u, tile, rb, k0, len)) {
        const GtTile un = tile_at(tile);
        const int rows = p.c.perm != nullptr ? un.nhalf : cdiv(un.nhalf, Cfg::kChunk) * Cfg::kChunk;
        const uint32_t bytes = 2u * (Cfg::kBytesW + rows * 128);
        const int r = (2 * rb + (int)rank) * kRows;
        for (int x = k0 * kF8K; x < (k0 + len) * kF8K; x += kF8K, ++issued) {
          if (!mbar_wait_warp(&done[s], phase ^ 1, err)) {
            ok = false;
            break;
          }
          if (lane == 0) {
            publish_count(s_fills, issued + 1);
            const uint32_t bar = bar0 + 8 * s;
            if (rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
            uint8_t* a = st + s * Cfg::kStage;
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
          advance();
        }
      }
      if (lane == 0) {
        // the last fills have been multiplied: nothing arrives at this CTA's barriers any more
        for (int j = max(0, issued - S); ok && j < issued; ++j)
          ok = mbar_wait(&done[j % S], (j / S) & 1, err);
        if (!ok && rank == 0) drain_stage_loads<S>(full, issued, err);
      }
    } else if (warp == 1) {
      // operand descriptors: only the address changes from stage to stage and from K block to K block
      const uint64_t desc0 = desc_sw128(st);
      const uint32_t hi = (uint32_t)(desc0 >> 32), lo0 = (uint32_t)desc0;
      uint32_t hand = 0;               // turns that have gone to tensor memory
      bool ready = false;              // the next step's operands and buffer are known to be
      // nothing commits to this phase before the first step's MMAs
      if (p.d.probe_ns != 0 && blockIdx.x == 0)
        ok = __all_sync(0xffffffffu, mbar_wait(&done[0], 0, err, p.d.probe_ns));
      while (rank == 0 && ok && work.next(u, tile, rb, k0, len)) {
        const GtTile un = tile_at(tile);
        const uint32_t idesc = idesc_pair8(Cfg::kTokenRows ? 256 : 2 * un.nhalf);
        for (int i = 0; i < len; ++i) {
          const uint32_t b = hand % TURNS;
          if (!ready) {
            if (i % Cfg::kTurn == 0)
              ok = mbar_wait2_warp(&tempty[b], ((hand / TURNS) & 1) ^ 1, &full[s], phase, err);
            else
              ok = mbar_wait_warp(&full[s], phase, err);
          }
          if (!ok) break;
          tc_fence_after();
          // the next step, of this unit or another
          const bool end = i % Cfg::kTurn == Cfg::kTurn - 1 || i + 1 == len;     // of the turn
          const uint32_t s1 = s + 1 == S ? 0 : s + 1, h1 = hand + 1;
          const bool next = mbar_test(&full[s1], phase ^ (s1 == 0)) &&
                            (!end || mbar_test(&tempty[h1 % TURNS], ((h1 / TURNS) & 1) ^ 1));
          if (elect_one()) {
            const uint32_t lo = lo0 + s * (Cfg::kStage >> 4);
#pragma unroll
            for (int kb = 0; kb < 4; ++kb) {
              const uint64_t dw = ((uint64_t)hi << 32) | (lo + 2 * kb);
              const uint64_t dx = ((uint64_t)hi << 32) | (lo + (Cfg::kBytesW >> 4) + 2 * kb);
              mma2_f8(tmem + (b * Cfg::kTurn + i % Cfg::kTurn) * BN, Cfg::kTokenRows ? dx : dw, Cfg::kTokenRows ? dw : dx, idesc, kb != 0);
            }
            tc2_commit(&done[s]);
          }
          advance();
          hand += end;
          ready = __all_sync(0xffffffffu, next);
        }
      }
    } else if (warp < 2 + Cfg::kTokenWarps) {
      const int tl = lane * Cfg::kTokenWarps + (warp - 2);
      const uint32_t bar0 = map_rank(&full[0], 0);
      // rows 4 tl .. 4 tl + 3 of this CTA's tokens by permutation (past the tile its last row again);
      // a unit's entries are loaded under the copies of the one before it
      int f[4] = {0, 0, 0, 0};
      GtTile un = {};
      const auto look_up = [&](int tile) {
        un = tile_at(tile);
        if (p.c.perm != nullptr) {
          const int first = un.p0 + (int)rank * un.nhalf + 4 * tl;
#pragma unroll
          for (int i = 0; i < 4; ++i) f[i] = p.c.perm[min(first + i, un.p0 + un.n - 1)];
        }
        if (warp == 2) {
          const int h = (lane >> 3) & 1, of = lane >> 4;   // set, and the CTA whose weight rows (tokens as M: both)
          if (h < Cfg::kSets && (Cfg::kTokenRows || of == (int)rank))
            f8_prefetch(scales_of(un.e, h, (2 * rb + of) * kRows) + k0, len, lane & 7);
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
        const int x0 = k0 * kF8K, steps = len;
        more = work.next(u, tile, rb, k0, len);
        if (more) look_up(tile);
        if (active) {
          s = fill % S;
          for (int i = 0; i < steps; ++i) {
            if (!wait_count_warp(s_fills, fill + i + 1, err)) {
              ok = false;
              break;
            }
            uint8_t* bs = st + s * Cfg::kStage + Cfg::kBytesW;
            const int x = x0 + i * kF8K;
            if (gathers) tma2_gather4(bs + tl * 512, &p.tm_x, x, rows, bar0 + 8 * s);
            if (copies) tma2_load_2d(bs + tl * Cfg::kChunk * 128, &p.tm_x, x, first, bar0 + 8 * s);
            if (++s == S) s = 0;
          }
        }
        fill += steps;
      }
    } else if constexpr (Cfg::kTokenRows) {
      // tokens as M: units alone, the epilogue warps fetch their few scales themselves
      while (ok && work.next(u, tile, rb, k0, len)) {
        const GtTile un = tile_at(tile);
        ok = mbar_wait_warp(&sempty[slot], (turn & 1) ^ 1, err);
        if (!ok) break;
        if (lane == 0) head(un, len, true);
        publish();
      }
      if (ok && mbar_wait_warp(&sempty[slot], (turn & 1) ^ 1, err)) {
        if (lane == 0) s_head[slot * kF8Head + kF8Steps] = 0;
        publish();
      }
    } else {
      // Scales of the tokens' columns: warp 6 columns 0 .. 31 and 64 .. 95, warp 7 the others.  Those of the next
      // four steps, of the next unit too, are on their way while these wait for their slot.
      constexpr int M = (BN + 63) / 64, SETS = Cfg::kSets;
      const int c0 = (warp - 6) * 32 + lane;
      float nx[M][4], nw[SETS][4];
      const float* xs[M];
      const float* w[SETS];
      GtTile un = {};
      int i0 = 0, n = 0;
      len = 0;
      const auto fetch = [&]() {         // steps of the block that it asks for, 0 at the end
        i0 += n;
        if (i0 >= len) {
          if (!work.next(u, tile, rb, k0, len)) return 0;
          un = tile_at(tile);
#pragma unroll
          for (int m = 0; m < M; ++m)
            xs[m] = p.xs + row_of(un.p0 + min(c0 + 64 * m, un.n - 1)) * p.ldxs + k0;
#pragma unroll
          for (int h = 0; h < SETS; ++h) w[h] = scales_of(un.e, h, (2 * rb + (int)rank) * kRows) + k0;
          i0 = 0;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = min(i0 + j, len - 1);
#pragma unroll
          for (int m = 0; m < M; ++m) nx[m][j] = xs[m][i];
#pragma unroll
          for (int h = 0; h < SETS; ++h) nw[h][j] = w[h][i];
        }
        return min(4, len - i0);
      };
      n = fetch();
      while (ok) {
        ok = mbar_wait_warp(&sempty[slot], (turn & 1) ^ 1, err);
        if (!ok) break;
        if (warp == 6 && lane == 0) head(un, n, i0 + 4 >= len);
        if (n == 0) {
          publish();
          break;
        }
        float now[M][SETS][4];
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
          for (int h = 0; h < SETS; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j) now[m][h][j] = nx[m][j] * nw[h][j];
        n = fetch();
        float* to = s_scale + slot * Cfg::kSlot + c0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int h = 0; h < SETS; ++h)
#pragma unroll
            for (int m = 0; m < M; ++m)
              if (c0 + 64 * m < BN) to[j * Cfg::kStep + h * Cfg::kPad + 64 * m] = now[m][h][j];
        publish();
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Cfg::kRegsMore));
    // Groups of four warps share the columns of every step.  They follow the slots of scales, which say where
    // units end; nothing of the schedule is kept in their registers.
    constexpr int CW = Cfg::kWide, SETS = Cfg::kSets;
    const int q = warp & 3, g = (warp - 8) >> 2, t = q * 32 + lane;
    const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16) + g * CW;
    const uint32_t bempty = map_rank(&tempty[0], 0);
    uint32_t hand = 0, at = 0, syncs = 0;
    int j = 0, steps = 0;              // in the slot
    uint64_t acc[CW / 2];
    uint32_t v[2][32];
    const auto clear = [&]() {
#pragma unroll
      for (int c = 0; c < CW / 2; ++c) acc[c] = 0;
    };
    // the group's four warps, with a bound like every wait
    const auto sync_group = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(&gbar[g]);
      return mbar_wait_warp(&gbar[g], syncs++ & 1, err);
    };
    // the next slot of scales; false at the end of the work
    const auto open = [&]() {
      if (!mbar_wait_warp(&sfull[slot], turn & 1, err)) return false;
      steps = s_head[slot * kF8Head + kF8Steps];
      j = 0;
      return steps > 0;
    };
    // the slot's scales have been read
    const auto leave = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(&sempty[slot]);
      if (++slot == Cfg::kSlots) {
        slot = 0;
        ++turn;
      }
    };
    // the products of the next turn, of one step or two
    const auto begin = [&](int n) {
      if (n == 2) advance();
      if (!mbar_wait_warp(&done[s], phase, err)) return false;
      advance();
      tc_fence_after();
      at = trow + (hand % TURNS) * (Cfg::kTurn * BN);
      return true;
    };
    // the turn's buffers have been read
    const auto release = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_read(bempty + 8 * (hand % TURNS));
      ++hand;
    };
    // 32 of the group's columns to the output
    const auto store = [&](const int* h, int b, float (&x)[32]) {
      const int n = h[kF8N];
      if constexpr (Cfg::kTokenRows) {
        const int i = (int)rank * h[kF8Half] + t;
        if (t < h[kF8Half] && i < n)
          f8_store_row<T, ACT>(p, x, h[kF8P0] + i, (2 * h[kF8Rb] + g) * kRows + b * (ACT ? 16 : 32));
      } else if (g * CW + 32 * b < n) {
        const GtTile un{0, h[kF8P0], n, h[kF8Half]};
        gt_store<T, ACT>(p, x, un, (2 * h[kF8Rb] + (int)rank) * kRows, g * CW + 32 * b, q, lane);
      }
    };
    // The unit's sums to the output; those of a piece to the scratch buffer, and the piece that arrives last
    // adds them all in K order.
    const auto finish = [&]() {
      const int* h = s_head + slot * kF8Head;
      const int n = h[kF8N];
      if (h[kF8Piece]) {
        GtWork w;
        w.init(*s_total, p.KT, p.RB, 0, gridDim.x >> 1, blockIdx.x >> 1, p.fix_steps, false);
        const int unit = h[kF8Unit];
        // four columns of a lane are adjacent: 16-byte accesses
        const size_t stride = (size_t)2 * BN * 32;       // 16-byte words of one slot of the scratch buffer
        float4* part = reinterpret_cast<float4*>(p.part) + ((size_t)rank * BN + g * CW) * 32 + t;
        float4* mine = part + (size_t)w.slot_of(blockIdx.x >> 1, unit) * stride;
        const int m = Cfg::kTokenRows ? CW : n - g * CW;
#pragma unroll
        for (int c = 0; c < CW / 4; ++c) {
          const float2 lo = unpair_f32(acc[2 * c]), hi = unpair_f32(acc[2 * c + 1]);
          if (4 * c < m) __stcg(mine + c * 128, make_float4(lo.x, lo.y, hi.x, hi.y));
        }
        if (!sync_group()) return false;
        int c_lo, c_hi;
        w.owners(unit, c_lo, c_hi);
        if (t == 0) {
          __threadfence();                               // the group's sums, ordered by its barrier
          int32_t* ticket = p.tickets + 4 * (unit - w.first) + 2 * rank + g;
          const int last = atomicAdd(ticket, 1) == c_hi - c_lo;
          if (last) *ticket = 0;                         // ready for the next call
          __threadfence();
          s_flag[g] = last;                              // read by all before they meet again
        }
        if (!sync_group()) return false;
        if (!s_flag[g]) return true;
#pragma unroll 1
        for (int b = 0; b < CW / 32; ++b) {
          if (32 * b >= m) break;
          float x[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) x[c] = 0.f;
          for (int o = c_lo; o <= c_hi; o += 2) {        // two pieces in flight, added in K order
            float4 y[2][8];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float4* src = part + (size_t)w.slot_of(min(o + k, c_hi), unit) * stride + b * 8 * 128;
#pragma unroll
              for (int c = 0; c < 8; ++c) y[k][c] = __ldcg(src + (32 * b + 4 * c < m ? c : 0) * 128);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const bool there = o + k <= c_hi;
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                x[4 * c] += there ? y[k][c].x : 0.f;
                x[4 * c + 1] += there ? y[k][c].y : 0.f;
                x[4 * c + 2] += there ? y[k][c].z : 0.f;
                x[4 * c + 3] += there ? y[k][c].w : 0.f;
              }
            }
          }
          store(h, b, x);
        }
        return true;
      }
#pragma unroll
      for (int b = 0; b < CW / 32; ++b) {
        float x[32];
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float2 f = unpair_f32(acc[16 * b + c]);
          x[2 * c] = f.x;
          x[2 * c + 1] = f.y;
        }
        store(h, b, x);
      }
      return true;
    };
    clear();
    // A step's columns come 64 at a time: what is in flight at a wait, which takes all of it.
    if constexpr (Cfg::kTokenRows) {
      while (ok && g < Cfg::kGroups && open()) {
        const int* h = s_head + slot * kF8Head;
        const int n = steps;
        const int pos = h[kF8P0] + min((int)rank * h[kF8Half] + t, h[kF8N] - 1);
        const float* xs = p.xs + row_of(pos) * p.ldxs + h[kF8K0];
        const float* w[SETS];
#pragma unroll
        for (int k = 0; k < SETS; ++k) w[k] = scales_of(h[kF8Expert], k, (2 * h[kF8Rb] + g) * kRows) + h[kF8K0];
        // scales of the next two steps are on their way
        float x1 = xs[0], x2 = xs[min(1, n - 1)], w1[SETS], w2[SETS];
#pragma unroll
        for (int k = 0; k < SETS; ++k) {
          w1[k] = w[k][0];
          w2[k] = w[k][min(1, n - 1)];
        }
        for (int i = 0; i < n; ++i) {
          uint64_t f[SETS];
          const int i2 = min(i + 2, n - 1);
#pragma unroll
          for (int k = 0; k < SETS; ++k) {
            const uint32_t b = __float_as_uint(x1 * w1[k]);
            f[k] = pair_f32(b, b);
            w1[k] = w2[k];
            w2[k] = w[k][i2];
          }
          x1 = x2;
          x2 = xs[i2];
          const auto add = [&](int c) {
#pragma unroll
            for (int k = 0; k < 16; ++k)
              fma_pair_f32(acc[16 * c + k], pair_f32(v[c & 1][2 * k], v[c & 1][2 * k + 1]), f[ACT ? k / 8 : 0]);
          };
          ok = begin(1);
          if (!ok) break;
          tmem_ld32_start(at, v[0]);
          tmem_ld32_start(at + 32, v[1]);
          tmem_ld_wait(v[0]);
          tmem_after_wait(v[1]);
          add(0);
          tmem_ld32_start(at + 64, v[0]);
          add(1);
          tmem_ld32_start(at + 96, v[1]);
          tmem_ld_wait(v[0]);
          tmem_after_wait(v[1]);
          release();
          add(2);
          add(3);
        }
        ok = ok && finish();
        clear();
        leave();
      }
    } else {
      ok = g < Cfg::kGroups && open();
      while (ok) {
        const int two = min(2, steps - j);               // steps of this turn
        const float* sc = s_scale + slot * Cfg::kSlot + j * Cfg::kStep + g * CW + (ACT && lane >= 16 ? Cfg::kPad : 0);
        ulonglong2 s4[8];
        const auto scales = [&](int step, int c) {       // of 32 columns
          const ulonglong2* f = reinterpret_cast<const ulonglong2*>(sc + step * Cfg::kStep + 32 * c);
#pragma unroll
          for (int k = 0; k < 8; ++k) s4[k] = f[k];
        };
        const auto add = [&](int c, const uint32_t (&x)[32]) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            fma_pair_f32(acc[16 * c + 2 * k], pair_f32(x[4 * k], x[4 * k + 1]), s4[k].x);
            fma_pair_f32(acc[16 * c + 2 * k + 1], pair_f32(x[4 * k + 2], x[4 * k + 3]), s4[k].y);
          }
        };
        scales(0, 0);
        ok = begin(two);
        if (!ok) break;
        if constexpr (CW == 32) {
          tmem_ld32_start(at, v[0]);
          if (two == 2) tmem_ld32_start(at + BN, v[1]);
          tmem_ld_wait(v[0]);
          tmem_after_wait(v[1]);
          release();
          add(0, v[0]);
          if (two == 2) {
            scales(1, 0);
            add(0, v[1]);
          }
        } else {
          tmem_ld32_start(at, v[0]);
          tmem_ld32_start(at + 32, v[1]);
          tmem_ld_wait(v[0]);
          tmem_after_wait(v[1]);
          if (two == 1) release();
          add(0, v[0]);
          if (two == 2) tmem_ld32_start(at + BN, v[0]);
          scales(0, 1);
          add(1, v[1]);
          if (two == 2) {
            tmem_ld32_start(at + BN + 32, v[1]);
            scales(1, 0);
            tmem_ld_wait(v[0]);
            tmem_after_wait(v[1]);
            release();
            add(0, v[0]);
            scales(1, 1);
            add(1, v[1]);
          }
        }
        j += two;
        if (j == steps) {
          if (s_head[slot * kF8Head + kF8Last]) {
            ok = finish();
            clear();
          }
          leave();
          ok = ok && open();
        }
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

// Scratch of cut units: [pairs][2][2 CTAs][BN][128] fp32 of the widest tile that calls of up to S positions may
// get.
size_t fp8_tc_part_bytes(int S, int E) {
  const int bn = E > 1 ? fp8_tc_by_rows(S, E).bn : (S <= 32 ? 32 : (S <= 64 ? 64 : (S <= 128 ? 128 : 256)));
  return (size_t)kGtMaxPairs * 2 * 2 * bn * 128 * sizeof(float);
}

static bool f8_tmap(CUtensorMap* tm, int rank, const void* base, const cuuint64_t* dims,
                    const cuuint64_t* strides, const cuuint32_t* box) {
  EncodeTiledFn enc = tc_encode_fn();
  if (!enc) return false;
  const cuuint32_t es[5] = {1, 1, 1, 1, 1};
  return enc(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box,
             es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, bool ACT, int BN>
static cudaError_t launch_f8(F8Params& p, cudaStream_t st) {
  using Cfg = F8Cfg<BN, ACT>;
  auto kernel = fp8_tc_kernel<T, ACT, BN>;
  static PerDevice<int> per;
  int pairs = 0;
  cudaError_t err = on_device(per, &pairs, [&](int* v) {
    cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
    if (e != cudaSuccess) return e;
    {
      // the split draws on the registers of the launch: with fewer it would wait forever
      cudaFuncAttributes a;
      e = cudaFuncGetAttributes(&a, kernel);
      if (e != cudaSuccess) return e;
      if (a.numRegs < kF8RegsLaunch) return cudaErrorInvalidConfiguration;
    }
    cudaLaunchConfig_t q = {};
    q.gridDim = dim3(2 * kGtMaxPairs);
    q.blockDim = dim3(kF8Threads);
    q.dynamicSmemBytes = Cfg::kSmem;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, kernel, &q);
    *v = n < 1 ? 1 : (n < kGtMaxPairs ? n : kGtMaxPairs);
    return e;
  });
  if (err != cudaSuccess) return err;
  const GroupedDims& d = p.d;
  const GroupedCall& c = p.c;
  bool ok;
  p.whole16 = ACT && (d.N / 2) % 16 == 0;
  const cuuint64_t row = (cuuint64_t)c.ldw;
  if (p.whole16) {
    // [E][I / 16 groups][2 halves][16 rows][K]
    const cuuint64_t dims[5] = {(cuuint64_t)d.K, 16, 2, (cuuint64_t)(d.N / 32), (cuuint64_t)d.E};
    const cuuint64_t str[4] = {row, row * (d.N / 2), row * 16, row * d.N};
    const cuuint32_t box[5] = {kF8K, 16, 2, 4, 1};
    ok = f8_tmap(&p.tm_w, 5, c.w, dims, str, box);
  } else if (ACT) {
    const cuuint64_t dims[4] = {(cuuint64_t)d.K, (cuuint64_t)(d.N / 2), 2, (cuuint64_t)d.E};
    const cuuint64_t str[3] = {row, row * (d.N / 2), row * d.N};
    const cuuint32_t box[4] = {kF8K, 16, 2, 1};
    ok = f8_tmap(&p.tm_w, 4, c.w, dims, str, box);
  } else {
    const cuuint64_t dims[3] = {(cuuint64_t)d.K, (cuuint64_t)d.N, (cuuint64_t)d.E};
    const cuuint64_t str[2] = {row, row * d.N};
    const cuuint32_t box[3] = {kF8K, 128, 1};
    ok = f8_tmap(&p.tm_w, 3, c.w, dims, str, box);
  }
  const cuuint64_t xdims[2] = {(cuuint64_t)d.K, (cuuint64_t)(c.perm ? c.x_rows : c.S)};
  const cuuint64_t xstr[1] = {(cuuint64_t)c.ldx};
  const cuuint32_t xbox[2] = {kF8K, c.perm ? 1u : (cuuint32_t)Cfg::kChunk};
  ok = ok && f8_tmap(&p.tm_x, 2, c.x, xdims, xstr, xbox);
  if (!ok) return cudaErrorInvalidValue;
  // no more pairs than K steps can keep busy
  const long long units = ((long long)cdiv(c.S, BN) + (d.E < c.S ? d.E : c.S)) * p.RB;
  const long long useful = units * (p.KT < kGtMinSteps ? 1 : cdiv(p.KT, kGtMinSteps));
  const int G = useful < pairs ? (int)useful : pairs;
  return launch_kernel(kernel, dim3(2 * G), dim3(kF8Threads), Cfg::kSmem, st, true, p);
}

template <typename T, bool ACT>
static cudaError_t launch_f8_bn(F8Params& p, cudaStream_t st) {
  static PerDevice<int> per;           // CTA pairs of the device
  int pairs = 0;
  const cudaError_t e = on_device(per, &pairs, [](int* v) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    *v = std::max(1, sms / 2);
    return e;
  });
  if (e != cudaSuccess) return e;
  p.RB = cdiv(p.cols, ACT ? 128 : 256);
  const F8Plan plan = fp8_tc_plan(p.c.S, p.d.E, p.KT, p.RB, pairs);
  p.fix_steps = plan.fix_steps;
  switch (plan.bn) {
    case 32: return launch_f8<T, ACT, 32>(p, st);
    case 64: return launch_f8<T, ACT, 64>(p, st);
    case 128: return launch_f8<T, ACT, 128>(p, st);
    default: return launch_f8<T, ACT, 256>(p, st);
  }
}

// Whether the tile copies can address the operands: 16-byte bases and strides.
bool fp8_tc_addressable(const GroupedDims& d, const Fp8Call& f) {
  const auto on16 = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0; };
  const GroupedCall& c = f.c;
  return on16(c.x) && on16(c.w) && c.ldx % 16 == 0 && c.ldw % 16 == 0 && c.ldx < (1LL << 39) &&
         c.ldw * d.N < (1LL << 39);
}

cudaError_t launch_fp8_tc(const GroupedDims& d, const Fp8Call& f, float* part, int32_t* tickets,
                          cudaStream_t st) {
  F8Params p;
  p.d = d;
  p.c = f.c;
  p.xs = f.xs;
  p.ws = f.ws;
  p.ldxs = f.ldxs;
  p.part = part;
  p.tickets = tickets;
  p.KT = fp8_blocks(d.K);
  p.cols = grouped_cols(d);
  p.tall = fp8_tall(d);
  const uintptr_t out = reinterpret_cast<uintptr_t>(f.c.out);
  p.packed = p.cols % 2 == 0 && f.c.ldo % 2 == 0 && (out & 3) == 0;
  p.vec = p.cols % 8 == 0 && f.c.ldo % 8 == 0 && (out & 15) == 0;
  if (d.dtype == MOE_DTYPE_F16)
    return d.act ? launch_f8_bn<__half, true>(p, st) : launch_f8_bn<__half, false>(p, st);
  return d.act ? launch_f8_bn<__nv_bfloat16, true>(p, st) : launch_f8_bn<__nv_bfloat16, false>(p, st);
}

}  // namespace moe
