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
//     The 128 sums of a thread and what is in flight need 208 registers: the other warps give theirs
//     up (setmaxnreg).
//
// Roles: warp 0 weight copies, warp 1 MMA issue (leader CTA), warps 2-5 or 2-7 token copies (tiles, or
// gathers of four rows by index; warp 3 also allocates the tensor memory, warp 2 asks for the next
// unit's weight scales), warps 6 and 7 scales up to 128 tokens, warps 8-15 epilogue.
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

template <int BN, bool ACT>
struct F8Cfg {
  static constexpr bool kTokenRows = BN == 256;              // tokens are the MMA's M operand
  // registers shared out anew by role: a thread's of the epilogue warps and of the others
  static constexpr bool kSplit = BN >= 128;
  static constexpr int kRegsMore = BN == 256 ? 208 : 184, kRegsLess = 256 - kRegsMore;
  static_assert(256 * (kRegsMore + kRegsLess) <= kF8Threads * kF8RegsLaunch, "register split");
  static constexpr int kHalf = BN / 2;                       // tokens a CTA loads
  static constexpr int kChunk = kHalf < 32 ? kHalf : 32;     // tokens per tile copy
  static constexpr int kBytesW = 128 * 128, kBytesB = kHalf * 128, kStage = kBytesW + kBytesB;
  static constexpr int kBuffers = BN == 256 ? 2 : 4;         // tensor-memory buffers of a step
  static constexpr int kCols = kBuffers * BN;                // tensor-memory columns
  static constexpr int kGroups = BN == 32 ? 1 : 2;           // groups of four epilogue warps
  static constexpr int kWide = BN == 32 ? 32 : BN / 2;       // accumulator columns of a group
  static constexpr int kSets = ACT ? 2 : 1;                  // scales of a lane's column: up and gate
  static constexpr int kTokenWarps = kTokenRows ? 6 : 4;     // from warp 2 on
  // ring of the tokens' scales: slots of four steps, each [4][sets][kPad]
  static constexpr int kPad = BN + 4;                        // both sets' words in other banks
  static constexpr int kSlots = 3, kSlot = 4 * kSets * kPad;
  static constexpr int kScales = kTokenRows ? 0 : kSlots * kSlot * 4;
  static constexpr int kTables = 3 * 1028 * 4 + 512 + kScales;
  static constexpr int kStages = (227 * 1024 - 1024 - kTables) / kStage > 12
                                     ? 12 : (227 * 1024 - 1024 - kTables) / kStage;
  static constexpr int kSmem = 1024 + kStages * kStage + kTables;
  // K steps that joining the pieces of a unit costs (as for the 16-bit products)
  static constexpr int kFixSteps = BN <= 32 ? 8 : (BN <= 64 ? 12 : (BN <= 128 ? 24 : 40));
};

struct F8Params {
  CUtensorMap tm_w, tm_x;
  GroupedDims d;
  GroupedCall c;
  const float* xs;
  const float* ws;
  long long ldxs;
  float* part;          // [pairs][2][2 CTAs][BN][128]
  int32_t* tickets;     // [pairs][2 CTAs][2 groups]
  int KT, RB, cols, tall;
  int packed, vec;      // output rows on 4 bytes, on 16
  int whole16;          // SwiGLU weights by whole 16-row groups: one 5-d copy per K step
};

// Asks for the scales of the next unit's weight rows (up to four rows of KT) in L2: from DRAM under load
// they would take longer than the steps that a fetch is ahead.
__device__ __forceinline__ void f8_prefetch(const float* row, int n, int line) {
  const char* at = reinterpret_cast<const char*>(reinterpret_cast<uintptr_t>(row) & ~(uintptr_t)127) + 128 * line;
  if (at < reinterpret_cast<const char*>(row + n)) asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
}

// One verdict for the 128 threads of a group, at its named barrier.
__device__ __forceinline__ bool f8_group_all(int group, bool ok) {
  int all;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %2, 0;\n"
      " barrier.cta.red.and.pred q, %1, 128, p;\n selp.b32 %0, 1, 0, q;\n}"
      : "=r"(all)
      : "r"(1 + group), "r"((int)ok)
      : "memory");
  return all != 0;
}

// Stores a lane's outputs of 128 accumulator columns, tokens in lanes: columns col0 .. of row `row`.
template <typename T, bool ACT>
__device__ __forceinline__ void f8_store_row(const F8Params& p, const uint64_t (&acc)[64], long long row, int col0) {
  T* o = static_cast<T*>(p.c.out) + row * p.c.ldo + col0;
  const bool up_first = p.d.layout == MOE_W13_UP_GATE;
  constexpr int kOut = ACT ? 64 : 128;
#pragma unroll
  for (int c = 0; c < kOut; c += 8) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      if constexpr (ACT) {
        // outputs 16 b .. 16 b + 15: half 0 in columns 32 b .., half 1 in 32 b + 16 ..
        const int at = (c / 16) * 32 + c % 16 + j;
        const float2 a = unpair_f32(acc[at / 2]), b = unpair_f32(acc[at / 2 + 8]);
        v[j] = swiglu_f32(up_first ? a.x : b.x, up_first ? b.x : a.x, p.d.limit, p.d.alpha, p.d.beta);
        v[j + 1] = swiglu_f32(up_first ? a.y : b.y, up_first ? b.y : a.y, p.d.limit, p.d.alpha, p.d.beta);
      } else {
        const float2 a = unpair_f32(acc[(c + j) / 2]);
        v[j] = a.x;
        v[j + 1] = a.y;
      }
    }
    const T t[8] = {from_f32<T>(v[0]), from_f32<T>(v[1]), from_f32<T>(v[2]), from_f32<T>(v[3]),
                    from_f32<T>(v[4]), from_f32<T>(v[5]), from_f32<T>(v[6]), from_f32<T>(v[7])};
    const int left = p.cols - col0 - c;
    if (p.vec) {
      if (left > 0) {
        uint4 w;
        memcpy(&w, t, 16);
        *reinterpret_cast<uint4*>(o + c) = w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < left) o[c + j] = t[j];
    }
  }
}

template <typename T, bool ACT, int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kF8Threads, 1)
fp8_tc_kernel(const __grid_constant__ F8Params p) {
  using Cfg = F8Cfg<BN, ACT>;
  constexpr int S = Cfg::kStages, NB = Cfg::kBuffers;
  extern __shared__ uint8_t raw[];
  uint8_t* st = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(st + S * Cfg::kStage);   // [S] (leader's are used)
  uint64_t* empty = full + S;          // [S]
  uint64_t* tfull = empty + S;         // [NB] a step's product is ready
  uint64_t* tempty = tfull + NB;       // [NB] and has been read (leader's are used)
  uint64_t* sfull = tempty + NB;       // [slots] scales of four steps are there
  uint64_t* sempty = sfull + Cfg::kSlots;   // [slots] and have been read
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(sempty + Cfg::kSlots);
  int* s_flag = reinterpret_cast<int*>(s_tmem + 1);   // [2]
  int* s_warp = s_flag + 2;            // [warps]
  int* s_fills = s_warp + kF8Threads / 32;   // fills whose stage the weight warp has found empty
  int* s_off = reinterpret_cast<int*>(st + S * Cfg::kStage + 512);
  int* s_cnt = s_off + 1028;
  int* s_tile = s_cnt + 1028;
  float* s_scale = reinterpret_cast<float*>(s_tile + 1028);   // [slots][4 steps][sets][kPad]
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
    for (int b = 0; b < NB; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 8 * Cfg::kGroups);        // the epilogue warps of both CTAs
    }
    for (int b = 0; b < Cfg::kSlots; ++b) {
      mbar_init(&sfull[b], 2);
      mbar_init(&sempty[b], 4 * Cfg::kGroups);
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
  int total = gt_number<BN, kF8Threads>(cnt, E, s_tile, s_warp);
  if (bad) {
    total = 0;
    if (tid == 0) set_error(err, kErrRouteBounds);
  }
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
  work.init(total, p.KT, p.RB, 0, G, pair, Cfg::kFixSteps, false);
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
  if (warp < 8) {
  if constexpr (Cfg::kSplit) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::kRegsLess));
  if (warp == 0) {
    const uint32_t bar0 = map_rank(&full[0], 0);
    while (ok && work.next(u, tile, rb, k0, len)) {
      const GtTile un = tile_at(tile);
      const int rows = p.c.perm != nullptr ? un.nhalf : cdiv(un.nhalf, Cfg::kChunk) * Cfg::kChunk;
      const uint32_t bytes = 2u * (Cfg::kBytesW + rows * 128);
      const int r = (2 * rb + (int)rank) * kRows;
      for (int x = k0 * kF8K; x < (k0 + len) * kF8K; x += kF8K, ++issued) {
        if (!mbar_wait_warp(&empty[s], phase ^ 1, err)) {
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
        ok = mbar_wait(&empty[j % S], (j / S) & 1, err);
      if (!ok && rank == 0) drain_stage_loads<S>(full, issued, err);
    }
  } else if (warp == 1) {
    // operand descriptors: only the address changes from stage to stage and from K block to K block
    const uint64_t desc0 = desc_sw128(st);
    const uint32_t hi = (uint32_t)(desc0 >> 32), lo0 = (uint32_t)desc0;
    uint32_t step = 0;               // steps that have gone to tensor memory
    // nothing commits to this phase before the first step's MMAs
    if (p.d.probe_ns != 0 && blockIdx.x == 0)
      ok = __all_sync(0xffffffffu, mbar_wait(&tfull[0], 0, err, p.d.probe_ns));
    while (rank == 0 && ok && work.next(u, tile, rb, k0, len)) {
      const GtTile un = tile_at(tile);
      const uint32_t idesc = idesc_pair8(Cfg::kTokenRows ? 256 : 2 * un.nhalf);
      for (int i = 0; i < len; ++i, ++step) {
        const uint32_t b = step % NB;
        ok = mbar_wait_warp(&tempty[b], ((step / NB) & 1) ^ 1, err) && mbar_wait_warp(&full[s], phase, err);
        if (!ok) break;
        tc_fence_after();
        if (lane == 0) {
          const uint32_t lo = lo0 + s * (Cfg::kStage >> 4);
#pragma unroll
          for (int kb = 0; kb < 4; ++kb) {
            const uint64_t dw = ((uint64_t)hi << 32) | (lo + 2 * kb);
            const uint64_t dx = ((uint64_t)hi << 32) | (lo + (Cfg::kBytesW >> 4) + 2 * kb);
            mma2_f8(tmem + b * BN, Cfg::kTokenRows ? dx : dw, Cfg::kTokenRows ? dw : dx, idesc, kb != 0);
          }
          tc2_commit(&empty[s]);
          tc2_commit(&tfull[b]);
        }
        advance();
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
  } else if constexpr (!Cfg::kTokenRows) {
    // Scales of the tokens' columns: warp 6 columns 0 .. 31 and 64 .. 95, warp 7 the others.  Those of the next
    // four steps, of the next unit too, are on their way while these wait for their slot.
    constexpr int M = (BN + 63) / 64, SETS = Cfg::kSets;
    const int c0 = (warp - 6) * 32 + lane;
    float nx[M][4], nw[SETS][4];
    const float* xs[M];
    const float* w[SETS];
    int i0 = 0, n = 0, slot = 0;
    uint32_t turn = 0;
    len = 0;
    const auto fetch = [&]() {         // steps of the block that it asks for, 0 at the end
      i0 += n;
      if (i0 >= len) {
        if (!work.next(u, tile, rb, k0, len)) return 0;
        const GtTile un = tile_at(tile);
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
    while (ok && n > 0) {
      float now[M][SETS][4];
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int h = 0; h < SETS; ++h)
#pragma unroll
          for (int j = 0; j < 4; ++j) now[m][h][j] = nx[m][j] * nw[h][j];
      n = fetch();
      ok = mbar_wait_warp(&sempty[slot], (turn & 1) ^ 1, err);
      if (!ok) break;
      float* to = s_scale + slot * Cfg::kSlot + c0;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int h = 0; h < SETS; ++h)
#pragma unroll
          for (int m = 0; m < M; ++m)
            if (c0 + 64 * m < BN) to[(j * SETS + h) * Cfg::kPad + 64 * m] = now[m][h][j];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sfull[slot]);
      if (++slot == Cfg::kSlots) {
        slot = 0;
        ++turn;
      }
    }
  }
  } else {
    if constexpr (Cfg::kSplit) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Cfg::kRegsMore));
    // groups of four warps share the columns of every step
    constexpr int CW = Cfg::kWide, SETS = Cfg::kSets;
    const int q = warp & 3, g = (warp - 8) >> 2, t = q * 32 + lane;
    const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16) + g * CW;
    const uint32_t bempty = map_rank(&tempty[0], 0);
    const auto sync_group = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(1 + g) : "memory"); };
    // a step's buffer has been read
    const auto release = [&](uint32_t b) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_read(bempty + 8 * b);
    };
    uint32_t step = 0, turn = 0;
    int slot = 0;
    uint64_t acc[CW / 2];
    // this group's sums, or those of all pieces of a cut unit, to the output
    const auto store = [&](const GtTile& un) {
      if constexpr (Cfg::kTokenRows) {
        const int i = (int)rank * un.nhalf + t;
        if (t < un.nhalf && i < un.n) f8_store_row<T, ACT>(p, acc, un.p0 + i, (2 * rb + g) * kRows);
      } else {
        const int col0 = (2 * rb + (int)rank) * kRows;
#pragma unroll
        for (int j = 0; j < CW / 32; ++j) {
          float v[32];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 f = unpair_f32(acc[16 * j + i]);
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
          }
          const int c0 = g * CW + 32 * j;
          if (c0 < un.n) gt_store<T, ACT>(p, v, un, col0, c0, q, lane);
        }
      }
    };
    while (ok && g < Cfg::kGroups && work.next(u, tile, rb, k0, len)) {
      const GtTile un = tile_at(tile);
#pragma unroll
      for (int j = 0; j < CW / 2; ++j) acc[j] = 0;
      uint32_t v[2][32];
      const auto add = [&](int j, const uint64_t (&f)[SETS]) {     // 32 columns, one factor (two: by 16)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          fma_pair_f32(acc[16 * j + i], pair_f32(v[j & 1][2 * i], v[j & 1][2 * i + 1]), f[ACT ? i / 8 : 0]);
      };
      if constexpr (Cfg::kTokenRows) {
        const float* xs = p.xs + row_of(un.p0 + min((int)rank * un.nhalf + t, un.n - 1)) * p.ldxs + k0;
        const float* w[SETS];
#pragma unroll
        for (int h = 0; h < SETS; ++h) w[h] = scales_of(un.e, h, (2 * rb + g) * kRows) + k0;
        // scales of the next two steps are on their way
        float x1 = xs[0], x2 = xs[min(1, len - 1)], w1[SETS], w2[SETS];
#pragma unroll
        for (int h = 0; h < SETS; ++h) {
          w1[h] = w[h][0];
          w2[h] = w[h][min(1, len - 1)];
        }
        for (int i = 0; i < len; ++i, ++step) {
          uint64_t f[SETS];
#pragma unroll
          for (int h = 0; h < SETS; ++h) {
            const uint32_t b = __float_as_uint(x1 * w1[h]);
            f[h] = pair_f32(b, b);
            w1[h] = w2[h];
            w2[h] = w[h][min(i + 2, len - 1)];
          }
          x1 = x2;
          x2 = xs[min(i + 2, len - 1)];
          const uint32_t b = step % NB, at = trow + b * BN;
          ok = mbar_wait_warp(&tfull[b], (step / NB) & 1, err);
          if (!ok) break;
          tc_fence_after();
          // 64 columns at a time in flight: a wait takes all loads that have been started
          tmem_ld32_start(at, v[0]);
          tmem_ld32_start(at + 32, v[1]);
          tmem_ld_wait(v[0]);
          tmem_after_wait(v[1]);
          add(0, f);
          tmem_ld32_start(at + 64, v[0]);
          add(1, f);
          tmem_ld32_start(at + 96, v[1]);
          tmem_ld_wait(v[0]);
          tmem_after_wait(v[1]);
          release(b);
          add(2, f);
          add(3, f);
        }
      } else {
        for (int i0 = 0; ok && i0 < len; i0 += 4) {
          ok = mbar_wait_warp(&sfull[slot], turn & 1, err);
          const float* now = s_scale + slot * Cfg::kSlot + g * CW + (ACT && lane >= 16 ? Cfg::kPad : 0);
#pragma unroll 1
          for (int j = 0; ok && j < 4 && i0 + j < len; ++j, ++step) {
            const ulonglong2* f = reinterpret_cast<const ulonglong2*>(now + j * SETS * Cfg::kPad);
            ulonglong2 s4[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) s4[i] = f[i];
            const uint32_t b = step % NB, at = trow + b * BN;
            ok = mbar_wait_warp(&tfull[b], (step / NB) & 1, err);
            if (!ok) break;
            tc_fence_after();
            if (g * CW < un.n) {
              tmem_ld32_start(at, v[0]);
              if (CW == 64) tmem_ld32_start(at + 32, v[1]);
              tmem_ld_wait(v[0]);
              if (CW == 64) tmem_after_wait(v[1]);
            }
            release(b);
            if (g * CW < un.n) {
#pragma unroll
              for (int h = 0; h < CW / 32; ++h) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  fma_pair_f32(acc[16 * h + 2 * i], pair_f32(v[h][4 * i], v[h][4 * i + 1]), s4[i].x);
                  fma_pair_f32(acc[16 * h + 2 * i + 1], pair_f32(v[h][4 * i + 2], v[h][4 * i + 3]), s4[i].y);
                  if (h + 1 < CW / 32) s4[i] = f[8 + i];
                }
              }
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sempty[slot]);
          if (++slot == Cfg::kSlots) {
            slot = 0;
            ++turn;
          }
        }
      }
      if (len == p.KT) {
        if (ok) store(un);             // no named barrier from here on: pieces come first
      } else {
        // one verdict for the four warps: all of them reach the named barriers below, or none
        ok = f8_group_all(g, ok);
        if (!ok) break;
        const size_t stride = (size_t)2 * BN * 128;      // floats of one slot
        const size_t at = ((size_t)rank * BN + g * CW) * 128 + t;
        float* out = p.part + (size_t)work.slot_of(pair, u) * stride + at;
        const int n = Cfg::kTokenRows ? CW : un.n - g * CW;
#pragma unroll
        for (int j = 0; j < CW / 2; ++j) {
          const float2 f = unpair_f32(acc[j]);
          if (2 * j < n) __stcg(out + (size_t)(2 * j) * 128, f.x);
          if (2 * j + 1 < n) __stcg(out + (size_t)(2 * j + 1) * 128, f.y);
        }
        sync_group();
        int c_lo, c_hi;
        work.owners(u, c_lo, c_hi);
        if (t == 0) {
          __threadfence();                               // the group's sums, ordered by its barrier
          int32_t* ticket = p.tickets + 4 * (u - work.first) + 2 * rank + g;
          const int last = atomicAdd(ticket, 1) == c_hi - c_lo;
          if (last) *ticket = 0;                         // ready for the next call
          __threadfence();
          s_flag[g] = last;
        }
        sync_group();
        if (s_flag[g]) {
#pragma unroll
          for (int j = 0; j < CW / 2; ++j) acc[j] = 0;
          for (int c = c_lo; c <= c_hi; ++c) {
            const float* src = p.part + (size_t)work.slot_of(c, u) * stride + at;
#pragma unroll
            for (int j = 0; j < CW / 2; ++j) {
              if (2 * j < n) {
                const float lo = __ldcg(src + (size_t)(2 * j) * 128), hi = 2 * j + 1 < n ? __ldcg(src + (size_t)(2 * j + 1) * 128) : 0.f;
                const float2 f = unpair_f32(acc[j]);
                acc[j] = pair_f32(__float_as_uint(f.x + lo), __float_as_uint(f.y + hi));
              }
            }
          }
          store(un);
        }
        sync_group();                                    // s_flag read by all
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

// Token-tile width by the mean positions per expert, as for the 16-bit products; of one matrix without
// offsets, whose rows are known, the narrowest that holds them.
static int fp8_tc_bn(int S, int E, bool dense) {
  const long long many = dense ? 1 : 4;
  if ((long long)S * many <= 32LL * E) return 32;
  if (dense ? S <= 64 : (long long)S <= 24LL * E) return 64;
  if (dense ? S <= 128 : (long long)S <= 64LL * E) return 128;
  return 256;
}

size_t fp8_tc_part_bytes(int S, int E) {
  // a call may have fewer rows than the plan, and offsets or none: the widest tile of any of them
  const int bn = std::max(fp8_tc_bn(S, E, false), fp8_tc_bn(S, E, E == 1));
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
    if (Cfg::kSplit) {
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
  p.RB = cdiv(p.cols, ACT ? 128 : 256);
  // no more pairs than K steps can keep busy
  const long long units = ((long long)cdiv(c.S, BN) + (d.E < c.S ? d.E : c.S)) * p.RB;
  const long long useful = units * (p.KT < kGtMinSteps ? 1 : cdiv(p.KT, kGtMinSteps));
  const int G = useful < pairs ? (int)useful : pairs;
  return launch_kernel(kernel, dim3(2 * G), dim3(kF8Threads), Cfg::kSmem, st, true, p);
}

template <typename T, bool ACT>
static cudaError_t launch_f8_bn(F8Params& p, cudaStream_t st) {
  switch (fp8_tc_bn(p.c.S, p.d.E, p.c.offsets == nullptr)) {
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
