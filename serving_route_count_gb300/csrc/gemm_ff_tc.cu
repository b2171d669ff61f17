// gemm_ff_tc.cu - products of the gated feed-forward block on the tensor cores: out[c][r] = sum_k
// R(r, k) C(c, k), either operand stored along K or the other way round, with the block's epilogues.
//
// The layout is the grouped products' (gemm_grouped_tc.cu): a pair of CTAs (tcgen05 cta_group::2) owns a
// unit of 256 rows of R (the MMA's M operand: weights, so that one token still streams them through
// full-size MMAs) x up to BN rows of C (tokens); the gated product's unit has 128 up and 128 gate rows,
// interleaved 16 by 16, so that a warp's 32 accumulator lanes hold both halves of 16 outputs.  The
// accumulators are double-buffered in tensor memory, so a unit's epilogue runs under the next unit's
// MMAs.  What a backward pass adds is the other storage order: W2 and W13 are read by columns (dh, dx)
// and tokens are summed over (dW).  Nothing is transposed in memory; such an operand's tiles are boxes of
// 64 rows along K x 64 elements, which land in shared memory as the MMA's 128-byte-swizzled MN-major
// form, and the instruction descriptor says so.
//
// Bounds and measurements (GB300, bf16, measured 1910 TFLOP/s in a burst, 1726 sustained): 2048 tokens of 7168 ->
// 4608 -> 7168, us of each product and TFLOP/s under the counters, one kernel at a time at 1.45 to 1.55 GHz (floor 142
// for the two-halves ones, 71 for the others): up projections with the saved sums 168 / 1610; down 82 / 1650; dh with
// the activation's gradient 104 / 1300; dx 155 / 1740; dW13 167 / 1625; dW2 88 / 1540: bound by the tensor cores (pipe 78
// to 83 % active; dW 67 to 70, dh 58, whose epilogue reads two fp32 sums for every value).  The whole step of 4096 tokens
// 1520 to 1640 us from box to box (1.48 to 1.60 PFLOP/s, 86 to 93 % of sustained).  777 tokens of 6144 -> 512 -> 6144: 91
// us with the weights in L2, 111 to 118 from HBM, floor 23:
// sixteen to fifty units for 76 pairs, and a unit's 96 steps take 23 us.
//
// Roles: warp 0 tile copies, warp 1 MMA issue (leader CTA), warp 2 tensor memory, warps 4-11 epilogue.
#include "feed_forward.cuh"
#include "tc_pair.cuh"
#include "tc_tile.cuh"
#include "tc_units.cuh"
#include "../../include/moe_gb300.h"

namespace moe {
using namespace tc;

constexpr int kFtThreads = 384;
constexpr int kFtK = 64;                 // K step: one 128-byte swizzled row

template <int BN>
struct FtCfg {
  static constexpr int kHalf = BN / 2;                       // rows of C that a CTA loads
  static constexpr int kBytesR = 128 * 128, kBytesC = kHalf * 128, kStage = kBytesR + kBytesC;
  static constexpr int kTables = 512;                        // barriers
  static constexpr int kStages = (227 * 1024 - 1024 - kTables) / kStage > 12
                                     ? 12 : (227 * 1024 - 1024 - kTables) / kStage;
  static constexpr int kSmem = 1024 + kStages * kStage + kTables;
  static constexpr int kCols = 2 * BN;                       // tensor-memory columns: two buffers
};

struct FtParams {
  CUtensorMap tm_r, tm_c;
  FfDims d;
  FfGemm g;
  float* part;          // [pairs][2][2 CTAs][BN / 4][128][4]
  int32_t* tickets;     // [pairs][2 CTAs][2 groups]
  int KT, RB;           // K steps; row blocks
  int tiles, size;      // tiles of C, rows of a tile (the last may have fewer)
  int cut;              // whether the units left over are cut along K
  int r_mn, c_mn;       // operand stored with its rows along the contiguous dimension
  int bf16, packed, whole16;
};

__device__ __forceinline__ uint32_t ft_pack(bool bf16, float a, float b) {
  if (bf16) {
    __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return reinterpret_cast<uint32_t&>(v);
  }
  __half2 v = __floats2half2_rn(a, b);
  return reinterpret_cast<uint32_t&>(v);
}
// Epilogue of 32 accumulator columns (rows c0 .. c0 + 31 of the unit's tile of n rows of C from p0) of
// this lane's row of R; col0: output column of the CTA's first row.  A lane and its neighbour exchange
// every other row of C, so that each access takes two adjacent columns; where rows do not start on 4 bytes
// each lane takes its own column.
template <int EPI>
__device__ __forceinline__ void ft_store(const FtParams& p, float (&v)[32], int p0, int n, int col0, int c0,
                                         int q, int lane) {
  uint16_t* out = static_cast<uint16_t*>(p.g.out);
  float* pre = p.g.pre;
  const int odd = lane & 1, nr = p.g.nr;
  const bool bf16 = p.bf16;
  const long long ldo = p.g.ldo;
  if constexpr (EPI == kFfStore) {
    const int col = col0 + q * 32 + lane;
    if (p.packed) {
      uint16_t* o = out + (long long)(p0 + c0 + odd) * ldo + (col & ~1);
      const int m = col < nr ? n - c0 - odd : 0;
#pragma unroll
      for (int c = 0; c < 32; c += 2) {
        const float got = __shfl_xor_sync(0xffffffffu, odd ? v[c] : v[c + 1], 1);
        const uint32_t w = ft_pack(bf16, odd ? got : v[c], odd ? v[c + 1] : got);
        if (c < m) *reinterpret_cast<uint32_t*>(o) = w;
        o += 2 * ldo;
      }
    } else {
      uint16_t* o = out + (long long)(p0 + c0) * ldo + col;
      const int m = col < nr ? n - c0 : 0;
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        if (c < m) *o = (uint16_t)ft_pack(bf16, v[c], 0.f);
        o += ldo;
      }
    }
  } else if constexpr (EPI == kFfGlu) {
    // lanes 0-15: half 0 of outputs i .. i + 15, lanes 16-31: half 1; after the exchange lanes 0-15 hold
    // rows c0 .. c0 + 15 of both halves, lanes 16-31 rows c0 + 16 .. c0 + 31
    const bool hi = lane >= 16, up_first = p.d.layout == MOE_W13_UP_GATE;
    const int col = col0 + q * 16 + (lane & 15), t0 = c0 + (hi ? 16 : 0);
    float a[16], b[16];
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      const float got = __shfl_xor_sync(0xffffffffu, hi ? v[c] : v[c + 16], 16);
      a[c] = hi ? got : v[c];
      b[c] = hi ? v[c + 16] : got;
    }
    const auto act = [&](int c) {
      return swiglu_f32(up_first ? a[c] : b[c], up_first ? b[c] : a[c], p.d.limit, p.d.alpha, p.d.beta);
    };
    if (pre != nullptr) {
      const int m = col < nr ? n - t0 : 0;
      float* s = pre + (long long)(p0 + t0) * 2 * nr + col;
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        if (c < m) {
          s[0] = a[c];
          s[nr] = b[c];
        }
        s += 2LL * nr;
      }
    }
    if (p.packed) {
      const int m = col < nr ? n - t0 - odd : 0;
      uint16_t* o = out + (long long)(p0 + t0 + odd) * ldo + (col & ~1);
#pragma unroll
      for (int c = 0; c < 16; c += 2) {
        const float h0 = act(c), h1 = act(c + 1);
        const float got = __shfl_xor_sync(0xffffffffu, odd ? h0 : h1, 1);
        const uint32_t w = ft_pack(bf16, odd ? got : h0, odd ? h1 : got);
        if (c < m) *reinterpret_cast<uint32_t*>(o) = w;
        o += 2 * ldo;
      }
    } else {
      const int m = col < nr ? n - t0 : 0;
      uint16_t* o = out + (long long)(p0 + t0) * ldo + col;
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        if (c < m) *o = (uint16_t)ft_pack(bf16, act(c), 0.f);
        o += ldo;
      }
    }
  } else {
    const bool up_first = p.d.layout == MOE_W13_UP_GATE;
    const int col = col0 + q * 32 + lane;
    const auto grad = [&](float x0, float x1, float dh, float* d0, float* d1) {
      float du, dg;
      swiglu_grad(up_first ? x0 : x1, up_first ? x1 : x0, dh, p.d.limit, p.d.alpha, p.d.beta, &du, &dg);
      *d0 = up_first ? du : dg;
      *d1 = up_first ? dg : du;
    };
    if (p.packed) {
      const int m = col < nr ? n - c0 - odd : 0;
      const float* s = pre + (long long)(p0 + c0 + odd) * 2 * nr + (col & ~1);
      uint16_t* o = out + (long long)(p0 + c0 + odd) * ldo + (col & ~1);
      float2 x0[16], x1[16];
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        x0[c] = x1[c] = make_float2(0.f, 0.f);
        if (2 * c < m) {
          x0[c] = __ldcg(reinterpret_cast<const float2*>(s));
          x1[c] = __ldcg(reinterpret_cast<const float2*>(s + nr));
        }
        s += 4LL * nr;
      }
#pragma unroll
      for (int c = 0; c < 32; c += 2) {
        const float got = __shfl_xor_sync(0xffffffffu, odd ? v[c] : v[c + 1], 1);
        const float h0 = odd ? got : v[c], h1 = odd ? v[c + 1] : got;
        const float2 f0 = x0[c / 2], f1 = x1[c / 2];
        float d00, d01, d10, d11;
        grad(f0.x, f1.x, h0, &d00, &d01);
        grad(f0.y, f1.y, h1, &d10, &d11);
        if (c < m) {
          *reinterpret_cast<uint32_t*>(o) = ft_pack(bf16, d00, d10);
          *reinterpret_cast<uint32_t*>(o + nr) = ft_pack(bf16, d01, d11);
        }
        o += 2 * ldo;
      }
    } else {
      const int m = col < nr ? n - c0 : 0;
      const float* s = pre + (long long)(p0 + c0) * 2 * nr + col;
      uint16_t* o = out + (long long)(p0 + c0) * ldo + col;
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        if (c < m) {
          float d0, d1;
          grad(s[0], s[nr], v[c], &d0, &d1);
          o[0] = (uint16_t)ft_pack(bf16, d0, 0.f);
          o[nr] = (uint16_t)ft_pack(bf16, d1, 0.f);
        }
        s += 2LL * nr;
        o += ldo;
      }
    }
  }
}

template <int EPI, int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kFtThreads, 1)
ff_tc_kernel(const __grid_constant__ FtParams p) {
  using Cfg = FtCfg<BN>;
  constexpr int S = Cfg::kStages;
  extern __shared__ uint8_t raw[];
  uint8_t* st = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(st + S * Cfg::kStage);   // [S] (leader's are used)
  uint64_t* empty = full + S;          // [S]
  uint64_t* tfull = empty + S;         // [2] accumulators ready
  uint64_t* tempty = tfull + 2;        // [2] accumulators read (leader's are used)
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(tempty + 2);
  int* s_flag = reinterpret_cast<int*>(s_tmem + 1);   // [2]
  int* s_ok = s_flag + 2;              // [8]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, G = gridDim.x >> 1;
  int32_t* err = p.g.err;

  if (warp == 2) {
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
      mbar_init(&tempty[b], 16);       // eight epilogue warps of each CTA
    }
    fence_barrier_init();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  // the next launch may start now that this CTA's tensor memory is allocated
  pdl_wait_prev();
  pdl_launch_next();

  // Every loop below is taken by whole warps; one lane issues.
  constexpr int kRows = EPI == kFfGlu ? 64 : 128;    // output columns of one CTA
  GtWork work;
  work.init(p.tiles, p.KT, p.RB, 0, G, pair, p.cut ? 0 : 0x7FFFFFFF, false);
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
  // a tile's first row, its rows, and how many of them (padded) belong to each CTA
  const auto tile_at = [&](int tile, int& p0, int& n, int& nhalf) {
    p0 = tile * p.size;
    n = min(p.size, p.g.nc - p0);
    nhalf = 8 * cdiv(n, 16);
  };
  if (warp == 0) {
    const uint32_t bar0 = map_rank(&full[0], 0);
    while (ok && work.next(u, tile, rb, k0, len)) {
      int p0, n, nhalf;
      tile_at(tile, p0, n, nhalf);
      const int r = (2 * rb + (int)rank) * kRows, c0 = p0 + (int)rank * nhalf;
      for (int x = k0 * kFtK; x < (k0 + len) * kFtK; x += kFtK, ++issued) {
        if (!mbar_wait_warp(&empty[s], phase ^ 1, err)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          const uint32_t bar = bar0 + 8 * s;
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * Cfg::kStage);
          uint8_t* a = st + s * Cfg::kStage;
          uint8_t* b = a + Cfg::kBytesR;
          if constexpr (EPI == kFfGlu) {
            if (p.whole16) {
              tma2_load_4d(a, &p.tm_r, x, 0, 0, r >> 4, bar);
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j) tma2_load_3d(a + j * 4096, &p.tm_r, x, r + 16 * j, 0, bar);
            }
          } else if (p.r_mn) {
            tma2_load_2d(a, &p.tm_r, r, x, bar);
            tma2_load_2d(a + 8192, &p.tm_r, r + 64, x, bar);
          } else {
            tma2_load_2d(a, &p.tm_r, x, r, bar);
          }
          if (Cfg::kHalf >= 64 && p.c_mn) {
#pragma unroll
            for (int j = 0; j < Cfg::kHalf / 64; ++j) tma2_load_2d(b + j * 8192, &p.tm_c, c0 + 64 * j, x, bar);
          } else {
            tma2_load_2d(b, &p.tm_c, x, c0, bar);
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
    // operand descriptors: only the address changes from stage to stage and from K block to K block.  Along
    // K 16 elements are 32 bytes of a row; the other way round 16 rows of 128 bytes, and 64 elements on is
    // the next box (8192 bytes)
    const uint64_t dr = p.r_mn ? smem_desc(st, 8192, 1024, 2) : desc_sw128(st);
    const uint64_t dc = p.c_mn ? smem_desc(st, 8192, 1024, 2) : desc_sw128(st);
    const uint32_t hir = (uint32_t)(dr >> 32), lor = (uint32_t)dr, hic = (uint32_t)(dc >> 32), loc = (uint32_t)dc;
    const uint32_t stepr = p.r_mn ? 2048 >> 4 : 32 >> 4, stepc = p.c_mn ? 2048 >> 4 : 32 >> 4;
    uint32_t seg = 0;                // units so far
    bool ready = false;              // the next step's operands are known to be there
    // nothing commits to this phase before the first unit's MMAs
    if (p.d.probe_ns != 0 && blockIdx.x == 0)
      ok = __all_sync(0xffffffffu, mbar_wait(&tfull[0], 0, err, p.d.probe_ns));
    while (rank == 0 && ok && work.next(u, tile, rb, k0, len)) {
      int p0, n, nhalf;
      tile_at(tile, p0, n, nhalf);
      const int b = seg & 1;           // the buffer's turns: seg / 2
      ok = mbar_wait_warp(&tempty[b], ((seg >> 1) & 1) ^ 1, err);
      if (!ok) break;
      tc_fence_after();
      const uint32_t idesc = idesc_pair16(p.bf16, 2 * nhalf) | (p.r_mn ? 1u << 15 : 0u) | (p.c_mn ? 1u << 16 : 0u);
      uint32_t accumulate = 0;
      for (int i = 0; i < len; ++i) {
        if (!ready && !mbar_wait_warp(&full[s], phase, err)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t s1 = s + 1 == S ? 0 : s + 1;
        const bool next = mbar_test(&full[s1], phase ^ (s1 == 0));     // of this unit or another
        if (elect_one()) {
          const uint32_t at = s * (Cfg::kStage >> 4);
#pragma unroll
          for (int kb = 0; kb < 4; ++kb) {
            const uint64_t da = ((uint64_t)hir << 32) | (lor + at + kb * stepr);
            const uint64_t db = ((uint64_t)hic << 32) | (loc + at + (Cfg::kBytesR >> 4) + kb * stepc);
            mma2_f16(tmem + b * BN, da, db, idesc, kb == 0 ? accumulate : 1u);
          }
          tc2_commit(&empty[s]);
        }
        accumulate = 1;
        advance();
        ready = __all_sync(0xffffffffu, next);
      }
      if (elect_one()) tc2_commit(&tfull[b]);
      ++seg;
    }
  } else if (warp >= 4) {
    // Two groups of four warps take every other 32 columns of each unit, so that the last unit's epilogue, which
    // nothing covers, and joining take half as long as with a unit to a group (us: 6144 -> 512, 200 tokens cut at
    // 256 72 -> 54, 100 at 128 47 -> 35; the training step of 4096 tokens 1543 -> 1520).
    const int q = warp & 3, g = (warp - 4) >> 2;
    const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16);
    const uint32_t bempty = map_rank(&tempty[0], 0);
    const auto sync_group = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(1 + g) : "memory"); };
    for (uint32_t seg = 0; ok && work.next(u, tile, rb, k0, len); ++seg) {
      int p0, n, nhalf;
      tile_at(tile, p0, n, nhalf);
      const int col0 = (2 * rb + (int)rank) * kRows;
      const uint32_t buf = seg & 1, tbuf = trow + buf * BN;
      const auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_read(bempty + 8 * buf);
      };
      ok = mbar_wait_warp(&tfull[buf], (seg >> 1) & 1, err);
      float v[32];
      if (len == p.KT) {               // no named barrier from here on: pieces come first
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int c0 = 32 * g; c0 < n; c0 += 64) {
          tmem_ld32(tbuf + c0, v);
          if (c0 + 64 >= n) release();
          ft_store<EPI>(p, v, p0, n, col0, c0, q, lane);
        }
        if (32 * g >= n) release();
      } else {
        // one verdict for the four warps: all of them reach the named barriers below, or none
        if (lane == 0) s_ok[4 * g + q] = ok;
        sync_group();
        ok = s_ok[4 * g] && s_ok[4 * g + 1] && s_ok[4 * g + 2] && s_ok[4 * g + 3];
        if (!ok) break;
        tc_fence_after();
        if (32 * g >= n) {             // no columns of this group
          release();
          sync_group();                                 // s_ok read by all
          continue;
        }
        const size_t stride = (size_t)2 * BN * 128;      // floats of one slot
        // four columns of a lane are adjacent: 16-byte accesses
        const size_t at = (size_t)rank * BN * 128 + (q * 32 + lane) * 4;
        float* mine = p.part + (size_t)work.slot_of(pair, u) * stride + at;
#pragma unroll 1
        for (int c0 = 32 * g; c0 < n; c0 += 64) {
          tmem_ld32(tbuf + c0, v);
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            if (c0 + j < n)
              __stcg(reinterpret_cast<float4*>(mine + (size_t)(c0 + j) * 128), make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]));
        }
        release();
        sync_group();
        int c_lo, c_hi;
        work.owners(u, c_lo, c_hi);
        if (q == 0 && lane == 0) {
          __threadfence();                              // the group's sums, ordered by its barrier
          int32_t* ticket = p.tickets + 4 * (u - work.first) + 2 * rank + g;
          const int last = atomicAdd(ticket, 1) == c_hi - c_lo;
          if (last) *ticket = 0;                        // ready for the next call
          __threadfence();
          s_flag[g] = last;
        }
        sync_group();
        if (s_flag[g]) {
          // K order; few rows: the sums of four pieces in flight at a time, else of two
          const auto piece = [&](int c) {
            return reinterpret_cast<const float4*>(p.part + (size_t)work.slot_of(min(c, c_hi), u) * stride + at);
          };
          const auto add = [&](float* x, const float4& y, bool there) {
            x[0] += there ? y.x : 0.f;
            x[1] += there ? y.y : 0.f;
            x[2] += there ? y.z : 0.f;
            x[3] += there ? y.w : 0.f;
          };
          if (n <= 8) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = 0.f;
            for (int c = c_lo; c <= c_hi; c += 4) {
              float4 x[4][2];
#pragma unroll
              for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) x[i][j] = __ldcg(piece(c + i) + (4 * j < n ? j : 0) * 128);
#pragma unroll
              for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) add(&v[4 * j], x[i][j], c + i <= c_hi);
            }
            ft_store<EPI>(p, v, p0, n, col0, 0, q, lane);
          } else {
#pragma unroll 1
            for (int c0 = 32 * g; c0 < n; c0 += 64) {
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = 0.f;
              for (int c = c_lo; c <= c_hi; c += 2) {
                float4 x[2][8];
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                  for (int j = 0; j < 8; ++j) x[i][j] = __ldcg(piece(c + i) + (c0 / 4 + j) * 128);
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                  for (int j = 0; j < 8; ++j) add(&v[4 * j], x[i][j], c + i <= c_hi);
              }
              ft_store<EPI>(p, v, p0, n, col0, c0, q, lane);
            }
          }
        }
        sync_group();                                   // s_flag and s_ok read by all
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();        // no CTA leaves while the other may still signal it
  tc_fence_after();
  if (warp == 2) tmem2_dealloc(tmem, Cfg::kCols);
}

// ---------------------------------------------------------------------------------- host side

// Tile width, and whether the units that whole waves leave over are cut along K: the least of the estimated
// times.  A K step of a unit takes what its MMAs or its loads take, whichever is more; joining the pieces of a
// unit takes time by its rows of C and its pieces, two groups of warps adding them.  Estimates from
// us of the up projection and the down projection, at widths 32 / 64 / 128 / 256, c cut, w whole: H = 6144, I =
// 512, M = 48 27c / 24c / 24c / 25c (whole 30 to 33), M = 200 27c / 25c / 37c / 54c (35w / 33w / 34w / 36w), M = 777
// - / 39c / 36c / 44c (40w / 40w / 40w);  H = 7168, I = 1152, M = 400 71c / 49c / 45c / 53c (80w / 47w / 46w / 44w);
// H = I = 4096, M = 2048 - / 315w / 187w / 129w.
// Sums over tokens have both operands the other way round, whose boxes are 64 wide for each CTA: 128 at
// least.
// Units are cut at widths up to cut_bn, which the scratch buffer holds the pieces of.
struct FtPlan {
  int bn, cut;
};
static FtPlan ff_tc_plan(const FfGemm& g, int epilogue, int pairs, int cut_bn) {
  FtPlan best{256, 0};
  double least = 1e300;
  for (int bn = g.ck != 1 ? 128 : 32; bn <= 256; bn *= 2) {
    const int KT = cdiv(g.K, kFtK), tiles = cdiv(g.nc, bn);
    const double step = bn == 32 ? 235 : (bn == 64 ? 240 : (bn == 128 ? 267 : 334));     // ns
    const long long units = (long long)tiles * cdiv(g.nr, epilogue == kFfGlu ? 128 : 256);
    const long long waves = units / pairs, left = units % pairs;
    const double base = (double)waves * KT * step;
    double whole = base + (left ? KT * step : 0), cut = 1e300;
    if (left && bn <= cut_bn) {
      const double pieces = (double)pairs / left + 1, rows = cdiv(g.nc, tiles);
      cut = base + (double)left * KT / pairs * step + 3500 + rows * (75 + 4.3 * pieces);
    }
    if (whole <= least) {
      least = whole;
      best = {bn, 0};
    }
    if (cut < least) {
      least = cut;
      best = {bn, 1};
    }
    if (bn >= g.nc) break;             // one tile holds them all
  }
  return best;
}

// The widest tile that a plan of up to max_rows tokens cuts: the one that holds them all.  Wider ones are of
// the sums over tokens, whose K is the tokens: up to 128 of them are two K steps, which take less time than joining
// pieces does, so those products would not be cut anyway.
static int ff_cut_width(int max_rows) {
  return max_rows <= 32 ? 32 : (max_rows <= 64 ? 64 : (max_rows <= 128 ? 128 : 256));
}
// Scratch of cut units: [pairs][2][2 CTAs][BN][128] fp32 of that tile (5 MB up to 32 tokens, 42 past 128).
size_t ff_tc_part_bytes(int max_rows) {
  return (size_t)kGtMaxPairs * 2 * 2 * ff_cut_width(max_rows) * 128 * sizeof(float);
}

static bool ft_tmap(CUtensorMap* tm, bool bf16, int rank, const void* base, const cuuint64_t* dims,
                    const cuuint64_t* strides, const cuuint32_t* box) {
  EncodeTiledFn enc = tc_encode_fn();
  if (!enc) return false;
  const cuuint32_t es[5] = {1, 1, 1, 1, 1};
  return enc(tm, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
             (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int EPI, int BN>
static cudaError_t launch_ft(FtParams& p, cudaStream_t st) {
  using Cfg = FtCfg<BN>;
  auto kernel = ff_tc_kernel<EPI, BN>;
  static PerDevice<int> per;
  int pairs = 0;
  cudaError_t err = on_device(per, &pairs, [&](int* v) {
    cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t q = {};
    q.gridDim = dim3(2 * kGtMaxPairs);
    q.blockDim = dim3(kFtThreads);
    q.dynamicSmemBytes = Cfg::kSmem;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, kernel, &q);
    *v = n < 1 ? 1 : (n < kGtMaxPairs ? n : kGtMaxPairs);
    return e;
  });
  if (err != cudaSuccess) return err;
  const FfGemm& g = p.g;
  bool ok;
  p.whole16 = EPI == kFfGlu && g.nr % 16 == 0;
  const cuuint64_t row = (cuuint64_t)(p.r_mn ? g.rk : g.rs) * 2, half = (cuuint64_t)g.half * 2;
  if (EPI == kFfGlu && p.whole16) {
    // [I / 16 groups][2 halves][16 rows][K]
    const cuuint64_t dims[4] = {(cuuint64_t)g.K, 16, 2, (cuuint64_t)(g.nr / 16)};
    const cuuint64_t str[3] = {row, half, row * 16};
    const cuuint32_t box[4] = {kFtK, 16, 2, 4};
    ok = ft_tmap(&p.tm_r, p.bf16, 4, g.r, dims, str, box);
  } else if (EPI == kFfGlu) {
    const cuuint64_t dims[3] = {(cuuint64_t)g.K, (cuuint64_t)g.nr, 2};
    const cuuint64_t str[2] = {row, half};
    const cuuint32_t box[3] = {kFtK, 16, 2};
    ok = ft_tmap(&p.tm_r, p.bf16, 3, g.r, dims, str, box);
  } else {
    const cuuint64_t dims[2] = {(cuuint64_t)(p.r_mn ? g.nr : g.K), (cuuint64_t)(p.r_mn ? g.K : g.nr)};
    const cuuint32_t box[2] = {64, p.r_mn ? (cuuint32_t)kFtK : 128u};
    ok = ft_tmap(&p.tm_r, p.bf16, 2, g.r, dims, &row, box);
  }
  const cuuint64_t cdims[2] = {(cuuint64_t)(p.c_mn ? g.nc : g.K), (cuuint64_t)(p.c_mn ? g.K : g.nc)};
  const cuuint64_t crow = (cuuint64_t)(p.c_mn ? g.ck : g.cs) * 2;
  const cuuint32_t cbox[2] = {64, p.c_mn ? (cuuint32_t)kFtK : (cuuint32_t)Cfg::kHalf};
  ok = ok && ft_tmap(&p.tm_c, p.bf16, 2, g.c, cdims, &crow, cbox);
  if (!ok) return cudaErrorInvalidValue;
  p.RB = cdiv(g.nr, EPI == kFfGlu ? 128 : 256);
  p.tiles = cdiv(g.nc, BN);
  p.size = p.tiles > 1 ? 16 * cdiv(cdiv(g.nc, p.tiles), 16) : BN;
  // no more pairs than K steps can keep busy
  const long long units = (long long)p.tiles * p.RB;
  const long long useful = units * (p.KT < kGtMinSteps ? 1 : cdiv(p.KT, kGtMinSteps));
  const int G = useful < pairs ? (int)useful : pairs;
  return launch_kernel(kernel, dim3(2 * G), dim3(kFtThreads), Cfg::kSmem, st, true, p);
}

template <int EPI>
static cudaError_t launch_ft_bn(FtParams& p, cudaStream_t st) {
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
  const FtPlan plan = ff_tc_plan(p.g, EPI, pairs, ff_cut_width(p.d.max_rows));
  p.cut = plan.cut;
  switch (plan.bn) {
    case 32: return launch_ft<EPI, 32>(p, st);
    case 64: return launch_ft<EPI, 64>(p, st);
    case 128: return launch_ft<EPI, 128>(p, st);
    default: return launch_ft<EPI, 256>(p, st);
  }
}

// Whether the tile copies can address the operands: 16-byte bases and strides.
bool ff_tc_addressable(const FfGemm& g) {
  const auto on16 = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0; };
  const long long ldr = g.rk == 1 ? g.rs : g.rk, ldc = g.ck == 1 ? g.cs : g.ck;
  return on16(g.r) && on16(g.c) && ldr % 8 == 0 && ldc % 8 == 0 && g.half % 8 == 0 && ldr < (1LL << 38) &&
         ldc < (1LL << 38) && g.half < (1LL << 38);
}

cudaError_t launch_ff_tc(const FfDims& d, const FfGemm& g, int epilogue, float* part, int32_t* tickets,
                         cudaStream_t st) {
  FtParams p;
  p.d = d;
  p.g = g;
  p.part = part;
  p.tickets = tickets;
  p.KT = cdiv(g.K, kFtK);
  p.r_mn = g.rk != 1;
  p.c_mn = g.ck != 1;
  p.bf16 = d.dtype == MOE_DTYPE_BF16;
  p.packed = g.nr % 2 == 0 && g.ldo % 2 == 0 && (reinterpret_cast<uintptr_t>(g.out) & 3) == 0 &&
             (reinterpret_cast<uintptr_t>(g.pre) & 7) == 0;
  if (epilogue == kFfGlu) return launch_ft_bn<kFfGlu>(p, st);
  if (epilogue == kFfGrad) return launch_ft_bn<kFfGrad>(p, st);
  return launch_ft_bn<kFfStore>(p, st);
}

}  // namespace moe
