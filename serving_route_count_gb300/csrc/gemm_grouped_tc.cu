// gemm_grouped_tc.cu - products grouped by expert with ragged sizes on the tensor cores
// (moe_grouped_run): out[p] = act(W[e] . x[row(p)]).
//
// The weight rows are the MMA's M operand and the tile's tokens its N operand, so an expert with
// one row still streams its weights once, through full-size MMAs.  A pair of CTAs (one MMA of 256
// weight rows, tcgen05 cta_group::2) owns a unit: 256 weight rows of one expert (for a SwiGLU 128
// up and 128 gate rows, interleaved 16 by 16, so that a warp's 32 accumulator lanes hold both
// halves of 16 outputs) x up to BN of the expert's tokens.  Each CTA loads its 128 weight rows and
// half of the tokens per K step of 64; the accumulators are double-buffered in tensor memory, so
// a unit's epilogue runs under the next unit's loads and MMAs.
//
// The grid is persistent, one pair per two SMs.  The number of units is known on the device only
// (offsets); every CTA builds the table of the experts' tiles in shared memory.  Whole waves of
// units go round robin; the units left over are cut evenly by K steps, every piece's fp32 sums go
// to the scratch buffer, and the piece that arrives last adds them in K order (bit-stable, nobody
// waits).
//
// Roles: warp 0 weight copies, warp 1 MMA issue (leader CTA), warp 2 token copies (tiles, or
// gathers of four rows by index), warp 3 tensor memory, warps 4-7 epilogue.
#include <type_traits>

#include "block_ops.cuh"
#include "grouped.cuh"
#include "tc_ptx.cuh"
#include "tc_tile.cuh"
#include "../../include/moe_gb300.h"

namespace moe {
using namespace tc;

constexpr int kGtThreads = 384;
constexpr int kGtK = 64;                 // K step: one 128-byte swizzled row per operand row
constexpr int kGtMaxPairs = 80;          // pairs that the scratch buffer has partial slots for
constexpr int kGtTokenWarps = 6;         // warps 2-7
constexpr int kGtMinSteps = 4;           // K steps below which a piece is not cut further

template <int BN>
struct GtCfg {
  static constexpr int kHalf = BN / 2;                       // tokens a CTA loads
  static constexpr int kChunk = kHalf < 32 ? kHalf : 32;     // tokens per tile copy
  static constexpr int kBytesA = 128 * 128, kBytesB = kHalf * 128, kStage = kBytesA + kBytesB;
  static constexpr int kTables = 3 * 1028 * 4 + 512;         // expert tables, barriers
  static constexpr int kStages = (227 * 1024 - 1024 - kTables) / kStage > 12
                                     ? 12 : (227 * 1024 - 1024 - kTables) / kStage;
  static constexpr int kSmem = 1024 + kStages * kStage + kTables;
  static constexpr int kCols = 2 * BN;                       // tensor-memory columns
};

struct GtParams {
  CUtensorMap tm_w, tm_x;
  GroupedDims d;
  GroupedCall c;
  float* part;          // [pairs][2][2 CTAs][BN][128]
  int32_t* tickets;     // [pairs][2]
  int KT, RB, cols, packed;
};

// Units of one pair: first its range of the leftover units' K steps, then its whole units.
struct GtWork {
  int KT, G, Gs, c, D, first;      // first: units before it are whole
  uint32_t W, x, x1;
  int dp;
  __device__ __forceinline__ void init(int units, int kt, int g, int cta) {
    KT = kt; G = g; c = cta;
    D = units / g;
    first = D * g;
    const uint32_t R = (uint32_t)(units - first);
    W = R * (uint32_t)kt;
    // pairs that share the leftover steps: all of them, unless the pieces got too short
    const uint32_t most = W / kGtMinSteps > R ? W / kGtMinSteps : R;
    Gs = most < (uint32_t)g ? (int)most : g;
    x = cta < Gs ? begin_of(cta) : 0u;
    x1 = cta < Gs ? begin_of(cta + 1) : 0u;
    dp = 0;
  }
  __device__ __forceinline__ uint32_t begin_of(int cta) const {
    return (uint32_t)cta * W / (uint32_t)Gs;
  }
  __device__ __forceinline__ bool next(int& u, int& k0, int& len) {
    if (x < x1) {
      const uint32_t kt = (uint32_t)KT;
      u = first + (int)(x / kt);
      k0 = (int)(x % kt);
      len = (int)min(kt - (uint32_t)k0, x1 - x);
      x += (uint32_t)len;
      return true;
    }
    if (dp < D) {
      u = c + dp * G;
      k0 = 0;
      len = KT;
      ++dp;
      return true;
    }
    return false;
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

// A unit's expert, token range and weight row block.
struct GtUnit {
  int e, p0, n, nhalf, rb;
};
template <int BN>
__device__ __forceinline__ GtUnit gt_unit(int u, int RB, int E, const int* s_tile,
                                          const int* s_off, const int* s_cnt) {
  constexpr int kChunk = GtCfg<BN>::kChunk;
  const int tile = u / RB;
  int lo = 0, hi = E;                 // last e with s_tile[e] <= tile
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s_tile[mid] <= tile) lo = mid; else hi = mid;
  }
  GtUnit r;
  r.e = lo;
  const int t = tile - s_tile[lo];
  r.p0 = s_off[lo] + t * BN;
  r.n = min(BN, s_cnt[lo] - t * BN);
  r.nhalf = cdiv(r.n, 2 * kChunk) * kChunk;
  r.rb = u - tile * RB;
  return r;
}

// Stores 32 accumulator columns (tokens c0 .. c0 + 31 of the unit, n of them valid) of this
// lane's row.  A lane and its neighbour exchange every other token, so that each store writes
// two adjacent output columns.
template <typename T, bool ACT>
__device__ __forceinline__ void gt_store(const GtParams& p, float (&v)[32], const GtUnit& un,
                                         int c0, int rank, int q, int lane) {
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
    const int col = un.rb * 128 + rank * 64 + q * 16 + (lane & 15);
    const int t0 = c0 + (hi ? 16 : 0);
    if (p.packed) {
      T* o = out + (size_t)(un.p0 + t0 + odd) * p.c.ldo + (col & ~1);
#pragma unroll
      for (int c = 0; c < 16; c += 2) {
        const float got = __shfl_xor_sync(0xffffffffu, odd ? h[c] : h[c + 1], 1);
        const T pair[2] = {from_f32<T>(odd ? got : h[c]), from_f32<T>(odd ? h[c + 1] : got)};
        uint32_t w;
        memcpy(&w, pair, 4);
        if (t0 + c + odd < un.n && col < p.cols) *reinterpret_cast<uint32_t*>(o) = w;
        o += 2 * p.c.ldo;
      }
    } else {
#pragma unroll
      for (int c = 0; c < 16; ++c)
        if (t0 + c < un.n && col < p.cols)
          out[(size_t)(un.p0 + t0 + c) * p.c.ldo + col] = from_f32<T>(h[c]);
    }
  } else {
    const int col = un.rb * 256 + rank * 128 + q * 32 + lane;
    if (p.packed) {
      T* o = out + (size_t)(un.p0 + c0 + odd) * p.c.ldo + (col & ~1);
#pragma unroll
      for (int c = 0; c < 32; c += 2) {
        const float got = __shfl_xor_sync(0xffffffffu, odd ? v[c] : v[c + 1], 1);
        const T pair[2] = {from_f32<T>(odd ? got : v[c]), from_f32<T>(odd ? v[c + 1] : got)};
        uint32_t w;
        memcpy(&w, pair, 4);
        if (c0 + c + odd < un.n && col < p.cols) *reinterpret_cast<uint32_t*>(o) = w;
        o += 2 * p.c.ldo;
      }
    } else {
#pragma unroll
      for (int c = 0; c < 32; ++c)
        if (c0 + c < un.n && col < p.cols)
          out[(size_t)(un.p0 + c0 + c) * p.c.ldo + col] = from_f32<T>(v[c]);
    }
  }
}

template <typename T, bool ACT, int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGtThreads, 1)
grouped_tc_kernel(const __grid_constant__ GtParams p) {
  using Cfg = GtCfg<BN>;
  constexpr int S = Cfg::kStages;
  extern __shared__ uint8_t raw[];
  uint8_t* st = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(st + S * Cfg::kStage);   // [S] (leader's are used)
  uint64_t* empty = full + S;          // [S]
  uint64_t* tfull = empty + S;         // [2] accumulators ready
  uint64_t* tempty = tfull + 2;        // [2] accumulators read (leader's are used)
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(tempty + 2);
  int* s_flag = reinterpret_cast<int*>(s_tmem + 1);
  int* s_warp = s_flag + 1;            // [warps]
  int* s_off = reinterpret_cast<int*>(st + S * Cfg::kStage + 512);
  int* s_cnt = s_off + 1028;
  int* s_tile = s_cnt + 1028;
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
      mbar_init(&tempty[b], 8);
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

  // the experts' tiles: thread t owns experts 4 t .. 4 t + 3
  int cnt[4], tiles = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = 4 * tid + i;
    cnt[i] = 0;
    if (e < E) {
      const int a = p.c.offsets[e], b = p.c.offsets[e + 1];
      if (a < 0 || b < a || b > p.c.S)
        set_error(err, kErrRouteBounds);
      else
        cnt[i] = b - a;
      s_off[e] = a;
      s_cnt[e] = cnt[i];
    }
    tiles += cdiv(cnt[i], BN);
  }
  int incl = tiles;
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  int before = incl - tiles, total = 0;
#pragma unroll
  for (int w = 0; w < kGtThreads / 32; ++w) {
    if (w < warp) before += s_warp[w];
    total += s_warp[w];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (4 * tid + i < E) s_tile[4 * tid + i] = before;
    before += cdiv(cnt[i], BN);
  }
  // rows past the last group
  {
    const int end = max(0, min(p.c.S, p.c.offsets[E]));
    T* out = static_cast<T*>(p.c.out);
    for (long long r = end + (long long)blockIdx.x; r < p.c.S; r += gridDim.x)
      for (int c = tid; c < p.cols; c += kGtThreads) out[r * p.c.ldo + c] = from_f32<T>(0.f);
  }
  __syncthreads();

  GtWork work;
  work.init(total * p.RB, p.KT, G, pair);
  int u, k0, len;
  bool ok = true;
  if (warp == 0) {
    if (lane == 0) {
      int it = 0;
      while (ok && work.next(u, k0, len)) {
        const GtUnit un = gt_unit<BN>(u, p.RB, E, s_tile, s_off, s_cnt);
        const uint32_t bytes = 2u * (Cfg::kBytesA + un.nhalf * 128);
        const int r0 = ACT ? un.rb * 128 + (int)rank * 64 : un.rb * 256 + (int)rank * 128;
        for (int k = k0; k < k0 + len; ++k, ++it) {
          const int s = it % S;
          if (!mbar_wait(&empty[s], ((it / S) & 1) ^ 1, err)) {
            ok = false;
            break;
          }
          uint8_t* a = st + s * Cfg::kStage;
          const uint32_t bar = map_rank(&full[s], 0);
          if (rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
          if constexpr (ACT) {
#pragma unroll
            for (int b = 0; b < 4; ++b)
              tma2_load_4d(a + b * 4096, &p.tm_w, k * kGtK, r0 + 16 * b, 0, un.e, bar);
          } else {
            tma2_load_3d(a, &p.tm_w, k * kGtK, r0, un.e, bar);
          }
        }
      }
      if (ok) {
        // the last fills have been multiplied: nothing arrives at this CTA's barriers any more
        for (int j = it > S ? it - S : 0; j < it; ++j) mbar_wait(&empty[j % S], (j / S) & 1, err);
      } else if (rank == 0) {
        drain_stage_loads<S>(full, it, err);
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      int it = 0, seg = 0;
      while (ok && work.next(u, k0, len)) {
        const GtUnit un = gt_unit<BN>(u, p.RB, E, s_tile, s_off, s_cnt);
        const int b = seg & 1;
        if (!mbar_wait(&tempty[b], ((seg >> 1) & 1) ^ 1, err)) break;
        tc_fence_after();
        const uint32_t idesc = idesc_pair16(std::is_same<T, __nv_bfloat16>::value, 2 * un.nhalf);
        for (int i = 0; i < len; ++i, ++it) {
          const int s = it % S;
          if (!mbar_wait(&full[s], (it / S) & 1, err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint8_t* a = st + s * Cfg::kStage;
#pragma unroll
          for (int kb = 0; kb < 4; ++kb)
            mma2_f16(tmem + b * BN, desc_sw128(a + 32 * kb), desc_sw128(a + Cfg::kBytesA + 32 * kb),
                     idesc, (i > 0 || kb > 0) ? 1u : 0u);
          tc2_commit(&empty[s]);
        }
        tc2_commit(&tfull[b]);
        ++seg;
      }
    }
  } else if (warp < 2 + kGtTokenWarps) {
    const int tl = lane * kGtTokenWarps + (warp - 2);
    int it = 0;
    while (ok && work.next(u, k0, len)) {
      const GtUnit un = gt_unit<BN>(u, p.RB, E, s_tile, s_off, s_cnt);
      const int first = un.p0 + (int)rank * un.nhalf;
      int4 rows = make_int4(0, 0, 0, 0);
      if (p.c.perm != nullptr) {
        // rows 4 tl .. 4 tl + 3 of this CTA's tokens; past the tile its last row again
        int r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int f = p.c.perm[min(first + 4 * tl + i, un.p0 + un.n - 1)];
          r[i] = f < 0 ? -1 : f / p.c.topk;
          if (r[i] < 0 || r[i] >= p.c.x_rows) {
            set_error(err, kErrRouteBounds);
            r[i] = 0;
          }
        }
        rows = make_int4(r[0], r[1], r[2], r[3]);
      }
      for (int k = k0; k < k0 + len; ++k, ++it) {
        const int s = it % S;
        if (!mbar_wait_warp(&empty[s], ((it / S) & 1) ^ 1, err)) {
          ok = false;
          break;
        }
        uint8_t* bs = st + s * Cfg::kStage + Cfg::kBytesA;
        const uint32_t bar = map_rank(&full[s], 0);
        if (p.c.perm != nullptr) {
          if (tl < un.nhalf / 4) tma2_gather4(bs + tl * 512, &p.tm_x, k * kGtK, rows, bar);
        } else if (tl * Cfg::kChunk < un.nhalf) {
          tma2_load_2d(bs + tl * Cfg::kChunk * 128, &p.tm_x, k * kGtK, first + tl * Cfg::kChunk, bar);
        }
      }
    }
  } else {
    const int q = warp & 3;
    const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16);
    int seg = 0;
    while (work.next(u, k0, len)) {
      const GtUnit un = gt_unit<BN>(u, p.RB, E, s_tile, s_off, s_cnt);
      const int b = seg & 1;
      if (!mbar_wait_warp(&tfull[b], (seg >> 1) & 1, err)) ok = false;
      // one verdict for the four warps, whose named barriers below all of them must reach
      if (lane == 0) s_warp[q] = ok;
      asm volatile("bar.sync 1, 128;" ::: "memory");
      ok = s_warp[0] && s_warp[1] && s_warp[2] && s_warp[3];
      asm volatile("bar.sync 1, 128;" ::: "memory");
      if (!ok) break;
      tc_fence_after();
      float v[32];
      if (len == p.KT) {
#pragma unroll 1
        for (int c0 = 0; c0 < un.n; c0 += 32) {
          tmem_ld32(trow + b * BN + c0, v);
          gt_store<T, ACT>(p, v, un, c0, (int)rank, q, lane);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(map_rank(&tempty[b], 0));
      } else {
        const size_t stride = (size_t)2 * BN * 128;     // floats of one slot
        const size_t at = (size_t)rank * BN * 128 + q * 32 + lane;
        float* mine = p.part + (size_t)work.slot_of(pair, u) * stride + at;
#pragma unroll 1
        for (int c0 = 0; c0 < un.n; c0 += 32) {
          tmem_ld32(trow + b * BN + c0, v);
#pragma unroll
          for (int j = 0; j < 32; ++j) __stcg(mine + (size_t)(c0 + j) * 128, v[j]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(map_rank(&tempty[b], 0));
        __threadfence();
        asm volatile("bar.sync 1, 128;" ::: "memory");
        int c_lo, c_hi;
        work.owners(u, c_lo, c_hi);
        if (tid == kGtThreads - 128) {
          int32_t* ticket = p.tickets + 2 * (u - work.first) + rank;
          const int last = atomicAdd(ticket, 1) == c_hi - c_lo;
          if (last) *ticket = 0;                        // ready for the next call
          *s_flag = last;
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (*s_flag) {
          __threadfence();
#pragma unroll 1
          for (int c0 = 0; c0 < un.n; c0 += 32) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = 0.f;
#pragma unroll 1
            for (int c = c_lo; c <= c_hi; ++c) {
              const float* src = p.part + (size_t)work.slot_of(c, u) * stride + at;
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] += __ldcg(src + (size_t)(c0 + j) * 128);
            }
            gt_store<T, ACT>(p, v, un, c0, (int)rank, q, lane);
          }
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");  // s_flag read by all
      }
      ++seg;
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();        // no CTA leaves while the other may still signal it
  tc_fence_after();
  if (warp == 3) tmem2_dealloc(tmem, Cfg::kCols);
}

// ---------------------------------------------------------------------------------- host side

// Token-tile width by the expected positions per expert.
int grouped_tc_bn(int S, int E) {
  if ((long long)S <= 8LL * E) return 32;
  if ((long long)S <= 24LL * E) return 64;
  if ((long long)S <= 64LL * E) return 128;
  return 256;
}

size_t grouped_tc_part_bytes(int S, int E) {
  return (size_t)kGtMaxPairs * 2 * 2 * grouped_tc_bn(S, E) * 128 * sizeof(float);
}
size_t grouped_tc_ticket_bytes() { return (size_t)kGtMaxPairs * 2 * sizeof(int32_t); }

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

template <typename T, bool ACT, int BN>
static cudaError_t launch_gt(GtParams& p, cudaStream_t st) {
  using Cfg = GtCfg<BN>;
  auto kernel = grouped_tc_kernel<T, ACT, BN>;
  static int pairs = 0;
  if (pairs == 0) {
    cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t q = {};
    q.gridDim = dim3(2 * kGtMaxPairs);
    q.blockDim = dim3(kGtThreads);
    q.dynamicSmemBytes = Cfg::kSmem;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, kernel, &q);
    if (e != cudaSuccess) return e;
    pairs = n < 1 ? 1 : (n < kGtMaxPairs ? n : kGtMaxPairs);
  }
  const bool bf16 = std::is_same<T, __nv_bfloat16>::value;
  const GroupedDims& d = p.d;
  const GroupedCall& c = p.c;
  bool ok;
  if (ACT) {
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
  // no more pairs than K steps can keep busy
  const long long units = ((long long)cdiv(c.S, BN) + (d.E < c.S ? d.E : c.S)) * p.RB;
  const long long useful = units * (p.KT < kGtMinSteps ? 1 : cdiv(p.KT, kGtMinSteps));
  const int G = useful < pairs ? (int)useful : pairs;
  return launch_kernel(kernel, dim3(2 * G), dim3(kGtThreads), Cfg::kSmem, st, true, p);
}

template <typename T, bool ACT>
static cudaError_t launch_gt_bn(GtParams& p, cudaStream_t st) {
  switch (grouped_tc_bn(p.c.S, p.d.E)) {
    case 32: return launch_gt<T, ACT, 32>(p, st);
    case 64: return launch_gt<T, ACT, 64>(p, st);
    case 128: return launch_gt<T, ACT, 128>(p, st);
    default: return launch_gt<T, ACT, 256>(p, st);
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
  p.RB = cdiv(p.cols, d.act ? 128 : 256);
  p.packed = p.cols % 2 == 0 && c.ldo % 2 == 0 && (reinterpret_cast<uintptr_t>(c.out) & 3) == 0;
  if (d.dtype == MOE_DTYPE_F16)
    return d.act ? launch_gt_bn<__half, true>(p, st) : launch_gt_bn<__half, false>(p, st);
  return d.act ? launch_gt_bn<__nv_bfloat16, true>(p, st) : launch_gt_bn<__nv_bfloat16, false>(p, st);
}

}  // namespace moe
