// block_route.cu - the router's top-k selection (moe_router) and the grouping of the slots by
// expert (moe_group) for callers of the grouped products.
#include <cooperative_groups.h>

#include <cmath>

#include "block_ops.cuh"
#include "../../include/moe_gb300.h"

namespace moe {

// ---------------------------------------------------------------------------------- router
//
// One warp per token; lane l holds the keys of experts l, l + 32, ... (VPL of them) as integers
// that order like the floats, with 0 for a masked expert.  The j-th choice is a warp maximum of
// the lanes' best keys and, among the lanes that hold it, the minimum of their lowest indices
// (two reductions of the warp's integer unit); the winner's lane clears that key and every lane
// rescans its own.  With eight keys a lane and more, the rounds run over the few keys that can be
// chosen at all.  8192 tokens: 256 fp32 logits, top-8 7.0 us (with all keys in every round 8.3), 512
// top-10 9.6 (15.9), 1024 top-16 19.5 (43); bound by instruction issue (8192 x 256 are 1.3 us of HBM
// time).  One token x 384, top-6, sigmoid + bias: 3.4 us of latency.
constexpr int kRouterWarps = 4;

// Integer that orders like v (0: NaN or -inf, which are never chosen; -0 and +0 alike).
__device__ __forceinline__ uint32_t order_key(float v) {
  if (!(v > -INFINITY)) return 0u;
  const uint32_t u = __float_as_uint(v + 0.f);
  return (u >> 31) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t k) {
  if (k == 0u) return -INFINITY;
  return __uint_as_float((k >> 31) ? (k & 0x7FFFFFFFu) : ~k);
}

// 1 / (1 + e^-l): IEEE operations only, so that equal logits and biases give the keys of the
// same formula computed elsewhere.
__device__ __forceinline__ float sigmoid_ieee(float l) {
  return __fdiv_rn(1.f, __fadd_rn(1.f, expf(-l)));
}

template <typename T, int VPL>
__global__ void __launch_bounds__(kRouterWarps * 32)
router_kernel(const T* __restrict__ logits, long long ld, const float* __restrict__ bias, int M,
              int E, int topk, int score, int n_group, int topk_group, int renorm, float scale,
              int32_t* __restrict__ ids, float* __restrict__ weights) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kRouterWarps + (threadIdx.x >> 5);
  pdl_wait_prev();
  pdl_launch_next();
  if (t >= M) return;
  const unsigned full = 0xffffffffu;
  const T* row = logits + (size_t)t * ld;

  float v[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 32 * i;
    v[i] = e < E ? to_f32(row[e]) : -INFINITY;
  }
  // the bias with the logits, not under their tests below (one token x 384: 5.2 -> 3.4 us), while
  // registers allow (1024 experts: 19 -> 25 us)
  constexpr bool kHeld = VPL <= 16;
  float b[kHeld ? VPL : 1];
  if constexpr (kHeld) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane + 32 * i;
      b[i] = bias != nullptr && e < E ? bias[e] : 0.f;
    }
  }
  // softmax over every expert that is not masked (max and sum; needed when not renormalised)
  float smax = -INFINITY, ssum = 0.f;
  if (score == MOE_SCORE_SOFTMAX && !renorm) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) smax = fmaxf(smax, v[i]);   // fmaxf drops NaN
    for (int o = 16; o > 0; o >>= 1) smax = fmaxf(smax, __shfl_xor_sync(full, smax, o));
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (v[i] > -INFINITY) ssum += v[i] == smax ? 1.f : expf(v[i] - smax);
    for (int o = 16; o > 0; o >>= 1) ssum += __shfl_xor_sync(full, ssum, o);
  }
  uint32_t key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    float k = v[i];
    if (score == MOE_SCORE_SIGMOID && k > -INFINITY) {
      k = sigmoid_ieee(k);
      if (bias != nullptr) k = __fadd_rn(k, kHeld ? b[kHeld ? i : 0] : bias[lane + 32 * i]);
    }
    key[i] = order_key(k);
  }

  if (n_group > 1) {
    const int gs = E / n_group;
    uint32_t mine = 0u;                       // lane g: run g's key
    for (int g = 0; g < n_group; ++g) {
      uint32_t a = 0u, b = 0u;                // this lane's two largest keys of the run
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int e = lane + 32 * i;
        if (e >= g * gs && e < (g + 1) * gs) {
          b = max(b, min(a, key[i]));
          a = max(a, key[i]);
        }
      }
      const uint32_t m1 = __reduce_max_sync(full, a);
      uint32_t r = m1;
      if (score == MOE_SCORE_SIGMOID && gs > 1) {
        const int first = __ffs(__ballot_sync(full, a == m1)) - 1;
        const uint32_t m2 = __reduce_max_sync(full, lane == first ? b : a);
        r = order_key(__fadd_rn(order_value(m1), order_value(m2)));
      }
      if (lane == g) mine = r;
    }
    int rank = 0;
    for (int g = 0; g < n_group; ++g) {
      const uint32_t other = __shfl_sync(full, mine, g);
      rank += other > mine || (other == mine && g < lane);
    }
    const unsigned stay = __ballot_sync(full, lane < n_group && rank < topk_group);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane + 32 * i;
      if (e < E && !((stay >> (e / gs)) & 1u)) key[i] = 0u;
    }
  }

  int id = -1;                                // lane j: the j-th choice
  bool chosen = false;
  if (VPL >= 8 && topk <= 16) {
    // The topk-th largest of the lanes' largest keys bounds the choice from below, and few keys reach
    // it (about 12 of 256 for top-8): those are packed one to a lane, in ascending index, and the
    // rounds go over them alone.  Where more than 32 reach it (ties, or topk near 32: 26.5 against 22.9
    // us at top-32 of 256) the rounds below go over all keys.
    __shared__ uint2 s_few[kRouterWarps][32];
    uint2* few = s_few[threadIdx.x >> 5];
    uint32_t best = 0u;
#pragma unroll
    for (int i = 0; i < VPL; ++i) best = max(best, key[i]);
    uint32_t bound = 1u;                      // every key that is not masked
    for (int left = topk; left > 0;) {
      const uint32_t top = __reduce_max_sync(full, best);
      if (top == 0u) {
        bound = 1u;
        break;
      }
      bound = top;
      left -= __popc(__ballot_sync(full, best == top));
      if (best == top) best = 0u;
    }
    unsigned reach[VPL];
    int n = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      reach[i] = __ballot_sync(full, key[i] >= bound);
      n += __popc(reach[i]);
    }
    if (n <= 32) {
      n = 0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        if (key[i] >= bound)
          few[n + __popc(reach[i] & ((1u << lane) - 1u))] = make_uint2(key[i], lane + 32 * i);
        n += __popc(reach[i]);
      }
      __syncwarp();
      const uint2 mine = lane < n ? few[lane] : make_uint2(0u, 0u);
      uint32_t k = mine.x;
      for (int j = 0; j < topk; ++j) {
        const uint32_t top = __reduce_max_sync(full, k);
        if (top == 0u) break;
        const int at = __ffs(__ballot_sync(full, k == top)) - 1;   // the lowest index
        const int e = __shfl_sync(full, (int)mine.y, at);
        if (lane == j) id = e;
        if (lane == at) k = 0u;
      }
      chosen = true;
    }
  }
  for (int j = 0; !chosen && j < topk; ++j) {
    uint32_t best = 0u;
    int at = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (key[i] > best) {                    // strict: the lowest of the lane's equal keys
        best = key[i];
        at = i;
      }
    const uint32_t top = __reduce_max_sync(full, best);
    if (top == 0u) break;                     // uniform: nothing left to choose
    const int e = (int)__reduce_min_sync(full, best == top ? (unsigned)(lane + 32 * at) : ~0u);
    if (lane == j) id = e;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (e == lane + 32 * i) key[i] = 0u;
  }

  float s = 0.f;
  if (id >= 0) s = to_f32(row[id]);
  if (score == MOE_SCORE_SIGMOID) {
    s = id >= 0 ? sigmoid_ieee(s) : 0.f;
  } else {
    if (renorm) {                             // the softmax's sum cancels: relative to the best chosen
      smax = id >= 0 ? s : -INFINITY;
      for (int o = 16; o > 0; o >>= 1) smax = fmaxf(smax, __shfl_xor_sync(full, smax, o));
      ssum = 1.f;
    }
    s = id >= 0 ? (s == smax ? 1.f : expf(s - smax)) / ssum : 0.f;
  }
  if (renorm) {
    float sum = s;
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(full, sum, o);
    s = sum > 0.f ? s / sum : 0.f;
  }
  if (lane < topk) {
    ids[(size_t)t * topk + lane] = id;
    weights[(size_t)t * topk + lane] = s * scale;
  }
}

template <typename T>
static cudaError_t launch_router_t(const void* logits, long long ld, const float* bias, int M,
                                   int E, int topk, int score, int n_group, int topk_group,
                                   int renorm, float scale, int32_t* ids, float* weights,
                                   cudaStream_t st) {
  const dim3 grid(cdiv(M, kRouterWarps)), block(kRouterWarps * 32);
  const T* l = static_cast<const T*>(logits);
  auto go = [&](auto kernel) {
    return launch_kernel(kernel, grid, block, 0, st, true, l, ld, bias, M, E, topk, score, n_group,
                         topk_group, renorm, scale, ids, weights);
  };
  if (E <= 64) return go(router_kernel<T, 2>);
  if (E <= 128) return go(router_kernel<T, 4>);
  if (E <= 256) return go(router_kernel<T, 8>);
  if (E <= 384) return go(router_kernel<T, 12>);
  if (E <= 512) return go(router_kernel<T, 16>);
  return go(router_kernel<T, 32>);
}

cudaError_t launch_router(const void* logits, int dtype, long long ld, const float* bias, int M,
                          int E, int topk, int score, int n_group, int topk_group, int renorm,
                          float scale, int32_t* ids, float* weights, cudaStream_t st) {
  auto go = dtype == MOE_DTYPE_F32   ? launch_router_t<float>
            : dtype == MOE_DTYPE_F16 ? launch_router_t<__half>
                                     : launch_router_t<__nv_bfloat16>;
  return go(logits, ld, bias, M, E, topk, score, n_group, topk_group, renorm, scale, ids, weights,
            st);
}

// ---------------------------------------------------------------------------------- group
//
// Stable counting sort of S slots by expert in one launch: a cluster of C CTAs, each warp of
// which owns a contiguous range of slots.  Every warp counts its range in its own row of a
// shared-memory table; a CTA turns the table's columns into prefixes over its warps and
// publishes its totals; after a cluster barrier each CTA adds up all CTAs' totals through
// distributed shared memory (offsets, and what comes before its own slots), and the warps walk
// their ranges again, ranking equal experts of 32 slots by a warp match.  Bound by the second walk
// (the 4-byte stores of perm in expert order) per CTA: 8192 tokens top-8 over 256 experts take 77 /
// 40 / 22 / 13 / 9.6 us on 1 / 2 / 4 / 8 / 16 CTAs; 16 tokens top-6 3.3 us.
constexpr int kGroupMaxExperts = 1024;

inline size_t group_smem(int warps, int E) { return (size_t)(warps + 3) * E * sizeof(int); }

__global__ void __launch_bounds__(kGroupThreads)
group_kernel(const int32_t* __restrict__ ids, int S, int E, int first, int per_cta, int per_warp,
             int warps, int32_t* __restrict__ offsets, int32_t* __restrict__ perm,
             int32_t* __restrict__ slot_of) {
  namespace cg = cooperative_groups;
  extern __shared__ int sm[];
  int* cnt = sm;                       // [warps][E] counts, then prefixes over the warps
  int* tot = sm + (size_t)warps * E;   // [E] this CTA's totals, read by the other CTAs
  int* base = tot + E;                 // [E] position of this CTA's first slot of the expert
  int* all = base + E;                 // [E] totals of all CTAs
  __shared__ int s_warp[32];
  cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)cl.block_rank(), C = (int)cl.num_blocks();
  pdl_wait_prev();
  pdl_launch_next();

  const int lo = min(S, rank * per_cta + warp * per_warp);
  const int hi = min(min(S, lo + per_warp), (rank + 1) * per_cta);
  for (int i = tid; i < warps * E; i += kGroupThreads) cnt[i] = 0;
  __syncthreads();
  if (warp < warps)
    for (int f = lo + lane; f < hi; f += 32) {
      const int e = local_expert(ids[f], first, E);
      if (e >= 0) atomicAdd(&cnt[warp * E + e], 1);
    }
  __syncthreads();
  for (int e = tid; e < E; e += kGroupThreads) {
    int run = 0;
    for (int w = 0; w < warps; ++w) {
      const int c = cnt[w * E + e];
      cnt[w * E + e] = run;
      run += c;
    }
    tot[e] = run;
  }
  cl.sync();
  for (int e = tid; e < E; e += kGroupThreads) {
    int before = 0, total = 0;
    for (int r = 0; r < C; ++r) {
      const int c = cl.map_shared_rank(tot, r)[e];
      before += r < rank ? c : 0;
      total += c;
    }
    base[e] = before;
    all[e] = total;
  }
  __syncthreads();
  // E <= kGroupThreads: one expert per thread
  const int mine = tid < E ? all[tid] : 0;
  int x = mine;
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = s_warp[lane];
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  const int excl = x - mine + (warp ? s_warp[warp - 1] : 0);
  const int valid = s_warp[31];
  if (tid < E) {
    base[tid] += excl;
    if (rank == 0) offsets[tid] = excl;
  }
  if (rank == 0 && tid == 0) offsets[E] = valid;
  __syncthreads();
  if (warp < warps) {
    const unsigned below = (1u << lane) - 1u;
    for (int f0 = lo; f0 < hi; f0 += 32) {
      const int f = f0 + lane;
      const int e = f < hi ? local_expert(ids[f], first, E) : -1;
      const unsigned peers = __match_any_sync(0xffffffffu, e);
      const int r = __popc(peers & below);
      int pos = -1;
      if (e >= 0) pos = base[e] + cnt[warp * E + e] + r;
      __syncwarp();
      if (e >= 0 && r == 0) cnt[warp * E + e] += __popc(peers);
      __syncwarp();
      if (f < hi) {
        slot_of[f] = pos;
        if (pos >= 0) perm[pos] = f;
      }
    }
  }
  for (int p = valid + rank * kGroupThreads + tid; p < S; p += C * kGroupThreads) perm[p] = -1;
  cl.sync();                           // no CTA leaves while another reads its totals
}

cudaError_t launch_group(const int32_t* ids, int S, int E, int first, int32_t* offsets,
                         int32_t* perm, int32_t* slot_of, cudaStream_t st) {
  static PerDevice<int> per;
  int widest = 8;
  cudaError_t err = on_device(per, &widest, [](int* w) {
    cudaError_t e = cudaFuncSetAttribute(group_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)group_smem(kGroupWarps, kGroupMaxExperts));
    if (e != cudaSuccess) return e;
    *w = 8;
    // 16 CTAs are beyond the portable cluster size: used where the device can hold one
    if (cudaFuncSetAttribute(group_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess) {
      cudaLaunchConfig_t q = {};
      q.gridDim = dim3(16);
      q.blockDim = dim3(kGroupThreads);
      q.dynamicSmemBytes = group_smem(kGroupWarps, kGroupMaxExperts);
      cudaLaunchAttribute at;
      at.id = cudaLaunchAttributeClusterDimension;
      at.val.clusterDim.x = 16;
      at.val.clusterDim.y = at.val.clusterDim.z = 1;
      q.attrs = &at;
      q.numAttrs = 1;
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, group_kernel, &q) == cudaSuccess && n > 0) *w = 16;
    }
    (void)cudaGetLastError();
    return cudaSuccess;
  });
  if (err != cudaSuccess) return err;
  const GroupShape g = group_shape(S, widest);
  const size_t smem = group_smem(g.warps, E);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(g.ctas);
  cfg.blockDim = dim3(kGroupThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = g.ctas;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, group_kernel, ids, S, E, first, g.per_cta, g.per_warp, g.warps,
                            offsets, perm, slot_of);
}

}  // namespace moe
