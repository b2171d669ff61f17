// gemm_grouped_simt.cu - products grouped by expert on the CUDA cores, for operands whose rows do not
// start on 16-byte boundaries, as the tensor-core kernel's tile copies need.  Such operands are taken,
// and not meant to be fast.
//
// One CTA of 256 threads per tile of 64 positions of one expert x 64 output columns; a thread
// owns 4 x 4 sums in fp32 (two sets for a SwiGLU: up and gate), operands pass through shared
// memory 16 K at a time.  Bound by the fp32 FMA rate and the scalar operand loads: fc1 + SwiGLU of
// 2048 tokens top-8 (E = 256, K = 6144, N = 1024) takes 9.9 ms here, 0.5 ms on the tensor cores.
#include "block_ops.cuh"
#include "grouped.cuh"
#include "../../include/moe_gb300.h"

namespace moe {

constexpr int kGsK = 16, kGsThreads = 256;

struct GsParams {
  GroupedDims d;
  GroupedCall c;
  int cols;
};

template <typename T, bool ACT>
__global__ void __launch_bounds__(kGsThreads)
grouped_simt_kernel(const GsParams p) {
  __shared__ float sx[kGsK][kGsTile + 4];
  __shared__ float sw[ACT ? 2 : 1][kGsK][kGsTile + 4];
  __shared__ int s_tile[4];            // expert, first position, positions, end of the last group
  __shared__ long long s_row[kGsTile];
  const int tid = threadIdx.x, E = p.d.E, S = p.c.S;
  pdl_wait_prev();
  pdl_launch_next();
  if (tid < 32) {
    // lane l owns experts [l * per, (l + 1) * per): a warp scan of their tile counts
    const int per = cdiv(E, 32), e0 = min(E, tid * per), e1 = min(E, e0 + per);
    int tiles = 0;
    for (int e = e0; e < e1; ++e) {
      const int a = p.c.offsets[e], b = p.c.offsets[e + 1];
      if (a < 0 || b < a || b > S)
        set_error(p.c.err, kErrRouteBounds);
      else
        tiles += cdiv(b - a, kGsTile);
    }
    int incl = tiles;
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (tid >= o) incl += y;
    }
    if (tid == 0) s_tile[0] = -1;
    __syncwarp();
    int t = (int)blockIdx.x - (incl - tiles);
    if (t >= 0 && t < tiles) {
      for (int e = e0; e < e1; ++e) {
        const int a = p.c.offsets[e], b = p.c.offsets[e + 1];
        if (a < 0 || b < a || b > S) continue;
        const int n = cdiv(b - a, kGsTile);
        if (t < n) {
          s_tile[0] = e;
          s_tile[1] = a + t * kGsTile;
          s_tile[2] = min(kGsTile, b - s_tile[1]);
          break;
        }
        t -= n;
      }
    }
    if (tid == 0) s_tile[3] = max(0, min(S, p.c.offsets[E]));
  }
  __syncthreads();
  T* out = static_cast<T*>(p.c.out);
  const int c_first = blockIdx.y * kGsTile, c_step = gridDim.y * kGsTile;
  // rows past the last group: this CTA's share of them
  for (int c0 = c_first; c0 < p.cols; c0 += c_step)
    for (int i = tid; i < kGsTile * kGsTile; i += kGsThreads) {
      const long long r = (long long)s_tile[3] + (long long)blockIdx.x * kGsTile + i / kGsTile;
      const int col = c0 + i % kGsTile;
      if (r < S && col < p.cols) out[r * p.c.ldo + col] = from_f32<T>(0.f);
    }
  const int e = s_tile[0];
  if (e < 0) return;
  const int p0 = s_tile[1], n = s_tile[2];
  if (tid < kGsTile) {
    long long row = p0 + min(tid, n - 1);
    if (p.c.perm != nullptr) {
      const int f = p.c.perm[row];
      row = f < 0 ? -1 : f / p.c.topk;
      if (row < 0 || row >= p.c.x_rows) {
        set_error(p.c.err, kErrRouteBounds);
        row = 0;
      }
    }
    s_row[tid] = row;
  }
  __syncthreads();
  const int K = p.d.K, half = p.d.N / 2;
  const T* x = static_cast<const T*>(p.c.x);
  const T* w = static_cast<const T*>(p.c.w) + (size_t)e * p.d.N * p.c.ldw;
  const int tr = tid / 16, tc = tid % 16;       // 4 positions x 4 columns of this thread
  for (int c0 = c_first; c0 < p.cols; c0 += c_step) {
    float acc[ACT ? 2 : 1][4][4] = {};
    for (int k0 = 0; k0 < K; k0 += kGsK) {
      for (int i = tid; i < kGsTile * kGsK; i += kGsThreads) {
        const int r = i / kGsK, k = i % kGsK;
        sx[k][r] = k0 + k < K ? to_f32(x[s_row[r] * p.c.ldx + k0 + k]) : 0.f;
#pragma unroll
        for (int h = 0; h < (ACT ? 2 : 1); ++h)
          sw[h][k][r] = (k0 + k < K && c0 + r < p.cols)
                            ? to_f32(w[(size_t)(c0 + r + h * half) * p.c.ldw + k0 + k]) : 0.f;
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kGsK; ++k) {
        const float4 a = *reinterpret_cast<const float4*>(&sx[k][4 * tr]);
        const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int h = 0; h < (ACT ? 2 : 1); ++h) {
          const float4 b = *reinterpret_cast<const float4*>(&sw[h][k][4 * tc]);
          const float bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[h][i][j] = fmaf(av[i], bv[j], acc[h][i][j]);
        }
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = 4 * tr + i, col = c0 + 4 * tc + j;
        if (r >= n || col >= p.cols) continue;
        float v = acc[0][i][j];
        if constexpr (ACT) {
          const float u = p.d.layout == MOE_W13_UP_GATE ? acc[0][i][j] : acc[1][i][j];
          const float g = p.d.layout == MOE_W13_UP_GATE ? acc[1][i][j] : acc[0][i][j];
          v = swiglu_f32(u, g, p.d.limit, p.d.alpha, p.d.beta);
        }
        out[(size_t)(p0 + r) * p.c.ldo + col] = from_f32<T>(v);
      }
  }
}

cudaError_t launch_grouped_simt(const GroupedDims& d, const GroupedCall& c, cudaStream_t st) {
  GsParams p{d, c, grouped_cols(d)};
  const GsGrid g = grouped_simt_grid(c.S, d.E, p.cols);
  auto go = [&](auto kernel) {
    return launch_kernel(kernel, dim3(g.x, g.y), dim3(kGsThreads), 0, st, true, p);
  };
  if (d.dtype == MOE_DTYPE_F16)
    return d.act ? go(grouped_simt_kernel<__half, true>) : go(grouped_simt_kernel<__half, false>);
  return d.act ? go(grouped_simt_kernel<__nv_bfloat16, true>)
               : go(grouped_simt_kernel<__nv_bfloat16, false>);
}

}  // namespace moe
