// gemm_fp8_simt.cu - 8-bit products with block scales on the CUDA cores, for operands whose rows do not
// start on 16-byte boundaries, as the tensor-core kernel's tile copies need.  Such operands are taken,
// and not meant to be fast.
//
// One CTA of 256 threads per tile of 64 positions of one expert x 64 output columns; a thread owns 4 x 4
// sums in fp32 (two sets for a SwiGLU: up and gate).  Operands pass through shared memory 16 K at a
// time, as the values they stand for (code * scale, rounded to fp32 once).
#include <cuda_fp8.h>

#include "block_ops.cuh"
#include "fp8.cuh"
#include "../../include/moe_gb300.h"

namespace moe {

constexpr int kFsK = 16, kFsThreads = 256;

struct FsParams {
  GroupedDims d;
  Fp8Call f;
  int cols;
};

__device__ __forceinline__ float e4m3_f32(uint8_t code) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(code, __NV_E4M3)));
}

template <typename T, bool ACT>
__global__ void __launch_bounds__(kFsThreads)
fp8_simt_kernel(const FsParams p) {
  __shared__ float sx[kFsK][kGsTile + 4];
  __shared__ float sw[ACT ? 2 : 1][kFsK][kGsTile + 4];
  __shared__ int s_tile[4];            // expert, first position, positions, end of the last group
  __shared__ long long s_row[kGsTile];
  const GroupedCall& c = p.f.c;
  const int tid = threadIdx.x, E = p.d.E, S = c.S;
  pdl_wait_prev();
  pdl_launch_next();
  if (tid < 32) {
    // lane l owns experts [l * per, (l + 1) * per): a warp scan of their tile counts
    const auto first = [&](int e) { return c.offsets ? c.offsets[e] : 0; };
    const auto last = [&](int e) { return c.offsets ? c.offsets[e + 1] : S; };
    const int per = cdiv(E, 32), e0 = min(E, tid * per), e1 = min(E, e0 + per);
    int tiles = 0;
    for (int e = e0; e < e1; ++e) {
      const int a = first(e), b = last(e);
      if (a < 0 || b < a || b > S)
        set_error(c.err, kErrRouteBounds);
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
        const int a = first(e), b = last(e);
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
    if (tid == 0) s_tile[3] = max(0, min(S, last(E - 1)));
  }
  __syncthreads();
  T* out = static_cast<T*>(c.out);
  const int c_first = blockIdx.y * kGsTile, c_step = gridDim.y * kGsTile;
  // rows past the last group: this CTA's share of them
  for (int c0 = c_first; c0 < p.cols; c0 += c_step)
    for (int i = tid; i < kGsTile * kGsTile; i += kFsThreads) {
      const long long r = (long long)s_tile[3] + (long long)blockIdx.x * kGsTile + i / kGsTile;
      const int col = c0 + i % kGsTile;
      if (r < S && col < p.cols) out[r * c.ldo + col] = from_f32<T>(0.f);
    }
  const int e = s_tile[0];
  if (e < 0) return;
  const int p0 = s_tile[1], n = s_tile[2];
  if (tid < kGsTile) {
    long long row = p0 + min(tid, n - 1);
    if (c.perm != nullptr) {
      const int f = c.perm[row];
      row = f < 0 ? -1 : f / c.topk;
      if (row < 0 || row >= c.x_rows) {
        set_error(c.err, kErrRouteBounds);
        row = 0;
      }
    }
    s_row[tid] = row;
  }
  __syncthreads();
  const int K = p.d.K, half = p.d.N / 2, KB = fp8_blocks(K);
  const uint8_t* x = static_cast<const uint8_t*>(c.x);
  const uint8_t* w = static_cast<const uint8_t*>(c.w) + (size_t)e * p.d.N * c.ldw;
  const float* ws = p.f.ws + (size_t)e * fp8_tall(p.d) * KB;
  const int tr = tid / 16, tc = tid % 16;       // 4 positions x 4 columns of this thread
  for (int c0 = c_first; c0 < p.cols; c0 += c_step) {
    float acc[ACT ? 2 : 1][4][4] = {};
    for (int k0 = 0; k0 < K; k0 += kFsK) {
      const int b = k0 / kFp8Block;             // kFsK divides a block
      for (int i = tid; i < kGsTile * kFsK; i += kFsThreads) {
        const int r = i / kFsK, k = i % kFsK;
        sx[k][r] = k0 + k < K ? e4m3_f32(x[s_row[r] * c.ldx + k0 + k]) * p.f.xs[s_row[r] * p.f.ldxs + b] : 0.f;
#pragma unroll
        for (int h = 0; h < (ACT ? 2 : 1); ++h) {
          const int wr = c0 + r + h * half;
          sw[h][k][r] = (k0 + k < K && c0 + r < p.cols)
                            ? e4m3_f32(w[(size_t)wr * c.ldw + k0 + k]) * ws[(size_t)fp8_scale_row(p.d, wr) * KB + b] : 0.f;
        }
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kFsK; ++k) {
        const float4 a = *reinterpret_cast<const float4*>(&sx[k][4 * tr]);
        const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int h = 0; h < (ACT ? 2 : 1); ++h) {
          const float4 v = *reinterpret_cast<const float4*>(&sw[h][k][4 * tc]);
          const float bv[4] = {v.x, v.y, v.z, v.w};
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
        out[(long long)(p0 + r) * c.ldo + col] = from_f32<T>(v);
      }
  }
}

cudaError_t launch_fp8_simt(const GroupedDims& d, const Fp8Call& f, cudaStream_t st) {
  FsParams p{d, f, grouped_cols(d)};
  const GsGrid g = grouped_simt_grid(f.c.S, d.E, p.cols);
  auto go = [&](auto kernel) {
    return launch_kernel(kernel, dim3(g.x, g.y), dim3(kFsThreads), 0, st, true, p);
  };
  if (d.dtype == MOE_DTYPE_F16)
    return d.act ? go(fp8_simt_kernel<__half, true>) : go(fp8_simt_kernel<__half, false>);
  return d.act ? go(fp8_simt_kernel<__nv_bfloat16, true>) : go(fp8_simt_kernel<__nv_bfloat16, false>);
}

}  // namespace moe
