// gemm_ff_simt.cu - products of the gated feed-forward block on the CUDA cores, for operands whose rows
// do not start on 16-byte boundaries, as the tensor-core kernel's tile copies need.  Such operands are
// taken, and not meant to be fast.
//
// One CTA of 256 threads per tile of 64 x 64 outputs; a thread owns 4 x 4 sums in fp32 (two sets for
// the gated product).  Operands pass through shared memory 16 K at a time, read along whichever of
// their dimensions is contiguous.
#include "feed_forward.cuh"
#include "../../include/moe_gb300.h"

namespace moe {

constexpr int kFfsK = 16, kFfsThreads = 256;

struct FfsParams {
  FfDims d;
  FfGemm g;
};

template <typename T, int EPI>
__global__ void __launch_bounds__(kFfsThreads)
ff_simt_kernel(const FfsParams p) {
  constexpr int kSets = EPI == kFfGlu ? 2 : 1;
  __shared__ float sc[kFfsK][kGsTile + 4];
  __shared__ float sr[kSets][kFfsK][kGsTile + 4];
  const FfGemm& g = p.g;
  const int tid = threadIdx.x, tr = tid / 16, tc = tid % 16;   // 4 rows of C x 4 of R of this thread
  pdl_wait_prev();
  pdl_launch_next();
  const T* R = static_cast<const T*>(g.r);
  const T* C = static_cast<const T*>(g.c);
  T* out = static_cast<T*>(g.out);
  const int c0 = blockIdx.x * kGsTile;
  for (int r0 = blockIdx.y * kGsTile; r0 < g.nr; r0 += gridDim.y * kGsTile) {
    float acc[kSets][4][4] = {};
    for (int k0 = 0; k0 < g.K; k0 += kFfsK) {
      for (int i = tid; i < kGsTile * kFfsK; i += kFfsThreads) {
        {
          const int j = g.ck == 1 ? i / kFfsK : i % kGsTile, k = g.ck == 1 ? i % kFfsK : i / kGsTile;
          sc[k][j] = k0 + k < g.K && c0 + j < g.nc ? to_f32(C[(c0 + j) * g.cs + (k0 + k) * g.ck]) : 0.f;
        }
        const int j = g.rk == 1 ? i / kFfsK : i % kGsTile, k = g.rk == 1 ? i % kFfsK : i / kGsTile;
#pragma unroll
        for (int h = 0; h < kSets; ++h)
          sr[h][k][j] = k0 + k < g.K && r0 + j < g.nr
                            ? to_f32(R[(r0 + j) * g.rs + (k0 + k) * g.rk + h * g.half]) : 0.f;
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kFfsK; ++k) {
        const float4 a = *reinterpret_cast<const float4*>(&sc[k][4 * tr]);
        const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int h = 0; h < kSets; ++h) {
          const float4 b = *reinterpret_cast<const float4*>(&sr[h][k][4 * tc]);
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
        const int c = c0 + 4 * tr + i, r = r0 + 4 * tc + j;
        if (c >= g.nc || r >= g.nr) continue;
        T* o = out + c * g.ldo + r;
        float* s = EPI == kFfStore ? nullptr : g.pre + (long long)c * 2 * g.nr + r;
        const bool up_first = p.d.layout == MOE_W13_UP_GATE;
        if constexpr (EPI == kFfStore) {
          *o = from_f32<T>(acc[0][i][j]);
        } else if constexpr (EPI == kFfGlu) {
          const float u = acc[up_first ? 0 : kSets - 1][i][j], gt = acc[up_first ? kSets - 1 : 0][i][j];
          *o = from_f32<T>(swiglu_f32(u, gt, p.d.limit, p.d.alpha, p.d.beta));
          if (g.pre != nullptr) {
            s[up_first ? 0 : g.nr] = u;
            s[up_first ? g.nr : 0] = gt;
          }
        } else {
          float du, dg;
          swiglu_grad(s[up_first ? 0 : g.nr], s[up_first ? g.nr : 0], acc[0][i][j], p.d.limit,
                      p.d.alpha, p.d.beta, &du, &dg);
          o[up_first ? 0 : g.nr] = from_f32<T>(du);
          o[up_first ? g.nr : 0] = from_f32<T>(dg);
        }
      }
  }
}

cudaError_t launch_ff_simt(const FfDims& d, const FfGemm& g, int epilogue, cudaStream_t st) {
  const FfsParams p{d, g};
  const dim3 grid(cdiv(g.nc, kGsTile), (unsigned)std::min(cdiv(g.nr, kGsTile), 65535));
  const auto go = [&](auto kernel) { return launch_kernel(kernel, grid, dim3(kFfsThreads), 0, st, true, p); };
  const bool h = d.dtype == MOE_DTYPE_F16;
  if (epilogue == kFfGlu) return h ? go(ff_simt_kernel<__half, kFfGlu>) : go(ff_simt_kernel<__nv_bfloat16, kFfGlu>);
  if (epilogue == kFfGrad) return h ? go(ff_simt_kernel<__half, kFfGrad>) : go(ff_simt_kernel<__nv_bfloat16, kFfGrad>);
  return h ? go(ff_simt_kernel<__half, kFfStore>) : go(ff_simt_kernel<__nv_bfloat16, kFfStore>);
}

}  // namespace moe
