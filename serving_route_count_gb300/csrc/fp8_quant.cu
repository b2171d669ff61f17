// fp8_quant.cu - quantisation to e4m3 with fp32 scales (moe_fp8_quant): a scale for each 128 values of
// a row (activations), or for each 128 x 128 tile (weights).
//   scale = max(max |x| / 448, 2^-126),  code = e4m3(x / scale)
// Both quotients are IEEE divisions: x / scale meets the middle of two codes for about one element in
// 250 (448 = 7 * 64, so elements of 3/4 of the largest one's mantissa do), where a product by a
// reciprocal, an ulp off, would go to the other side.  The largest may not be skipped by a NaN or be
// one: fmaxf takes the other value, so a NaN spoils its own code alone and an infinity its whole block
// (scale inf, codes 0 and NaN), and any product over either is NaN.
#include <cuda_fp8.h>

#include "block_ops.cuh"
#include "fp8.cuh"
#include "../../include/moe_gb300.h"

namespace moe {

struct QuantParams {
  const void* x;
  long long ldx;
  int rows, K, KB;
  uint8_t* q;
  long long ldq;
  float* scale;
  long long lds;            // scales of a row (rows), of a tile row (tiles)
};

__device__ __forceinline__ float quant_scale(float top) {
  return fmaxf(__fdiv_rn(top, kFp8Max), 1.17549435e-38f);
}
__device__ __forceinline__ uint8_t quant_code(float v, float scale) {
  return (uint8_t)__nv_cvt_float_to_fp8(__fdiv_rn(v, scale), __NV_SATFINITE, __NV_E4M3);
}

// Rows: a warp per block of 128 values.
template <typename T>
__global__ void __launch_bounds__(256) quant_rows_kernel(const QuantParams p) {
  const int lane = threadIdx.x & 31;
  pdl_wait_prev();
  pdl_launch_next();
  const long long n = (long long)p.rows * p.KB;
  for (long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); i < n; i += (long long)gridDim.x * 8) {
    const long long r = i / p.KB;
    const int b = (int)(i - r * p.KB), k0 = b * kFp8Block;
    const T* x = static_cast<const T*>(p.x) + r * p.ldx;
    float v[4], top = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = k0 + lane + 32 * j;
      v[j] = k < p.K ? to_f32(x[k]) : 0.f;
      top = fmaxf(top, fabsf(v[j]));
    }
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float scale = quant_scale(top);
    if (lane == 0) p.scale[r * p.lds + b] = scale;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = k0 + lane + 32 * j;
      if (k < p.K) p.q[r * p.ldq + k] = quant_code(v[j], scale);
    }
  }
}

// Tiles: a CTA per tile of 128 rows x 128 values.
template <typename T>
__global__ void __launch_bounds__(256) quant_tiles_kernel(const QuantParams p, int tiles) {
  __shared__ float s_top[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tall = fp8_blocks(p.rows);       // of one matrix
  pdl_wait_prev();
  pdl_launch_next();
  for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int b = t % p.KB, rb = t / p.KB;   // rb: tile row over all matrices
    const int e = rb / tall, r0 = (rb - e * tall) * kFp8Block, k0 = b * kFp8Block;
    const int n = min(kFp8Block, p.rows - r0);
    const long long first = (long long)e * p.rows + r0;
    float top = 0.f;
    for (int r = warp; r < n; r += 8)
      for (int k = k0 + lane; k < min(p.K, k0 + kFp8Block); k += 32)
        top = fmaxf(top, fabsf(to_f32(static_cast<const T*>(p.x)[(first + r) * p.ldx + k])));
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) s_top[warp] = top;
    __syncthreads();
    for (int w = 0; w < 8; ++w) top = fmaxf(top, s_top[w]);
    const float scale = quant_scale(top);
    if (threadIdx.x == 0) p.scale[(long long)rb * p.lds + b] = scale;
    for (int r = warp; r < n; r += 8)
      for (int k = k0 + lane; k < min(p.K, k0 + kFp8Block); k += 32)
        p.q[(first + r) * p.ldq + k] = quant_code(to_f32(static_cast<const T*>(p.x)[(first + r) * p.ldx + k]), scale);
    __syncthreads();
  }
}

template <typename T>
static cudaError_t launch_quant(const QuantParams& p, int E, bool tiles, cudaStream_t st) {
  if (tiles) {
    const long long n = (long long)E * fp8_blocks(p.rows) * p.KB;
    return launch_kernel(quant_tiles_kernel<T>, dim3((unsigned)(n < (1 << 20) ? n : 1 << 20)), dim3(256), 0, st, true, p, (int)n);
  }
  const long long n = ((long long)p.rows * p.KB + 7) / 8;
  return launch_kernel(quant_rows_kernel<T>, dim3((unsigned)(n < 152 * 64 ? n : 152 * 64)), dim3(256), 0, st, true, p);
}

cudaError_t launch_fp8_quant(const void* x, int dtype, long long ldx, int E, int rows, int K, bool tiles,
                             uint8_t* q, long long ldq, float* scale, long long lds, cudaStream_t st) {
  const QuantParams p{x, ldx, rows, K, fp8_blocks(K), q, ldq, scale, lds};
  if (dtype == MOE_DTYPE_F16) return launch_quant<__half>(p, E, tiles, st);
  if (dtype == MOE_DTYPE_BF16) return launch_quant<__nv_bfloat16>(p, E, tiles, st);
  return launch_quant<float>(p, E, tiles, st);
}

}  // namespace moe
