// block_ops.cuh - what the kernels of the 16-bit block share: element types, vector accesses,
// block reductions.
#pragma once

#include "block_launch.cuh"
#include "moe_common.cuh"

namespace moe {

// PerDevice's value of the current device; init as there, with CUDA's error codes.
template <typename V, typename Init>
cudaError_t on_device(PerDevice<V>& per, V* out, Init init) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  return e != cudaSuccess ? e : static_cast<cudaError_t>(per.get(dev, out, init));
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) {
  return __float2half_rn(v);
}
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// Clamped SwiGLU in fp32: g' * sigmoid(alpha g') * (u' + beta), g' = min(g, limit),
// u' = clamp(u, -limit, limit).  sigmoid(a) = 1 / (1 + e) or e / (1 + e), e = exp(-|a|): the divisor
// stays within [1, 2], where __fdividef is within 2 ulp (above 2^126 it returns 0, which lost every
// gate of a in -88.7 .. -87.3, values that bf16 can hold).  With __expf (2 + 1.2 |a| ulp) that is far
// below the rounding of the 16-bit result; with expf and an IEEE division the product's epilogue
// took 9 % of a tensor-bound call.
__device__ __forceinline__ float swiglu_f32(float u, float g, float limit, float alpha,
                                            float beta) {
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(g) : "f"(limit));      // NaN stays NaN
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(u) : "f"(limit));
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(u) : "f"(-limit));
  const float a = alpha * g, e = __expf(-fabsf(a));
  return __fdividef(a < 0.f ? g * e : g, 1.0f + e) * (u + beta);
}

}  // namespace moe
