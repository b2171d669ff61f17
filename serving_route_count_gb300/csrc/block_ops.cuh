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

// SMs of the current device.
inline cudaError_t device_sms(int* sms) {
  static PerDevice<int> per;
  return on_device(per, sms, [](int* v) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    return e != cudaSuccess ? e : cudaDeviceGetAttribute(v, cudaDevAttrMultiProcessorCount, dev);
  });
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

// Four times 16 bytes that are read once, `step` bytes apart, the first n of them; zeros for the others.  One
// statement, so that all four are under way before the first is used (apart, the compiler uses each in turn
// and saves the registers).
__device__ __forceinline__ void load_once16x4(uint4 (&v)[4], const void* p, long long step, int n) {
  const char* q = static_cast<const char*>(p);
  asm volatile(
      "{\n .reg .pred p0, p1, p2, p3;\n"
      " setp.gt.s32 p0, %20, 0;\n setp.gt.s32 p1, %20, 1;\n setp.gt.s32 p2, %20, 2;\n setp.gt.s32 p3, %20, 3;\n"
      " mov.u32 %0, 0;\n mov.u32 %1, 0;\n mov.u32 %2, 0;\n mov.u32 %3, 0;\n"
      " mov.u32 %4, 0;\n mov.u32 %5, 0;\n mov.u32 %6, 0;\n mov.u32 %7, 0;\n"
      " mov.u32 %8, 0;\n mov.u32 %9, 0;\n mov.u32 %10, 0;\n mov.u32 %11, 0;\n"
      " mov.u32 %12, 0;\n mov.u32 %13, 0;\n mov.u32 %14, 0;\n mov.u32 %15, 0;\n"
      " @p0 ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%16];\n"
      " @p1 ld.global.L1::no_allocate.v4.u32 {%4, %5, %6, %7}, [%17];\n"
      " @p2 ld.global.L1::no_allocate.v4.u32 {%8, %9, %10, %11}, [%18];\n"
      " @p3 ld.global.L1::no_allocate.v4.u32 {%12, %13, %14, %15}, [%19];\n}"
      : "=&r"(v[0].x), "=&r"(v[0].y), "=&r"(v[0].z), "=&r"(v[0].w), "=&r"(v[1].x), "=&r"(v[1].y),
        "=&r"(v[1].z), "=&r"(v[1].w), "=&r"(v[2].x), "=&r"(v[2].y), "=&r"(v[2].z), "=&r"(v[2].w),
        "=&r"(v[3].x), "=&r"(v[3].y), "=&r"(v[3].z), "=&r"(v[3].w)
      : "l"(q), "l"(q + step), "l"(q + 2 * step), "l"(q + 3 * step), "r"(n)
      : "memory");
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
