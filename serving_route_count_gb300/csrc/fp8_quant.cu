// fp8_quant.cu - quantisation to e4m3 with fp32 scales (moe_fp8_quant): a scale for each 128 values of
// a row (activations), or for each 128 x 128 tile (weights).
//   scale = max(max |x| / 448, 2^-126),  code = e4m3(x / scale)
// Both quotients are correctly rounded: x / scale meets the middle of two codes for about one element in
// 250 (448 = 7 * 64, so elements of 3/4 of the largest one's mantissa do), where a product by a
// reciprocal, an ulp off, would go to the other side.  The largest may not be skipped by a NaN or be
// one: fmaxf takes the other value, so a NaN spoils its own code alone and an infinity its whole block
// (scale inf, codes 0 and NaN), and any product over either is NaN.
//
// Bound by HBM: x is read once and codes and scales written once.  Rows on 16 bytes go 16 values to a
// thread, whole vectors in and out, eight threads to a block of a row; a tile stays in its CTA's
// registers between the maximum and the codes.  us: 8192 x 7168 bf16 rows 31 (floor 26; with 64-bit indexes
// and one value at a time in the maximum 42), tiles of 24 x 2304 x 7168 193 (floor 176; two CTAs of them on an SM
// instead of four 261), one row of 7168 2.9.  Rows off 16 bytes: 82 and 646, a value at a time.
#include <cuda_fp8.h>

#include <type_traits>

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

// 16 consecutive values.
template <typename T>
struct Quant16 {
  static constexpr int kWords = 16 * sizeof(T) / 16;
  uint4 w[kWords];
  __device__ __forceinline__ void load(const T* x) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = __ldcs(reinterpret_cast<const uint4*>(x) + i);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = make_uint4(0, 0, 0, 0);
  }
  // 16-bit values two at a time; either maximum leaves NaN out
  __device__ __forceinline__ float top() const {
    if constexpr (sizeof(T) == 2) {
      using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
      T2 v[8];
      memcpy(v, w, sizeof(v));
      T2 m = __habs2(v[0]);
#pragma unroll
      for (int i = 1; i < 8; ++i) m = __hmax2(m, __habs2(v[i]));
      return fmaxf(fmaxf(to_f32(m.x), to_f32(m.y)), 0.f);
    } else {
      float v[16], m = 0.f;
      memcpy(v, w, sizeof(v));
#pragma unroll
      for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(v[i]));
      return m;
    }
  }
  // Codes by one reciprocal, with Markstein's correction: for r = 1 / s rounded to nearest and q near x / s, the
  // two fused operations of q + r (x - q s) give x / s rounded to nearest.  His theorem asks for a q within an ulp;
  // q = x r may be 1.5 off (half an ulp of its own rounding, up to one by r's).  What is needed here is less: only
  // quotients next to the middle of two codes decide a code, and for every mantissa of s, every middle and all x
  // within 3 ulps of their product the result is the IEEE quotient (4.7e9 cases, on the host).  The residual must
  // not underflow: scales of 2^-60 and more keep it above the least subnormal wherever the quotient does not round
  // to a zero code; smaller scales and infinite ones take the division.
  __device__ __forceinline__ uint4 codes(float scale) const {
    T v[16];
    memcpy(v, w, sizeof(v));
    uint16_t c[8];
    if (scale >= 8.67361738e-19f && scale <= 3.40282347e38f) {
      const float r = __frcp_rn(scale);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float2 q;
        const float a = to_f32(v[2 * i]), b = to_f32(v[2 * i + 1]);
        q.x = a * r;
        q.y = b * r;
        q.x = copysignf(fmaf(fmaf(-q.x, scale, a), r, q.x), a);      // the sum of zeros loses the sign
        q.y = copysignf(fmaf(fmaf(-q.y, scale, b), r, q.y), b);
        c[i] = __nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        c[i] = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(to_f32(v[2 * i]), scale), __fdiv_rn(to_f32(v[2 * i + 1]), scale)),
                                        __NV_SATFINITE, __NV_E4M3);
    }
    uint4 o;
    memcpy(&o, c, 16);
    return o;
  }
};

// Rows on 16 bytes: eight threads per block of 128 values, kQuantAhead blocks of each in flight.
constexpr int kQuantAhead = 2;
template <typename T>
__global__ void __launch_bounds__(256) quant_rows16_kernel(const QuantParams p) {
  const int sub = threadIdx.x & 7;
  pdl_wait_prev();
  pdl_launch_next();
  // blocks are counted in 32 bits: a division in 64 costs a quarter of the call
  const unsigned n = (unsigned)p.rows * (unsigned)p.KB, step = gridDim.x * 32;
  for (unsigned i0 = blockIdx.x * 32 + (threadIdx.x >> 3); i0 < n; i0 += kQuantAhead * step) {
    Quant16<T> v[kQuantAhead];
    int row[kQuantAhead], k[kQuantAhead];
#pragma unroll
    for (int u = 0; u < kQuantAhead; ++u) {
      const unsigned i = i0 + u * step, r = i / p.KB;
      row[u] = i < n ? (int)r : -1;
      k[u] = row[u] < 0 ? p.K : (int)(i - r * p.KB) * kFp8Block + 16 * sub;
      if (k[u] < p.K)
        v[u].load(static_cast<const T*>(p.x) + row[u] * p.ldx + k[u]);
      else
        v[u].zero();
    }
#pragma unroll
    for (int u = 0; u < kQuantAhead; ++u) {
      float top = v[u].top();
#pragma unroll
      for (int o = 4; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float scale = quant_scale(top);
      if (row[u] < 0) continue;
      if (sub == 0) p.scale[row[u] * p.lds + k[u] / kFp8Block] = scale;
      if (k[u] < p.K) *reinterpret_cast<uint4*>(p.q + row[u] * p.ldq + k[u]) = v[u].codes(scale);
    }
  }
}

// Tiles on 16 bytes: a CTA per tile, 16 values of four rows to a thread.
template <typename T>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 4 : 2) quant_tiles16_kernel(const QuantParams p, int tiles) {
  __shared__ float s_top[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tall = fp8_blocks(p.rows);       // of one matrix
  pdl_wait_prev();
  pdl_launch_next();
  for (unsigned t = blockIdx.x; t < (unsigned)tiles; t += gridDim.x) {
    const int b = t % p.KB, rb = t / p.KB;   // rb: tile row over all matrices
    const int e = rb / tall, r0 = (rb - e * tall) * kFp8Block, k = b * kFp8Block + 16 * (threadIdx.x & 7);
    const long long first = (long long)e * p.rows + r0;
    Quant16<T> v[4];
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = 32 * j + (threadIdx.x >> 3);
      if (k < p.K && r0 + r < p.rows)
        v[j].load(static_cast<const T*>(p.x) + (first + r) * p.ldx + k);
      else
        v[j].zero();
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) top = fmaxf(top, v[j].top());
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) s_top[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) top = fmaxf(top, s_top[w]);
    const float scale = quant_scale(top);
    if (threadIdx.x == 0) p.scale[(long long)rb * p.lds + b] = scale;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = 32 * j + (threadIdx.x >> 3);
      if (k < p.K && r0 + r < p.rows) *reinterpret_cast<uint4*>(p.q + (first + r) * p.ldq + k) = v[j].codes(scale);
    }
    __syncthreads();                         // s_top read by all
  }
}

// Rows of any alignment: a warp per block of 128 values.
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

// Tiles of any alignment: a CTA per tile, which is read twice.
template <typename T>
__global__ void __launch_bounds__(256) quant_tiles_kernel(const QuantParams p, int tiles) {
  __shared__ float s_top[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tall = fp8_blocks(p.rows);       // of one matrix
  pdl_wait_prev();
  pdl_launch_next();
  for (unsigned t = blockIdx.x; t < (unsigned)tiles; t += gridDim.x) {
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
  // whole vectors of 16 values: K and row strides of them, bases on 16 bytes
  bool vec = p.K % 16 == 0 && p.ldq % 16 == 0 && p.ldx * (long long)sizeof(T) % 16 == 0 &&
                   (reinterpret_cast<uintptr_t>(p.x) & 15) == 0 && (reinterpret_cast<uintptr_t>(p.q) & 15) == 0;
  if (tiles) {
    const long long n = (long long)E * fp8_blocks(p.rows) * p.KB;
    return launch_kernel(vec ? quant_tiles16_kernel<T> : quant_tiles_kernel<T>, dim3((unsigned)(n < (1 << 20) ? n : 1 << 20)),
                         dim3(256), 0, st, true, p, (int)n);
  }
  const long long blocks = (long long)p.rows * p.KB;
  vec = vec && blocks < (1LL << 31);         // counted in 32 bits, a grid's step past the end too
  const long long n = vec ? (blocks + 32 * kQuantAhead - 1) / (32 * kQuantAhead) : (blocks + 7) / 8;
  return launch_kernel(vec ? quant_rows16_kernel<T> : quant_rows_kernel<T>, dim3((unsigned)(n < (1 << 20) ? n : 1 << 20)), dim3(256),
                       0, st, true, p);
}

cudaError_t launch_fp8_quant(const void* x, int dtype, long long ldx, int E, int rows, int K, bool tiles,
                             uint8_t* q, long long ldq, float* scale, long long lds, cudaStream_t st) {
  const QuantParams p{x, ldx, rows, K, fp8_blocks(K), q, ldq, scale, lds};
  if (dtype == MOE_DTYPE_F16) return launch_quant<__half>(p, E, tiles, st);
  if (dtype == MOE_DTYPE_BF16) return launch_quant<__nv_bfloat16>(p, E, tiles, st);
  return launch_quant<float>(p, E, tiles, st);
}

}  // namespace moe
