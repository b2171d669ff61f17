// block_norm.cu - norms before and after a block fused with the experts' top-k combine, the
// block's gate and the residual scale (moe_block_norm).
//
// One CTA per token; a thread keeps NCH chunks of 8 consecutive channels in fp32 registers from
// the loads to the stores, so every input is read once and every output written once, and a norm
// is one block-wide sum (two for the layer norm: the mean first, then the squares around it).
#include "block_ops.cuh"
#include "../../include/moe_gb300.h"

namespace moe {

struct NormParams {
  int M, H, kind, wide;             // wide: weights, biases and gate are fp32
  float eps, scale, woff;
  const void *residual, *rows;
  long long ld_res, ld_rows;
  const int32_t* slot_of;
  const float* topk_w;
  int topk, n_rows;
  const void* shared;
  long long ld_shared;
  const void *post_w, *post_b, *gate;
  long long gate_row, gate_col;
  const void *pre_w, *pre_b;
  void *res_out, *out;
  long long ld_res_out, ld_out;
};

// Eight elements of a row from element h on; VEC: 16-byte aligned and whole, else element by
// element up to H.
template <bool VEC, typename T>
__device__ __forceinline__ void load8(const T* __restrict__ row, int h, int H, float* v) {
  if constexpr (VEC && sizeof(T) == 2) {
    const uint4 u = *reinterpret_cast<const uint4*>(row + h);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      T p[2];
      memcpy(p, &w[i], 4);
      v[2 * i] = to_f32(p[0]);
      v[2 * i + 1] = to_f32(p[1]);
    }
  } else if constexpr (VEC) {
    const float4 a = *reinterpret_cast<const float4*>(row + h);
    const float4 b = *reinterpret_cast<const float4*>(row + h + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = h + i < H ? to_f32(row[h + i]) : 0.f;
  }
}
template <bool VEC, typename T>
__device__ __forceinline__ void store8(T* __restrict__ row, int h, int H, const float* v) {
  if constexpr (VEC && sizeof(T) == 2) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const T p[2] = {from_f32<T>(v[2 * i]), from_f32<T>(v[2 * i + 1])};
      memcpy(&w[i], p, 4);
    }
    *reinterpret_cast<uint4*>(row + h) = make_uint4(w[0], w[1], w[2], w[3]);
  } else if constexpr (VEC) {
    *reinterpret_cast<float4*>(row + h) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(row + h + 4) = make_float4(v[4], v[5], v[6], v[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (h + i < H) row[h + i] = from_f32<T>(v[i]);
  }
}
// Eight weights of type T or fp32.
template <bool VEC, typename T>
__device__ __forceinline__ void load8w(const void* w, int wide, int h, int H, float* v) {
  if (wide)
    load8<VEC>(static_cast<const float*>(w), h, H, v);
  else
    load8<VEC>(static_cast<const T*>(w), h, H, v);
}

// Sum over the CTA, the same value in every thread.  s: 33 words, free for the next call after
// the second barrier of the next sum (two buffers alternate).
__device__ __forceinline__ float block_sum(float v, float* s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = (blockDim.x + 31) >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane == 0) s[warp] = v;
  __syncthreads();
  v = lane < warps ? s[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// v = norm(v) * (w + woff) + b over the row's H channels.  s: two buffers of 32 words.
template <typename T, bool VEC, int NCH>
__device__ __forceinline__ void norm_row(float (&v)[NCH][8], const NormParams& p, const void* w,
                                         const void* b, float (*s)[32]) {
  const int T0 = blockDim.x;
  const float inv_h = 1.f / (float)p.H;
  float sum = 0.f;
  if (p.kind == MOE_NORM_LAYER) {
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += v[c][i];
    const float mean = block_sum(sum, s[1]) * inv_h;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int h = (c * T0 + threadIdx.x) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = h + i < p.H ? v[c][i] - mean : 0.f;
    }
    sum = 0.f;
  }
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += v[c][i] * v[c][i];
  const float inv = 1.f / sqrtf(block_sum(sum, s[0]) * inv_h + p.eps);
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int h = (c * T0 + threadIdx.x) * 8;
    if (h >= p.H) break;
    float g[8];
    load8w<VEC, T>(w, p.wide, h, p.H, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[c][i] *= inv * (g[i] + p.woff);
    if (b != nullptr) {
      load8w<VEC, T>(b, p.wide, h, p.H, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] += g[i];
    }
  }
}

template <typename T, typename R, bool VEC, int NCH>
__global__ void __launch_bounds__(1024)
block_norm_kernel(const NormParams p) {
  __shared__ float s_sum[4][32];
  const int t = blockIdx.x, T0 = blockDim.x, tid = threadIdx.x;
  pdl_wait_prev();
  pdl_launch_next();
  float v[NCH][8];
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) v[c][i] = 0.f;

  const bool block = p.rows != nullptr;
  if (block) {
    const T* rows = static_cast<const T*>(p.rows);
    if (p.slot_of == nullptr) {
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const int h = (c * T0 + tid) * 8;
        if (h < p.H) load8<VEC>(rows + (size_t)t * p.ld_rows, h, p.H, v[c]);
      }
    } else {
      for (int j = 0; j < p.topk; ++j) {
        const int slot = p.slot_of[(size_t)t * p.topk + j];
        if (slot < 0 || slot >= p.n_rows) continue;
        const float w = p.topk_w[(size_t)t * p.topk + j];
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
          const int h = (c * T0 + tid) * 8;
          if (h >= p.H) break;
          float y[8];
          load8<VEC>(rows + (size_t)slot * p.ld_rows, h, p.H, y);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[c][i] = fmaf(w, y[i], v[c][i]);
        }
      }
      if (p.shared != nullptr) {
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
          const int h = (c * T0 + tid) * 8;
          if (h >= p.H) break;
          float y[8];
          load8<VEC>(static_cast<const T*>(p.shared) + (size_t)t * p.ld_shared, h, p.H, y);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[c][i] += y[i];
        }
      }
    }
    if (p.post_w != nullptr) norm_row<T, VEC, NCH>(v, p, p.post_w, p.post_b, s_sum);
  }
  const R* res = static_cast<const R*>(p.residual) + (size_t)t * p.ld_res;
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int h = (c * T0 + tid) * 8;
    if (h >= p.H) break;
    float r[8];
    load8<VEC>(res, h, p.H, r);
    if (block) {
      float g[8];
      if (p.gate == nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = p.scale;
      } else if (p.gate_col != 0) {
        const size_t o = (size_t)t * p.gate_row;
        if (p.wide)
          load8<VEC>(static_cast<const float*>(p.gate) + o, h, p.H, g);
        else
          load8<VEC>(static_cast<const T*>(p.gate) + o, h, p.H, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] *= p.scale;
      } else {
        const size_t o = (size_t)t * p.gate_row;
        const float s = p.scale * (p.wide ? static_cast<const float*>(p.gate)[o]
                                          : to_f32(static_cast<const T*>(p.gate)[o]));
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = s;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = h + i < p.H ? fmaf(g[i], v[c][i], r[i]) : 0.f;
      if (p.res_out != nullptr)
        store8<VEC>(static_cast<R*>(p.res_out) + (size_t)t * p.ld_res_out, h, p.H, v[c]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = r[i];
    }
  }
  if (p.pre_w == nullptr) return;
  norm_row<T, VEC, NCH>(v, p, p.pre_w, p.pre_b, s_sum + 2);
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int h = (c * T0 + tid) * 8;
    if (h >= p.H) break;
    store8<VEC>(static_cast<T*>(p.out) + (size_t)t * p.ld_out, h, p.H, v[c]);
  }
}

template <typename T, typename R, bool VEC>
static cudaError_t launch_norm_v(const NormParams& p, cudaStream_t st) {
  const int chunks = cdiv(p.H, 8);
  const int nch = chunks <= 1024 ? 1 : (chunks <= 2048 ? 2 : 4);
  const dim3 block((unsigned)align_up((size_t)cdiv(chunks, nch), 32));
  auto go = [&](auto kernel) { return launch_kernel(kernel, dim3(p.M), block, 0, st, true, p); };
  if (nch == 1) return go(block_norm_kernel<T, R, VEC, 1>);
  if (nch == 2) return go(block_norm_kernel<T, R, VEC, 2>);
  return go(block_norm_kernel<T, R, VEC, 4>);
}
template <typename T, typename R>
static cudaError_t launch_norm_r(const NormParams& p, bool vec, cudaStream_t st) {
  return vec ? launch_norm_v<T, R, true>(p, st) : launch_norm_v<T, R, false>(p, st);
}
template <typename T>
static cudaError_t launch_norm_t(const NormParams& p, bool wide_res, bool vec, cudaStream_t st) {
  return wide_res ? launch_norm_r<T, float>(p, vec, st) : launch_norm_r<T, T>(p, vec, st);
}

// vec: every row of every operand starts on a 16-byte boundary and H % 8 == 0.
cudaError_t launch_block_norm(const moe_norm_args& a, bool vec, cudaStream_t st) {
  NormParams p;
  p.M = a.M; p.H = a.H; p.kind = a.kind; p.wide = a.weight_dtype == MOE_DTYPE_F32;
  p.eps = a.eps; p.scale = a.scale; p.woff = a.weight_offset;
  p.residual = a.residual; p.rows = a.rows; p.ld_res = a.ld_residual; p.ld_rows = a.ld_rows;
  p.slot_of = a.slot_of; p.topk_w = a.topk_weights; p.topk = a.topk; p.n_rows = a.n_rows;
  p.shared = a.shared; p.ld_shared = a.ld_shared;
  p.post_w = a.post_weight; p.post_b = a.post_bias; p.gate = a.gate;
  p.gate_row = a.gate_row; p.gate_col = a.gate_col;
  p.pre_w = a.pre_weight; p.pre_b = a.pre_bias;
  p.res_out = a.residual_out; p.out = a.out; p.ld_res_out = a.ld_residual_out; p.ld_out = a.ld_out;
  const bool wide_res = a.residual_dtype == MOE_DTYPE_F32;
  return a.dtype == MOE_DTYPE_F16 ? launch_norm_t<__half>(p, wide_res, vec, st)
                                  : launch_norm_t<__nv_bfloat16>(p, wide_res, vec, st);
}

}  // namespace moe
