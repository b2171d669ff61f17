// gemv_fp8.cu - 8-bit products with block scales for a few positions, of one matrix or over experts (one token's),
// where they are few enough for this launch (fp8_few_takes in block_launch.cuh: the rule and both sides' times).
//
// Bound by reading the weights once.  One to eight warps to an output column (SwiGLU: to a pair of weight
// rows), as many as fill the GPU; a lane takes 16 codes of every row at a time, all of one block, sums
// their products in fp32 and adds them times both scales.  Sums go lane by lane, then over the lanes, then
// over the warps: one order.  Positions of one matrix share its rows; where there are offsets each position reads its
// expert's, also where two have the same one: a matrix sweep apart, so from L2 only where the matrix fits there.
#include <cuda_fp8.h>

#include "block_ops.cuh"
#include "fp8.cuh"
#include "../../include/moe_gb300.h"

namespace moe {

struct F8vParams {
  GroupedDims d;
  Fp8Call f;
  int cols, KB, tall, warps;
};

// 16 codes as fp32.
__device__ __forceinline__ void e4m3_unpack16(const uint4& w, float (&f)[16]) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(v[i / 2] >> (16 * (i % 2))), __NV_E4M3);
    const float2 x = __half22float2(__half2(h));
    f[2 * i] = x.x;
    f[2 * i + 1] = x.y;
  }
}

template <typename T, bool ACT, int NC>
__global__ void __launch_bounds__(kF8vThreads) fp8_gemv_kernel(const F8vParams p) {
  constexpr int kSets = ACT ? 2 : 1, kF8vAhead = 4;
  __shared__ float s_sum[kF8vWarps][kSets * NC];
  const GroupedCall& c = p.f.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % p.warps;
  const int col = blockIdx.x * (kF8vWarps / p.warps) + warp / p.warps;
  const int p0 = blockIdx.y * NC;
  T* out = static_cast<T*>(c.out);
  pdl_wait_prev();
  pdl_launch_next();
  int e = 0;
  if (c.offsets != nullptr) {            // the expert of position p0 (NC is 1 then): experts that end at or before it
    bool bad = false;
    for (int i = lane; i < p.d.E; i += 32) {
      const int a = c.offsets[i], b = c.offsets[i + 1];
      bad |= a < 0 || b < a || b > c.S;
      e += b <= p0;
    }
    e = __reduce_add_sync(0xffffffffu, e);
    if (__any_sync(0xffffffffu, bad)) {
      set_error(c.err, kErrRouteBounds);
      return;                            // every thread of the call
    }
    if (e >= p.d.E) {                    // past the last group
      if (lane == 0 && part == 0 && col < p.cols) out[p0 * c.ldo + col] = from_f32<T>(0.f);
      return;                            // every thread of the CTA
    }
    if (c.offsets[e] > p0) return;       // before the first
  }
  long long row[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int pos = min(p0 + i, c.S - 1);
    row[i] = pos;
    if (c.perm != nullptr) {
      const int f = c.perm[pos];
      row[i] = f < 0 ? -1 : f / c.topk;
      if (row[i] < 0 || row[i] >= c.x_rows) {
        set_error(c.err, kErrRouteBounds);
        row[i] = 0;
      }
    }
  }
  const int half = p.d.N / 2, mine = min(col, p.cols - 1), K = p.d.K, stride = p.warps * 512;
  const uint8_t* x = static_cast<const uint8_t*>(c.x);
  const uint8_t* w[kSets];
  const float* ws[kSets];
#pragma unroll
  for (int h = 0; h < kSets; ++h) {
    const int wr = mine + h * half;
    w[h] = static_cast<const uint8_t*>(c.w) + ((size_t)e * p.d.N + wr) * c.ldw;
    ws[h] = p.f.ws + ((size_t)e * p.tall + fp8_scale_row(p.d, wr)) * p.KB;
  }
  float acc[kSets][NC] = {};
  for (int k0 = (part * 32 + lane) * 16; k0 < K; k0 += kF8vAhead * stride) {
    uint4 a[kSets][kF8vAhead];
#pragma unroll
    for (int h = 0; h < kSets; ++h) load_once16x4(a[h], w[h] + k0, stride, cdiv(K - k0, stride));
#pragma unroll
    for (int i = 0; i < kF8vAhead; ++i) {
      const int k = k0 + i * stride;
      const bool in = k < K;
      float wf[kSets][16], sa[kSets];
#pragma unroll
      for (int h = 0; h < kSets; ++h) {
        sa[h] = in ? ws[h][k / kFp8Block] : 0.f;
        e4m3_unpack16(a[h][i], wf[h]);
      }
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const float sb = in ? p.f.xs[row[j] * p.f.ldxs + k / kFp8Block] : 0.f;
        float xf[16];
        e4m3_unpack16(in ? *reinterpret_cast<const uint4*>(x + row[j] * c.ldx + k) : make_uint4(0, 0, 0, 0), xf);
#pragma unroll
        for (int h = 0; h < kSets; ++h) {
          float s = 0.f;
#pragma unroll
          for (int t = 0; t < 16; ++t) s = fmaf(wf[h][t], xf[t], s);
          acc[h][j] = fmaf(s, sa[h] * sb, acc[h][j]);
        }
      }
    }
  }
#pragma unroll
  for (int h = 0; h < kSets; ++h)
#pragma unroll
    for (int j = 0; j < NC; ++j) {
#pragma unroll
      for (int o = 16; o; o >>= 1) acc[h][j] += __shfl_xor_sync(0xffffffffu, acc[h][j], o);
      if (lane == 0) s_sum[warp][h * NC + j] = acc[h][j];
    }
  __syncthreads();
  if (part != 0 || col >= p.cols || lane >= min(NC, c.S - p0)) return;
  float v[kSets];
#pragma unroll
  for (int h = 0; h < kSets; ++h) {
    v[h] = 0.f;
    for (int i = 0; i < p.warps; ++i) v[h] += s_sum[warp + i][h * NC + lane];
  }
  float y = v[0];
  if constexpr (ACT) {
    const bool up_first = p.d.layout == MOE_W13_UP_GATE;
    y = swiglu_f32(v[up_first ? 0 : 1], v[up_first ? 1 : 0], p.d.limit, p.d.alpha, p.d.beta);
  }
  out[(long long)(p0 + lane) * c.ldo + col] = from_f32<T>(y);
}

// A few positions in whole vectors (their alignment as for the tensor cores).
cudaError_t fp8_gemv_takes(const GroupedDims& d, const Fp8Call& f, bool* takes) {
  int sms = 0;
  const cudaError_t e = device_sms(&sms);
  *takes = e == cudaSuccess && fp8_few_takes(f.c.S, d.E, f.c.offsets != nullptr, d.act != 0, d.N, d.K, sms);
  return e;
}

template <typename T, bool ACT>
static cudaError_t launch_f8v(F8vParams& p, cudaStream_t st) {
  int sms = 0;
  const cudaError_t e = device_sms(&sms);
  if (e != cudaSuccess) return e;
  const F8vShape f = fp8_few_shape(p.f.c.S, p.f.c.offsets != nullptr, p.cols, p.d.K, sms);
  p.warps = f.warps;
  const auto go = [&](auto kernel) { return launch_kernel(kernel, dim3(f.x, f.y), dim3(kF8vThreads), 0, st, true, p); };
  if (f.nc == 1) return go(fp8_gemv_kernel<T, ACT, 1>);
  return f.nc == 2 ? go(fp8_gemv_kernel<T, ACT, 2>) : go(fp8_gemv_kernel<T, ACT, 4>);
}

cudaError_t launch_fp8_gemv(const GroupedDims& d, const Fp8Call& f, cudaStream_t st) {
  F8vParams p{d, f, grouped_cols(d), fp8_blocks(d.K), fp8_tall(d), 1};
  if (d.dtype == MOE_DTYPE_F16)
    return d.act ? launch_f8v<__half, true>(p, st) : launch_f8v<__half, false>(p, st);
  return d.act ? launch_f8v<__nv_bfloat16, true>(p, st) : launch_f8v<__nv_bfloat16, false>(p, st);
}

}  // namespace moe
