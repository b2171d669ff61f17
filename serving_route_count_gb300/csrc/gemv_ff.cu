// gemv_ff.cu - products of the gated feed-forward block's forward pass for one or two tokens:
// out[c][r] = act(sum_k R(r, k) C(c, k)), both operands along K.
//
// Bound by reading the weights once.  One to eight warps to an output row (GLU: to a pair of rows, up and
// gate), as many as fill the GPU; a lane takes 16 bytes of every row at a time, four of them in flight, and
// multiplies in fp32 on the CUDA cores, which at so few tokens keep up with HBM.  Sums go lane by lane, then
// over the lanes, then over the warps: one order.  Units on the tensor cores are cut into pieces for this,
// which are joined: us of a forward pass here / there, weights in L2: 6144 -> 512 one token 7.3 / 20.0, two
// 9.3 / 17.8, four (were they taken) 16.4 / 17.8;  7168 -> 1152 11.9 / 21.2, 16.6 / 21.3, 31.7 / 21.3;  4096 -> 4096
// 21.5 / 28.5, 27.0 / 29.5, 50.5 / 28.8.  From HBM, one / two tokens: 7168 -> 1152 14.5 / 23.9, 19.4 / 23.9 (weights 7.3);
// 512 -> 512 3.8 / 9.9, 4.2 / 9.8;  7168 -> 4608 39.6 / 53.4, 49.5 / 51.4;  16384 -> 2048 40.3 / 48.4, 48.2 / 48.6; only the
// largest lose, 8192 -> 16384 142 / 135, 161 / 136.
#include "feed_forward.cuh"
#include "../../include/moe_gb300.h"

namespace moe {

constexpr int kFvThreads = 256, kFvWarps = kFvThreads / 32, kFvAhead = 4;

struct FvParams {
  FfDims d;
  FfGemm g;
  int warps;            // of an output
  int early;            // weights may be read before the kernel before this one is over
};

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& w, float (&f)[8]) {
  T t[8];
  memcpy(t, &w, 16);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = to_f32(t[i]);
}

template <typename T, int EPI, int NC>
__global__ void __launch_bounds__(kFvThreads) ff_gemv_kernel(const FvParams p) {
  constexpr int kSets = EPI == kFfGlu ? 2 : 1;
  __shared__ float s_sum[kFvWarps][kSets * NC];
  const FfGemm& g = p.g;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % p.warps;
  const int r = blockIdx.x * (kFvWarps / p.warps) + warp / p.warps;
  const int stride = p.warps * 256;
  const T* R = static_cast<const T*>(g.r) + min(r, g.nr - 1) * g.rs;
  const T* C = static_cast<const T*>(g.c);
  const int k00 = (part * 32 + lane) * 8;
  uint4 w[kSets][kFvAhead];
  const auto load = [&](int k0) {
#pragma unroll
    for (int h = 0; h < kSets; ++h)
      load_once16x4(w[h], R + h * g.half + k0, stride * (long long)sizeof(T), cdiv(g.K - k0, stride));
  };
  if (!p.early) pdl_wait_prev();
  load(k00);
  if (p.early) pdl_wait_prev();
  pdl_launch_next();
  float acc[kSets][NC] = {};
  for (int k0 = k00; k0 < g.K; k0 += kFvAhead * stride) {
    if (k0 != k00) load(k0);
#pragma unroll
    for (int i = 0; i < kFvAhead; ++i) {
      const int k = k0 + i * stride;
      float a[kSets][8];
#pragma unroll
      for (int h = 0; h < kSets; ++h) unpack8<T>(w[h][i], a[h]);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float b[8];
        unpack8<T>(k < g.K ? *reinterpret_cast<const uint4*>(C + min(c, g.nc - 1) * g.cs + k) : make_uint4(0, 0, 0, 0), b);
#pragma unroll
        for (int h = 0; h < kSets; ++h)
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[h][c] = fmaf(a[h][j], b[j], acc[h][c]);
      }
    }
  }
#pragma unroll
  for (int h = 0; h < kSets; ++h)
#pragma unroll
    for (int c = 0; c < NC; ++c) {
#pragma unroll
      for (int o = 16; o; o >>= 1) acc[h][c] += __shfl_xor_sync(0xffffffffu, acc[h][c], o);
      if (lane == 0) s_sum[warp][h * NC + c] = acc[h][c];
    }
  __syncthreads();
  if (part != 0 || r >= g.nr || lane >= min(NC, g.nc)) return;
  float v[kSets];
#pragma unroll
  for (int h = 0; h < kSets; ++h) {
    v[h] = 0.f;
    for (int i = 0; i < p.warps; ++i) v[h] += s_sum[warp + i][h * NC + lane];
  }
  T* o = static_cast<T*>(g.out) + lane * g.ldo + r;
  if constexpr (EPI == kFfStore) {
    *o = from_f32<T>(v[0]);
  } else {
    const bool up_first = p.d.layout == MOE_W13_UP_GATE;
    const float u = v[up_first ? 0 : 1], gt = v[up_first ? 1 : 0];
    *o = from_f32<T>(swiglu_f32(u, gt, p.d.limit, p.d.alpha, p.d.beta));
    if (g.pre != nullptr) {
      float* s = g.pre + (long long)lane * 2 * g.nr + r;
      s[up_first ? 0 : g.nr] = u;
      s[up_first ? g.nr : 0] = gt;
    }
  }
}

// One or two tokens, both operands along K in whole vectors (their alignment as for the tensor cores).
bool ff_gemv_takes(const FfGemm& g, int epilogue) {
  return g.nc <= 2 && g.rk == 1 && g.ck == 1 && g.K % 8 == 0 && epilogue != kFfGrad;
}

template <typename T, int EPI>
static cudaError_t launch_fv(FvParams& p, cudaStream_t st) {
  // warps enough for every SM to have 16, as far as each still has a vector of every lane
  int sms = 0;
  const cudaError_t e = device_sms(&sms);
  if (e != cudaSuccess) return e;
  p.warps = 1;
  while (p.warps < kFvWarps && p.g.nr * p.warps < sms * 16 && p.g.K > p.warps * 256) p.warps *= 2;
  const dim3 grid(cdiv(p.g.nr, kFvWarps / p.warps));
  const auto go = [&](auto kernel) { return launch_kernel(kernel, grid, dim3(kFvThreads), 0, st, true, p); };
  return p.g.nc == 1 ? go(ff_gemv_kernel<T, EPI, 1>) : go(ff_gemv_kernel<T, EPI, 2>);
}

// early: the launch before this one in the stream is the block's own first product, which does not write these
// weights, and which itself began after everything before it was over; they are then on their way while it
// runs (one token of 7168 -> 1152 -> 7168: 18.0 -> 15.2 us).
cudaError_t launch_ff_gemv(const FfDims& d, const FfGemm& g, int epilogue, bool early, cudaStream_t st) {
  FvParams p{d, g, 1, early};
  if (d.dtype == MOE_DTYPE_F16)
    return epilogue == kFfGlu ? launch_fv<__half, kFfGlu>(p, st) : launch_fv<__half, kFfStore>(p, st);
  return epilogue == kFfGlu ? launch_fv<__nv_bfloat16, kFfGlu>(p, st) : launch_fv<__nv_bfloat16, kFfStore>(p, st);
}

}  // namespace moe
