// block_norm.cu - norms before and after a block fused with the experts' top-k combine, the
// block's gate and the residual scale (moe_block_norm).
//
// A CTA works on one token at a time; a thread keeps NCH chunks of 8 consecutive channels in fp32
// registers from the loads to the stores, so every input is read once and every output written
// once, and a norm is one block-wide sum (two for the layer norm: the mean first, then the squares
// around it).  The arithmetic runs on pairs of channels (the packed fp32 instructions).  Two
// kernels: norm_stream_kernel, whose rows arrive by asynchronous copies in a shared-memory ring
// ahead of the arithmetic, and block_norm_kernel, plain loads, for short rows, rows that do not
// start on 16 bytes and rows too long for a ring.  Bound by HBM: 4096 x 7168 with a top-6 combine 91 us (85 % of the
// measured copy bandwidth), 8192 x 6144 with an fp32 residual 102 us (87 %); one token 4.9 us.  Further
// from it: a combine with an fp32 residual, whose ring holds fewer rows (4096 x 7168 117 us, 81 %), and
// rows above 7680 channels (4096 x 8192 top-6 163 us, 54 %; 12288 191 us, 70 %; with an fp32 residual,
// plain loads, 206 and 265 us, 53 and 62 %).
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "block_ops.cuh"
#include "tc_ptx.cuh"
#include "../../include/moe_gb300.h"

namespace moe {

struct NormParams {
  int M, H, kind, wide;             // wide: weights, biases and gate are fp32
  float eps, scale, woff, inv_h;
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
  unsigned long long probe_ns;      // test hook (0: off), see moe_block_norm_set_wait_probe
};

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Eight 16-bit elements of a register vector.
template <typename T>
__device__ __forceinline__ void unpack8(uint4 u, float2 (&v)[4]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2 && std::is_same<T, __half>::value) {
      v[i] = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    } else {
      v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    }
  }
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float2 v) {
  uint32_t w;
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 p = __float22half2_rn(v);
    memcpy(&w, &p, 4);
  } else {
    const __nv_bfloat162 p = __float22bfloat162_rn(v);
    memcpy(&w, &p, 4);
  }
  return w;
}
// Eight elements of a row from element h on; VEC: aligned to the eight (32 bytes of fp32, 16 else)
// and whole, else element by
// element up to H (zeros beyond).
template <bool VEC, typename T>
__device__ __forceinline__ void load8(const T* row, int h, int H, float2 (&v)[4]) {
  if constexpr (VEC && sizeof(T) == 2) {
    unpack8<T>(*reinterpret_cast<const uint4*>(row + h), v);
  } else if constexpr (VEC) {
    const float4 a = *reinterpret_cast<const float4*>(row + h);
    const float4 b = *reinterpret_cast<const float4*>(row + h + 4);
    v[0] = make_float2(a.x, a.y);
    v[1] = make_float2(a.z, a.w);
    v[2] = make_float2(b.x, b.y);
    v[3] = make_float2(b.z, b.w);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = make_float2(h + 2 * i < H ? to_f32(row[h + 2 * i]) : 0.f,
                         h + 2 * i + 1 < H ? to_f32(row[h + 2 * i + 1]) : 0.f);
  }
}
template <bool VEC, typename T>
__device__ __forceinline__ void store8(T* row, int h, int H, const float2 (&v)[4]) {
  if constexpr (VEC && sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(row + h) =
        make_uint4(pack2<T>(v[0]), pack2<T>(v[1]), pack2<T>(v[2]), pack2<T>(v[3]));
  } else if constexpr (VEC) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(row + h),
                 "f"(v[0].x), "f"(v[0].y), "f"(v[1].x), "f"(v[1].y), "f"(v[2].x), "f"(v[2].y),
                 "f"(v[3].x), "f"(v[3].y)
                 : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (h + 2 * i < H) row[h + 2 * i] = from_f32<T>(v[i].x);
      if (h + 2 * i + 1 < H) row[h + 2 * i + 1] = from_f32<T>(v[i].y);
    }
  }
}
// Eight weights of type T or fp32.
template <bool VEC, typename T>
__device__ __forceinline__ void load8w(const void* w, int wide, long long h0, int h, int H,
                                       float2 (&v)[4]) {
  if (wide)
    load8<VEC>(static_cast<const float*>(w) + h0, h, H, v);
  else
    load8<VEC>(static_cast<const T*>(w) + h0, h, H, v);
}

__device__ __forceinline__ void named_sync(int threads) {
  asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
}
// Sum over the first T0 threads of the CTA (whole warps), the same value in each.  s: 32 words of
// this sum's own: a token's sums have a buffer each.
__device__ __forceinline__ float block_sum(float v, float* s, int T0) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = T0 >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane == 0) s[warp] = v;
  named_sync(T0);
  v = lane < warps ? s[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// v = norm(v) * (w + woff) + b over the row's H channels.  s: two buffers of 32 words.  held: the
// thread's 16-bit weights, loaded before (NULL or fp32 weights: loaded here).
template <typename T, bool VEC, int NCH>
__device__ __forceinline__ void norm_row(float2 (&v)[NCH][4], const NormParams& p, int T0,
                                         const void* w, const void* b, float (*s)[32],
                                         const uint4* held = nullptr) {
  float2 sum = both(0.f);
  if (p.kind == MOE_NORM_LAYER) {
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) sum = __fadd2_rn(sum, v[c][i]);
    const float mean = block_sum(sum.x + sum.y, s[1], T0) * p.inv_h;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int h = (c * T0 + threadIdx.x) * 8;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[c][i].x = h + 2 * i < p.H ? v[c][i].x - mean : 0.f;
        v[c][i].y = h + 2 * i + 1 < p.H ? v[c][i].y - mean : 0.f;
      }
    }
    sum = both(0.f);
  }
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) sum = __ffma2_rn(v[c][i], v[c][i], sum);
  const float inv = rsqrtf(block_sum(sum.x + sum.y, s[0], T0) * p.inv_h + p.eps);   // within 2 ulp
  const float shift = inv * p.woff;
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int h = (c * T0 + threadIdx.x) * 8;
    if (h >= p.H) break;
    float2 g[4];
    if (held != nullptr && !p.wide)
      unpack8<T>(held[c], g);
    else
      load8w<VEC, T>(w, p.wide, 0, h, p.H, g);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[c][i] = __fmul2_rn(v[c][i], __ffma2_rn(g[i], both(inv), both(shift)));
    if (b != nullptr) {
      load8w<VEC, T>(b, p.wide, 0, h, p.H, g);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[c][i] = __fadd2_rn(v[c][i], g[i]);
    }
  }
}

// The token's factor of the block's output: scale, times the gate where it is one per token.
template <typename T>
__device__ __forceinline__ float token_factor(const NormParams& p, int t) {
  if (p.gate == nullptr || p.gate_col != 0) return p.scale;
  const size_t o = (size_t)t * p.gate_row;
  return p.scale * (p.wide ? static_cast<const float*>(p.gate)[o]
                           : to_f32(static_cast<const T*>(p.gate)[o]));
}
// One chunk of r = residual + factor * gate * v, stored; v becomes r.
template <typename T, typename R, bool VEC>
__device__ __forceinline__ void add_residual(float2 (&v)[4], const float2 (&r)[4],
                                             const NormParams& p, float factor, int t, int h) {
  if (p.rows == nullptr) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = r[i];
    return;
  }
  if (p.gate != nullptr && p.gate_col != 0) {
    float2 g[4];
    load8w<VEC, T>(p.gate, p.wide, (long long)t * p.gate_row, h, p.H, g);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __fmul2_rn(v[i], g[i]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __ffma2_rn(v[i], both(factor), r[i]);
  if constexpr (!VEC) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {        // nothing past the row, whatever the factors are
      if (h + 2 * i >= p.H) v[i].x = 0.f;
      if (h + 2 * i + 1 >= p.H) v[i].y = 0.f;
    }
  }
  if (p.res_out != nullptr)
    store8<VEC>(static_cast<R*>(p.res_out) + (size_t)t * p.ld_res_out, h, p.H, v);
}
template <typename T, bool VEC, int NCH>
__device__ __forceinline__ void store_normed(float2 (&v)[NCH][4], const NormParams& p, int T0,
                                             int t) {
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int h = (c * T0 + threadIdx.x) * 8;
    if (h >= p.H) break;
    store8<VEC>(static_cast<T*>(p.out) + (size_t)t * p.ld_out, h, p.H, v[c]);
  }
}

// ---------------------------------------------------------------------------------- plain loads

template <typename T, typename R, bool VEC, int NCH>
__global__ void __launch_bounds__(1024)
block_norm_kernel(const NormParams p) {
  __shared__ float s_sum[4][32];
  const int t = blockIdx.x, T0 = blockDim.x, tid = threadIdx.x;
  pdl_wait_prev();
  pdl_launch_next();
  float2 v[NCH][4];
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) v[c][i] = both(0.f);

  // v += w * row
  const auto add_row = [&](const void* base, long long at, float w) {
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int h = (c * T0 + tid) * 8;
      if (h >= p.H) break;
      float2 y[4];
      load8<VEC>(static_cast<const T*>(base) + at, h, p.H, y);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[c][i] = __ffma2_rn(both(w), y[i], v[c][i]);
    }
  };
  if (p.rows != nullptr) {
    if (p.slot_of == nullptr) {
      add_row(p.rows, (long long)t * p.ld_rows, 1.f);
    } else {
      for (int j = 0; j < p.topk; ++j) {
        const int slot = p.slot_of[(size_t)t * p.topk + j];
        if (slot >= 0 && slot < p.n_rows)
          add_row(p.rows, (long long)slot * p.ld_rows, p.topk_w[(size_t)t * p.topk + j]);
      }
      if (p.shared != nullptr) add_row(p.shared, (long long)t * p.ld_shared, 1.f);
    }
    if (p.post_w != nullptr) norm_row<T, VEC, NCH>(v, p, T0, p.post_w, p.post_b, s_sum);
  }
  const float factor = token_factor<T>(p, t);
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int h = (c * T0 + tid) * 8;
    if (h >= p.H) break;
    float2 r[4];
    load8<VEC>(static_cast<const R*>(p.residual) + (size_t)t * p.ld_res, h, p.H, r);
    add_residual<T, R, VEC>(v[c], r, p, factor, t, h);
  }
  if (p.pre_w == nullptr) return;
  norm_row<T, VEC, NCH>(v, p, T0, p.pre_w, p.pre_b, s_sum + 2);
  store_normed<T, VEC, NCH>(v, p, T0, t);
}

// ---------------------------------------------------------------------------------- row ring
//
// Persistent CTAs of T0 summing threads and one copying warp.  A token's rows (its experts', the
// shared one, the residual) come through a ring of `slots` buffers, one bulk copy each, in the
// order in which they are taken; the copying warp knows where they are, so the summing threads
// spend no instructions on addresses (with those in every thread the kernel was bound by
// instruction issue), and the copies of the next tokens are in flight while this one is summed,
// normalised and stored.

// Error word of the row copies' bounded waits (moe_block_norm_get_device_error).
__device__ int32_t g_norm_error;

template <typename T, typename R, int NCH, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT + 32, MINB)
norm_stream_kernel(const NormParams p, const int slots, const int slot_bytes) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(8) uint64_t full[kNormSlots], empty[kNormSlots];
  __shared__ float s_weight[kNormSlots];   // the row's router weight
  __shared__ int s_on[kNormSlots];         // 0: the slot was dropped, the buffer holds nothing
  __shared__ float s_sum[4][32];
  const int tid = threadIdx.x, lane = tid & 31, T0 = blockDim.x - 32;
  if (tid == 0) {
    for (int i = 0; i < slots; ++i) {
      tc::mbar_init(&full[i], 1);
      tc::mbar_init(&empty[i], T0 >> 5);
    }
    tc::fence_barrier_init();
  }
  __syncthreads();
  pdl_wait_prev();
  pdl_launch_next();
  const int experts = p.slot_of != nullptr ? p.topk : 0;
  const int n_rows = p.rows == nullptr ? 0 : (experts ? experts + (p.shared != nullptr) : 1);

  if (tid >= T0) {                         // the copying warp
    const int per = n_rows + 1;
    int b = 0, phase = 1, issued = 0;
    bool ok = true;
    // no buffer is freed before one is filled
    if (p.probe_ns != 0 && blockIdx.x == 0)
      ok = __all_sync(0xffffffffu, tc::mbar_wait(&empty[0], 0, &g_norm_error, p.probe_ns));
    // 32 rows at a time: lane l finds row l of them, then the rows are copied in order
    int t = blockIdx.x, j = 0;             // the first of the 32
    while (ok && t < p.M) {
      int lt = t, lj = j + lane;
      while (lj >= per) {
        lj -= per;
        lt += gridDim.x;
      }
      const uint8_t* src = nullptr;
      uint32_t bytes = (uint32_t)p.H * sizeof(T);
      float w = 1.f;
      if (lt < p.M) {
        if (lj == n_rows) {
          src = static_cast<const uint8_t*>(p.residual) + (size_t)lt * p.ld_res * sizeof(R);
          bytes = (uint32_t)p.H * sizeof(R);
        } else if (lj < experts) {
          const int slot = p.slot_of[(size_t)lt * experts + lj];
          w = p.topk_w[(size_t)lt * experts + lj];
          if (slot >= 0 && slot < p.n_rows)
            src = static_cast<const uint8_t*>(p.rows) + (size_t)slot * p.ld_rows * sizeof(T);
        } else if (experts) {
          src = static_cast<const uint8_t*>(p.shared) + (size_t)lt * p.ld_shared * sizeof(T);
        } else {
          src = static_cast<const uint8_t*>(p.rows) + (size_t)lt * p.ld_rows * sizeof(T);
        }
      }
      const int n = __popc(__ballot_sync(0xffffffffu, lt < p.M));
      for (int l = 0; ok && l < n; ++l) {
        if (lane == l) {
          ok = tc::mbar_wait(&empty[b], phase, &g_norm_error);
          if (ok) {
            s_weight[b] = w;
            s_on[b] = src != nullptr;
            if (src != nullptr) {
              tc::mbar_arrive_expect_tx(&full[b], bytes);
              tc::bulk_load(ring + (size_t)b * slot_bytes, src, bytes, &full[b]);
            } else {
              tc::mbar_arrive(&full[b]);
            }
          }
        }
        ok = __all_sync(0xffffffffu, ok);
        issued += ok;
        if (++b == slots) {
          b = 0;
          phase ^= 1;
        }
      }
      j += 32;
      while (j >= per) {
        j -= per;
        t += gridDim.x;
      }
    }
    // no copy may be in flight when the CTA ends, also where the summing threads gave up a wait
    if (lane == 0)
      for (int i = max(0, issued - slots); i < issued; ++i)
        tc::mbar_wait(&full[i % slots], (i / slots) & 1, &g_norm_error);
    return;
  }

  int b = 0, phase = 0;
  bool ok = true;                          // after a wait gave up, none is made any more
  const auto wait_row = [&]() {
    if (ok) ok = tc::mbar_wait(&full[b], phase, &g_norm_error);
  };
  const auto free_row = [&]() {
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&empty[b]);
    if (++b == slots) {
      b = 0;
      phase ^= 1;
    }
  };
  for (int t = blockIdx.x; t < p.M; t += gridDim.x) {
    float2 v[NCH][4];
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[c][i] = both(0.f);
    const float factor = token_factor<T>(p, t);
    // weights ahead of their use (they come from L2: the ring takes the L1's space)
    uint4 held[NCH];
    const auto hold = [&](const void* w) {
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const int h = (c * T0 + tid) * 8;
        if (w != nullptr && !p.wide && h < p.H)
          held[c] = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(w) + h));
      }
    };
    hold(p.post_w);
#pragma unroll 1
    for (int j = 0; j < n_rows; ++j) {
      wait_row();
      if (s_on[b]) {
        const float2 w = both(s_weight[b]);
        const uint8_t* row = ring + (size_t)b * slot_bytes + tid * 16;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
          if ((c * T0 + tid) * 8 >= p.H) break;
          float2 y[4];
          unpack8<T>(*reinterpret_cast<const uint4*>(row + c * T0 * 16), y);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[c][i] = __ffma2_rn(w, y[i], v[c][i]);
        }
      }
      free_row();
    }
    if (p.post_w != nullptr) norm_row<T, true, NCH>(v, p, T0, p.post_w, p.post_b, s_sum, held);
    hold(p.pre_w);
    wait_row();
    const R* res = reinterpret_cast<const R*>(ring + (size_t)b * slot_bytes);
    float2 r[NCH][4];
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int h = (c * T0 + tid) * 8;
      if (h < p.H) load8<true>(res, h, p.H, r[c]);
    }
    free_row();
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int h = (c * T0 + tid) * 8;
      if (h < p.H) add_residual<T, R, true>(v[c], r[c], p, factor, t, h);
    }
    if (p.pre_w != nullptr) {
      norm_row<T, true, NCH>(v, p, T0, p.pre_w, p.pre_b, s_sum + 2, held);
      store_normed<T, true, NCH>(v, p, T0, t);
    }
    // a sum's buffer is written again only after a barrier that follows its reads
    if (p.post_w == nullptr || p.pre_w == nullptr) named_sync(T0);
  }
}

// ---------------------------------------------------------------------------------- host side

static int sm_count() {
  static PerDevice<int> per;
  int n = 0;
  if (on_device(per, &n, [](int* v) {
        int dev = 0;
        const cudaError_t e = cudaGetDevice(&dev);
        return e != cudaSuccess ? e : cudaDeviceGetAttribute(v, cudaDevAttrMultiProcessorCount, dev);
      }) != cudaSuccess || n < 1) {
    (void)cudaGetLastError();
    return 152;
  }
  return n;
}

template <typename T, typename R, int NCH, int MAXT, int MINB>
static cudaError_t launch_stream(const NormParams& p, int threads, int slots, cudaStream_t st) {
  const int slot_bytes = p.H * (int)sizeof(R), smem = slots * slot_bytes;
  auto kernel = norm_stream_kernel<T, R, NCH, MAXT, MINB>;
  static PerDevice<bool> per;
  bool set = false;
  cudaError_t e = on_device(per, &set, [&](bool*) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormRings);
  });
  if (e != cudaSuccess) return e;
  int n = 0;
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads + 32, smem);
  if (e != cudaSuccess) return e;
  const int grid = std::min(p.M, std::max(1, n) * sm_count());
  return launch_kernel(kernel, dim3(grid), dim3(threads + 32), (size_t)smem, st, true, p, slots,
                       slot_bytes);
}

template <typename T, typename R, bool VEC>
static cudaError_t launch_norm_v(const NormParams& p, cudaStream_t st) {
  const NormShape n = norm_shape(p.M, p.H, (int)sizeof(R), VEC, p.slot_of != nullptr, sm_count());
  if constexpr (VEC) {
    if (n.ring && n.nch == 2) return launch_stream<T, R, 2, 480, 2>(p, n.threads, n.slots, st);
    // (two buffers of an fp32 residual's size do not fit where rows take four chunks)
    if constexpr (sizeof(R) == 2)
      if (n.ring) return launch_stream<T, R, 4, 480, 1>(p, n.threads, n.slots, st);
  }
  auto go = [&](auto kernel) {
    return launch_kernel(kernel, dim3(p.M), dim3(n.threads), 0, st, true, p);
  };
  if (n.nch == 1) return go(block_norm_kernel<T, R, VEC, 1>);
  if (n.nch == 2) return go(block_norm_kernel<T, R, VEC, 2>);
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

// Reads and clears the error word of the row copies' waits.
cudaError_t norm_device_error(int* code, cudaStream_t st) {
  int32_t word = 0;
  const int32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(&word, g_norm_error, sizeof(word), 0,
                                            cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && word != 0) {
    e = cudaMemcpyToSymbolAsync(g_norm_error, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  }
  *code = word;
  return e;
}

static std::atomic<unsigned long long> g_norm_probe{0};
void set_norm_probe(unsigned long long ns) { g_norm_probe = ns; }

// vec: every row of every operand starts on a boundary of eight elements and H % 8 == 0.
cudaError_t launch_block_norm(const moe_norm_args& a, bool vec, cudaStream_t st) {
  NormParams p;
  p.M = a.M; p.H = a.H; p.kind = a.kind; p.wide = a.weight_dtype == MOE_DTYPE_F32;
  p.eps = a.eps; p.scale = a.scale; p.woff = a.weight_offset; p.inv_h = 1.f / (float)a.H;
  p.residual = a.residual; p.rows = a.rows; p.ld_res = a.ld_residual; p.ld_rows = a.ld_rows;
  p.slot_of = a.slot_of; p.topk_w = a.topk_weights; p.topk = a.topk; p.n_rows = a.n_rows;
  p.shared = a.shared; p.ld_shared = a.ld_shared;
  p.post_w = a.post_weight; p.post_b = a.post_bias; p.gate = a.gate;
  p.gate_row = a.gate_row; p.gate_col = a.gate_col;
  p.pre_w = a.pre_weight; p.pre_b = a.pre_bias;
  p.res_out = a.residual_out; p.out = a.out; p.ld_res_out = a.ld_residual_out; p.ld_out = a.ld_out;
  p.probe_ns = g_norm_probe;
  const bool wide_res = a.residual_dtype == MOE_DTYPE_F32;
  return a.dtype == MOE_DTYPE_F16 ? launch_norm_t<__half>(p, wide_res, vec, st)
                                  : launch_norm_t<__nv_bfloat16>(p, wide_res, vec, st);
}

}  // namespace moe
