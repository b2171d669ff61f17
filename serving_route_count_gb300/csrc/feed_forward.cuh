// feed_forward.cuh - what the kernels of the gated feed-forward block (moe_ff_forward, moe_ff_backward)
// and the C ABI share: a block's products in one form, and the activation's pieces.
#pragma once

#include "block_ops.cuh"
#include "grouped.cuh"

namespace moe {

struct FfDims {
  int H, I, dtype, layout, max_rows;
  float limit, alpha, beta;
  unsigned long long probe_ns;         // test hook (0: off), see moe_ff_set_wait_probe
};

// One product of the block: out[c][r] = sum_k R(r, k) C(c, k).  R(r, k) is at r[r * rs + k * rk], one
// of rs and rk 1 (rows along K, or a matrix that is stored the other way round), C likewise.
enum FfEpilogue {
  kFfStore = 0,       // out = sum
  kFfGlu = 1,         // R has two halves of nr rows, `half` apart: out = act(their sums), and with pre
                      // both sums there (columns r and nr + r)
  kFfGrad = 2,        // sum = dh: out's columns r and nr + r get the gradients of the two halves, from pre
};
struct FfGemm {
  const void* r;
  long long rs, rk, half;              // half: elements between the halves' rows (kFfGlu)
  const void* c;
  long long cs, ck;
  int nr, nc, K;
  void* out;
  long long ldo;
  float* pre;                          // [nc, 2 nr]: written (kFfGlu, or NULL), read (kFfGrad)
  int32_t* err;                        // device error word
};

// Gradients of swiglu_f32 by up and gate, times dh.  A clamp passes the gradient within its bounds, the
// bounds included.  With s = sigmoid(a), a = alpha g': d/dg' (g' s (u' + beta)) = (u' + beta) (s + a s (1 - s)),
// s (1 - s) = e / (1 + e)^2, e = exp(-|a|).  Where e is 0 the second term is 0, whatever a is.
__device__ __forceinline__ void swiglu_grad(float u, float g, float dh, float limit, float alpha,
                                            float beta, float* du, float* dg) {
  const bool u_in = !(fabsf(u) > limit), g_in = !(g > limit);
  float gc = g, uc = u;
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(gc) : "f"(limit));      // NaN stays NaN
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(uc) : "f"(limit));
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(uc) : "f"(-limit));
  const float a = alpha * gc, e = __expf(-fabsf(a));
  const float inv = __fdividef(1.0f, 1.0f + e);                // divisor within [1, 2]
  const float s = a < 0.f ? e * inv : inv;
  const float slope = e == 0.f ? s : fmaf(a * e * inv, inv, s);
  *du = u_in ? dh * (gc * s) : 0.f;
  *dg = g_in ? dh * (uc + beta) * slope : 0.f;
}

}  // namespace moe
