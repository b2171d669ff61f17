// api_ff.cu - host side of the gated feed-forward block: argument checks, the products of a forward and
// of a backward pass, launches.
#include <cmath>
#include <new>

#include "feed_forward.cuh"
#include "../../include/moe_gb300.h"

namespace moe {
// api.cu: records the error for moe_last_cuda_error
int report_cuda(cudaError_t e);
// gemm_ff_simt.cu
cudaError_t launch_ff_simt(const FfDims& d, const FfGemm& g, int epilogue, cudaStream_t st);
// gemv_ff.cu
bool ff_gemv_takes(const FfGemm& g, int epilogue);
cudaError_t launch_ff_gemv(const FfDims& d, const FfGemm& g, int epilogue, bool early, cudaStream_t st);
// gemm_ff_tc.cu
size_t ff_tc_part_bytes(int max_rows);
bool ff_tc_addressable(const FfGemm& g);
cudaError_t launch_ff_tc(const FfDims& d, const FfGemm& g, int epilogue, float* part, int32_t* tickets,
                         cudaStream_t st);
}  // namespace moe

using namespace moe;

struct moe_ff_s {
  FfDims d;
  size_t rows_at, bytes;                  // scratch: the rows between two products; all of it
};

namespace {

moe_status status(cudaError_t e) { return static_cast<moe_status>(report_cuda(e)); }

// after: the launch before this one is this call's, and writes C alone of this product's operands
cudaError_t product(const moe_ff_s& f, const FfGemm& g, int epilogue, cudaStream_t st, bool after = false) {
  if (!ff_tc_addressable(g)) return launch_ff_simt(f.d, g, epilogue, st);
  if (ff_gemv_takes(g, epilogue)) return launch_ff_gemv(f.d, g, epilogue, after, st);
  uint8_t* base = reinterpret_cast<uint8_t*>(g.err);      // the scratch buffer begins with the error word
  return launch_ff_tc(f.d, g, epilogue, reinterpret_cast<float*>(base + kGtPartAt),
                      reinterpret_cast<int32_t*>(base + kGtTicketsAt), st);
}

bool scratch_ok(const moe_ff_s& f, const void* scratch, size_t bytes) {
  return scratch != nullptr && bytes >= f.bytes && (reinterpret_cast<uintptr_t>(scratch) & 255) == 0;
}

}  // namespace

extern "C" {

moe_status moe_ff_plan(int H, int I, int dtype, int layout, float limit, float alpha, float beta,
                       int max_rows, moe_ff_t** out) {
  if (out == nullptr) return MOE_ERR_ARG;
  *out = nullptr;
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16) return MOE_ERR_UNSUPPORTED;
  if (layout != MOE_W13_UP_GATE && layout != MOE_W13_GATE_UP) return MOE_ERR_ARG;
  if (std::isnan(limit) || limit <= 0.f || !std::isfinite(alpha) || !std::isfinite(beta))
    return MOE_ERR_ARG;
  if (H < 1 || H > (1 << 20) || I < 1 || I > (1 << 20) || max_rows < 0 || max_rows > (1 << 24))
    return MOE_ERR_SHAPE;
  moe_ff_s* f = new (std::nothrow) moe_ff_s();
  if (f == nullptr) return MOE_ERR_ARG;
  f->d = FfDims{H, I, dtype, layout, max_rows, limit, alpha, beta, 0};
  f->rows_at = kGtPartAt + ff_tc_part_bytes(max_rows);
  // h [M, I] of a forward pass, d(up, gate) [M, 2 I] of a backward one
  f->bytes = f->rows_at + align_up((size_t)max_rows * 2 * I * 2, 256);
  *out = f;
  return MOE_OK;
}

moe_status moe_ff_set_wait_probe(moe_ff_t* plan, unsigned long long ns) {
  if (plan == nullptr || ns > 1000000000ull) return MOE_ERR_ARG;
  plan->d.probe_ns = ns;
  return MOE_OK;
}

void moe_destroy_ff(moe_ff_t* plan) { delete plan; }

moe_status moe_ff_scratch_bytes(const moe_ff_t* plan, size_t* bytes) {
  if (plan == nullptr || bytes == nullptr) return MOE_ERR_ARG;
  *bytes = plan->bytes;
  return MOE_OK;
}

moe_status moe_ff_forward(const moe_ff_t* plan, void* scratch, size_t scratch_bytes, const void* x,
                          long long ldx, const void* w13, long long ldw13, const void* w2, long long ldw2,
                          float* pre, void* h, void* y, long long ldy, int M, void* stream) {
  if (plan == nullptr || M < 0) return MOE_ERR_ARG;
  const FfDims& d = plan->d;
  if (M > d.max_rows) return MOE_ERR_CAPACITY;
  if ((pre != nullptr) != (h != nullptr) && M > 0) return MOE_ERR_ARG;
  if (M == 0) return MOE_OK;
  if (!scratch_ok(*plan, scratch, scratch_bytes)) return MOE_ERR_ARG;
  if (x == nullptr || w13 == nullptr || w2 == nullptr || y == nullptr) return MOE_ERR_ARG;
  if (ldx < d.H || ldw13 < d.H || ldw2 < d.I || ldy < d.H) return MOE_ERR_ARG;
  int32_t* err = static_cast<int32_t*>(scratch);
  if (h == nullptr) h = static_cast<uint8_t*>(scratch) + plan->rows_at;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = product(*plan, FfGemm{w13, ldw13, 1, ldw13 * d.I, x, ldx, 1, d.I, M, d.H, h, d.I, pre, err},
                          kFfGlu, st);
  if (e == cudaSuccess)
    e = product(*plan, FfGemm{w2, ldw2, 1, 0, h, d.I, 1, d.H, M, d.I, y, ldy, nullptr, err}, kFfStore, st, true);
  return status(e);
}

moe_status moe_ff_backward(const moe_ff_t* plan, void* scratch, size_t scratch_bytes, const void* dy,
                           long long lddy, const void* x, long long ldx, const void* w13, long long ldw13,
                           const void* w2, long long ldw2, const float* pre, const void* h, void* dx,
                           long long lddx, void* dw13, long long lddw13, void* dw2, long long lddw2, int M,
                           void* stream) {
  if (plan == nullptr || M < 0) return MOE_ERR_ARG;
  const FfDims& d = plan->d;
  if (M > d.max_rows) return MOE_ERR_CAPACITY;
  if ((dw13 && lddw13 < d.H) || (dw2 && lddw2 < d.I)) return MOE_ERR_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (M == 0) {                           // sums over no tokens
    cudaError_t e = cudaSuccess;
    if (dw13) e = cudaMemset2DAsync(dw13, (size_t)lddw13 * 2, 0, (size_t)d.H * 2, 2 * (size_t)d.I, st);
    if (dw2 && e == cudaSuccess) e = cudaMemset2DAsync(dw2, (size_t)lddw2 * 2, 0, (size_t)d.I * 2, d.H, st);
    return status(e);
  }
  if (!scratch_ok(*plan, scratch, scratch_bytes)) return MOE_ERR_ARG;
  if (dy == nullptr || lddy < d.H) return MOE_ERR_ARG;
  const bool inner = dx != nullptr || dw13 != nullptr;
  if (inner && (w2 == nullptr || pre == nullptr || ldw2 < d.I)) return MOE_ERR_ARG;
  if (dx && (w13 == nullptr || ldw13 < d.H || lddx < d.H)) return MOE_ERR_ARG;
  if (dw13 && (x == nullptr || ldx < d.H)) return MOE_ERR_ARG;
  if (dw2 && h == nullptr) return MOE_ERR_ARG;
  int32_t* err = static_cast<int32_t*>(scratch);
  void* dp = static_cast<uint8_t*>(scratch) + plan->rows_at;      // d(up, gate), in w13's order
  const long long I2 = 2LL * d.I;
  cudaError_t e = cudaSuccess;
  if (inner)                              // dh = dy W2, then through the activation
    e = product(*plan, FfGemm{w2, 1, ldw2, 0, dy, lddy, 1, d.I, M, d.H, dp, I2, const_cast<float*>(pre), err}, kFfGrad, st);
  if (dx && e == cudaSuccess)             // dx = d(up, gate) W13
    e = product(*plan, FfGemm{w13, 1, ldw13, 0, dp, I2, 1, d.H, M, (int)I2, dx, lddx, nullptr, err}, kFfStore, st);
  if (dw13 && e == cudaSuccess)           // dW13 = d(up, gate)^T x
    e = product(*plan, FfGemm{x, 1, ldx, 0, dp, 1, I2, d.H, (int)I2, M, dw13, lddw13, nullptr, err}, kFfStore, st);
  if (dw2 && e == cudaSuccess)            // dW2 = dy^T h
    e = product(*plan, FfGemm{h, 1, d.I, 0, dy, 1, lddy, d.I, d.H, M, dw2, lddw2, nullptr, err}, kFfStore, st);
  return status(e);
}

moe_status moe_ff_get_device_error(const moe_ff_t* plan, void* scratch, void* stream, int* code) {
  if (plan == nullptr || scratch == nullptr || code == nullptr) return MOE_ERR_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int32_t word = 0;
  cudaError_t e = cudaMemcpyAsync(&word, scratch, sizeof(word), cudaMemcpyDeviceToHost, st);
  // with the word the tickets, which a call that gave up may have left anywhere
  if (e == cudaSuccess) e = cudaMemsetAsync(scratch, 0, kGtPartAt, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return status(e);
  *code = word;
  if (word & kErrTimeout) return MOE_ERR_TIMEOUT;
  return word ? MOE_ERR_DEVICE : MOE_OK;
}

}  // extern "C"
