// api_fp8.cu - host side of the 8-bit products with block scales and of the quantisation to that form:
// argument checks and launches.
#include <cmath>
#include <new>

#include "fp8.cuh"
#include "../../include/moe_gb300.h"

namespace moe {
// api.cu: records the error for moe_last_cuda_error
int report_cuda(cudaError_t e);
// fp8_quant.cu
cudaError_t launch_fp8_quant(const void* x, int dtype, long long ldx, int E, int rows, int K, bool tiles,
                             uint8_t* q, long long ldq, float* scale, long long lds, cudaStream_t st);
// gemm_fp8_simt.cu
cudaError_t launch_fp8_simt(const GroupedDims& d, const Fp8Call& f, cudaStream_t st);
// gemv_fp8.cu
cudaError_t fp8_gemv_takes(const GroupedDims& d, const Fp8Call& f, bool* takes);
cudaError_t launch_fp8_gemv(const GroupedDims& d, const Fp8Call& f, cudaStream_t st);
// gemm_fp8_tc.cu
size_t fp8_tc_part_bytes(int S, int E);
bool fp8_tc_addressable(const GroupedDims& d, const Fp8Call& f);
cudaError_t launch_fp8_tc(const GroupedDims& d, const Fp8Call& f, float* part, int32_t* tickets,
                          cudaStream_t st);
}  // namespace moe

using namespace moe;

struct moe_fp8_s {
  GroupedDims d;
  size_t bytes;                           // of the scratch buffer
};

namespace {
moe_status status(cudaError_t e) { return static_cast<moe_status>(report_cuda(e)); }
}  // namespace

extern "C" {

moe_status moe_fp8_quant(const void* x, int dtype, long long ldx, int E, int rows, int K, int form,
                         uint8_t* q, long long ldq, float* scale, long long lds, void* stream) {
  if (dtype < MOE_DTYPE_BF16 || dtype > MOE_DTYPE_F32) return MOE_ERR_UNSUPPORTED;
  if (form != MOE_FP8_ROWS && form != MOE_FP8_TILES) return MOE_ERR_ARG;
  if (E < 0 || rows < 0) return MOE_ERR_ARG;
  if (K < 1 || K > (1 << 24) || (form == MOE_FP8_ROWS && E != 1)) return MOE_ERR_SHAPE;
  if ((long long)E * rows > 0x7FFFFFFFLL ||
      (form == MOE_FP8_TILES && (long long)E * fp8_blocks(rows) * fp8_blocks(K) > 0x7FFFFFFFLL))
    return MOE_ERR_SHAPE;
  if (E == 0 || rows == 0) return MOE_OK;
  if (x == nullptr || q == nullptr || scale == nullptr) return MOE_ERR_ARG;
  if (ldx < K || ldq < K || lds < fp8_blocks(K)) return MOE_ERR_ARG;
  return status(launch_fp8_quant(x, dtype, ldx, E, rows, K, form == MOE_FP8_TILES, q, ldq, scale, lds,
                                 static_cast<cudaStream_t>(stream)));
}

moe_status moe_fp8_plan(int E, int N, int K, int dtype, int act, int layout, float limit, float alpha,
                        float beta, int max_rows, moe_fp8_t** out) {
  if (out == nullptr) return MOE_ERR_ARG;
  *out = nullptr;
  if ((dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16) || (act != MOE_ACT_NONE && act != MOE_ACT_SWIGLU))
    return MOE_ERR_UNSUPPORTED;
  if (layout != MOE_W13_UP_GATE && layout != MOE_W13_GATE_UP) return MOE_ERR_ARG;
  if (std::isnan(limit) || limit <= 0.f || !std::isfinite(alpha) || !std::isfinite(beta))
    return MOE_ERR_ARG;
  if (E < 1 || E > 1024 || N < 1 || N > (1 << 22) || K < 1 || max_rows < 0) return MOE_ERR_SHAPE;
  if (act == MOE_ACT_SWIGLU && N % 2 != 0) return MOE_ERR_SHAPE;
  if ((long long)N * K >= (1LL << 40) || (long long)E * N > 0x7FFFFFFFLL || K > (1 << 24) ||
      max_rows > (1 << 30) || ((long long)max_rows / 32 + E) * cdiv(N, 128) > 0x7FFFFFFFLL)
    return MOE_ERR_SHAPE;
  moe_fp8_s* g = new (std::nothrow) moe_fp8_s();
  if (g == nullptr) return MOE_ERR_ARG;
  g->d = GroupedDims{E, N, K, dtype, act, layout, max_rows, limit, alpha, beta, 0};
  g->bytes = kGtPartAt + fp8_tc_part_bytes(max_rows, E);
  *out = g;
  return MOE_OK;
}

moe_status moe_fp8_set_wait_probe(moe_fp8_t* plan, unsigned long long ns) {
  if (plan == nullptr || ns > 1000000000ull) return MOE_ERR_ARG;
  plan->d.probe_ns = ns;
  return MOE_OK;
}

void moe_destroy_fp8(moe_fp8_t* plan) { delete plan; }

moe_status moe_fp8_scratch_bytes(const moe_fp8_t* plan, size_t* bytes) {
  if (plan == nullptr || bytes == nullptr) return MOE_ERR_ARG;
  *bytes = plan->bytes;
  return MOE_OK;
}

moe_status moe_fp8_run(const moe_fp8_t* plan, void* scratch, size_t scratch_bytes, const uint8_t* x,
                       long long ldx, int x_rows, const float* x_scale, long long ldxs, const uint8_t* w,
                       long long ldw, const float* w_scale, const int32_t* offsets, const int32_t* perm,
                       int topk, void* out, long long ldo, int S, void* stream) {
  if (plan == nullptr || S < 0 || x_rows < 0) return MOE_ERR_ARG;
  const GroupedDims& d = plan->d;
  if (S > d.max_rows) return MOE_ERR_CAPACITY;
  if (offsets == nullptr && d.E != 1) return MOE_ERR_ARG;
  if (S == 0) return MOE_OK;
  if (scratch == nullptr || scratch_bytes < plan->bytes ||
      (reinterpret_cast<uintptr_t>(scratch) & 255) != 0)
    return MOE_ERR_ARG;
  if (x == nullptr || x_scale == nullptr || w == nullptr || w_scale == nullptr || out == nullptr)
    return MOE_ERR_ARG;
  if (ldx < d.K || ldxs < fp8_blocks(d.K) || ldw < d.K || ldo < grouped_cols(d)) return MOE_ERR_ARG;
  if (perm != nullptr ? (topk < 1 || x_rows < 1) : x_rows < S) return MOE_ERR_ARG;
  const Fp8Call f{{x, ldx, x_rows, w, ldw, offsets, perm, topk, out, ldo, S, static_cast<int32_t*>(scratch)},
                  x_scale, ldxs, w_scale};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!fp8_tc_addressable(d, f)) return status(launch_fp8_simt(d, f, st));
  bool few = false;
  const cudaError_t e = fp8_gemv_takes(d, f, &few);
  if (e != cudaSuccess) return status(e);
  if (few) return status(launch_fp8_gemv(d, f, st));
  uint8_t* base = static_cast<uint8_t*>(scratch);
  return status(launch_fp8_tc(d, f, reinterpret_cast<float*>(base + kGtPartAt),
                              reinterpret_cast<int32_t*>(base + kGtTicketsAt), st));
}

moe_status moe_fp8_get_device_error(const moe_fp8_t* plan, void* scratch, void* stream, int* code) {
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
