// api_block.cu - host side of the 16-bit block's entry points (router, grouping, grouped
// products, norms): argument checks and launches.
#include <cmath>
#include <new>

#include "grouped.cuh"
#include "../../include/moe_gb300.h"

namespace moe {
// api.cu: records the error for moe_last_cuda_error
int report_cuda(cudaError_t e);
// block_route.cu
cudaError_t launch_router(const void* logits, int dtype, long long ld, const float* bias, int M,
                          int E, int topk, int score, int n_group, int topk_group, int renorm,
                          float scale, int32_t* ids, float* weights, cudaStream_t st);
cudaError_t launch_group(const int32_t* ids, int S, int E, int first, int32_t* offsets,
                         int32_t* perm, int32_t* slot_of, cudaStream_t st);
// block_norm.cu
cudaError_t launch_block_norm(const moe_norm_args& a, bool vec, cudaStream_t st);
cudaError_t norm_device_error(int* code, cudaStream_t st);
void set_norm_probe(unsigned long long ns);
// gemm_grouped_simt.cu
cudaError_t launch_grouped_simt(const GroupedDims& d, const GroupedCall& c, cudaStream_t st);
// gemm_grouped_tc.cu
size_t grouped_tc_part_bytes(int S, int E);
bool grouped_tc_addressable(const GroupedDims& d, const GroupedCall& c);
cudaError_t launch_grouped_tc(const GroupedDims& d, const GroupedCall& c, float* part,
                              int32_t* tickets, cudaStream_t st);
}  // namespace moe

using namespace moe;

struct moe_grouped_s {
  GroupedDims d;
  size_t bytes;                           // of the scratch buffer
};

namespace {

moe_status status(cudaError_t e) { return static_cast<moe_status>(report_cuda(e)); }

bool dtype16(int d) { return d == MOE_DTYPE_BF16 || d == MOE_DTYPE_F16; }

}  // namespace

extern "C" {

moe_status moe_router(const void* logits, int dtype, long long ld_logits, const float* bias, int M,
                      int E, int topk, int score, int n_group, int topk_group, int renormalize,
                      float scale, int32_t* topk_ids, float* topk_weights, void* stream) {
  if (M < 0 || dtype < MOE_DTYPE_BF16 || dtype > MOE_DTYPE_F32) return MOE_ERR_ARG;
  if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) return MOE_ERR_ARG;
  if (E < 1 || E > 1024 || topk < 1 || topk > 32 || ld_logits < E) return MOE_ERR_SHAPE;
  if (n_group < 1 || n_group > 32 || E % n_group != 0 || topk_group < 1 || topk_group > n_group)
    return MOE_ERR_SHAPE;
  if (topk > topk_group * (E / n_group)) return MOE_ERR_SHAPE;
  if (bias != nullptr && score == MOE_SCORE_SOFTMAX) return MOE_ERR_UNSUPPORTED;
  if (M == 0) return MOE_OK;
  if (logits == nullptr || topk_ids == nullptr || topk_weights == nullptr) return MOE_ERR_ARG;
  return status(launch_router(logits, dtype, ld_logits, bias, M, E, topk, score, n_group,
                              topk_group, renormalize != 0, scale, topk_ids, topk_weights,
                              static_cast<cudaStream_t>(stream)));
}

moe_status moe_group(const int32_t* topk_ids, int M, int topk, int E, int first_expert,
                     int32_t* offsets, int32_t* perm, int32_t* slot_of, void* stream) {
  if (M < 0 || first_expert < 0 || offsets == nullptr) return MOE_ERR_ARG;
  if (E < 1 || E > 1024 || topk < 1 || (long long)M * topk > (1LL << 30)) return MOE_ERR_SHAPE;
  if ((long long)first_expert + E > 0x7FFFFFFFLL) return MOE_ERR_ARG;
  if (M > 0 && (topk_ids == nullptr || perm == nullptr || slot_of == nullptr)) return MOE_ERR_ARG;
  return status(launch_group(topk_ids, M * topk, E, first_expert, offsets, perm, slot_of,
                             static_cast<cudaStream_t>(stream)));
}

moe_status moe_grouped_plan(int E, int N, int K, int dtype, int act, int layout, float limit,
                            float alpha, float beta, int max_rows, moe_grouped_t** out) {
  if (out == nullptr) return MOE_ERR_ARG;
  *out = nullptr;
  if (!dtype16(dtype) || (act != MOE_ACT_NONE && act != MOE_ACT_SWIGLU)) return MOE_ERR_UNSUPPORTED;
  if (layout != MOE_W13_UP_GATE && layout != MOE_W13_GATE_UP) return MOE_ERR_ARG;
  if (std::isnan(limit) || limit <= 0.f || !std::isfinite(alpha) || !std::isfinite(beta))
    return MOE_ERR_ARG;
  if (E < 1 || E > 1024 || N < 1 || N > (1 << 22) || K < 1 || max_rows < 0) return MOE_ERR_SHAPE;
  if (act == MOE_ACT_SWIGLU && N % 2 != 0) return MOE_ERR_SHAPE;
  if ((long long)N * K >= (1LL << 40) || (long long)E * N > 0x7FFFFFFFLL || K > (1 << 24) ||
      max_rows > (1 << 30) || ((long long)max_rows / 32 + E) * cdiv(N, 128) > 0x7FFFFFFFLL)
    return MOE_ERR_SHAPE;
  moe_grouped_s* g = new (std::nothrow) moe_grouped_s();
  if (g == nullptr) return MOE_ERR_ARG;
  g->d = GroupedDims{E, N, K, dtype, act, layout, max_rows, limit, alpha, beta, 0};
  g->bytes = kGtPartAt + grouped_tc_part_bytes(max_rows, E);
  *out = g;
  return MOE_OK;
}

moe_status moe_grouped_set_wait_probe(moe_grouped_t* plan, unsigned long long ns) {
  if (plan == nullptr || ns > 1000000000ull) return MOE_ERR_ARG;
  plan->d.probe_ns = ns;
  return MOE_OK;
}

void moe_destroy_grouped(moe_grouped_t* plan) { delete plan; }

moe_status moe_grouped_scratch_bytes(const moe_grouped_t* plan, size_t* bytes) {
  if (plan == nullptr || bytes == nullptr) return MOE_ERR_ARG;
  *bytes = plan->bytes;
  return MOE_OK;
}

moe_status moe_grouped_run(const moe_grouped_t* plan, void* scratch, size_t scratch_bytes,
                           const void* x, long long ldx, int x_rows, const void* w, long long ldw,
                           const int32_t* offsets, const int32_t* perm, int topk, void* out,
                           long long ldo, int S, void* stream) {
  if (plan == nullptr || S < 0 || x_rows < 0) return MOE_ERR_ARG;
  const GroupedDims& d = plan->d;
  if (S > d.max_rows) return MOE_ERR_CAPACITY;
  if (S == 0) return MOE_OK;
  if (scratch == nullptr || scratch_bytes < plan->bytes ||
      (reinterpret_cast<uintptr_t>(scratch) & 255) != 0)
    return MOE_ERR_ARG;
  if (x == nullptr || w == nullptr || offsets == nullptr || out == nullptr) return MOE_ERR_ARG;
  if (ldx < d.K || ldw < d.K || ldo < grouped_cols(d)) return MOE_ERR_ARG;
  if (perm != nullptr ? (topk < 1 || x_rows < 1) : x_rows < S) return MOE_ERR_ARG;
  GroupedCall c{x, ldx, x_rows, w, ldw, offsets, perm, topk, out, ldo, S,
                static_cast<int32_t*>(scratch)};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!grouped_tc_addressable(d, c)) return status(launch_grouped_simt(d, c, st));
  uint8_t* base = static_cast<uint8_t*>(scratch);
  return status(launch_grouped_tc(d, c, reinterpret_cast<float*>(base + kGtPartAt),
                                  reinterpret_cast<int32_t*>(base + kGtTicketsAt), st));
}

moe_status moe_grouped_get_device_error(const moe_grouped_t* plan, void* scratch, void* stream,
                                        int* code) {
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

moe_status moe_block_norm(const moe_norm_args* a, void* stream) {
  if (a == nullptr || a->M < 0) return MOE_ERR_ARG;
  if (a->H < 1 || a->H > 32768) return MOE_ERR_SHAPE;
  if (!dtype16(a->dtype)) return MOE_ERR_UNSUPPORTED;
  if (a->residual_dtype != a->dtype && a->residual_dtype != MOE_DTYPE_F32) return MOE_ERR_UNSUPPORTED;
  if (a->weight_dtype != a->dtype && a->weight_dtype != MOE_DTYPE_F32) return MOE_ERR_UNSUPPORTED;
  if (a->kind != MOE_NORM_RMS && a->kind != MOE_NORM_LAYER) return MOE_ERR_ARG;
  if (!(a->eps >= 0.f) || std::isinf(a->eps)) return MOE_ERR_ARG;
  if (a->M == 0) return MOE_OK;           // addresses of nothing say nothing
  if (a->gate != nullptr && a->gate_col != 0 && a->gate_col != 1) return MOE_ERR_ARG;
  if (a->rows == nullptr &&
      (a->slot_of || a->shared || a->post_weight || a->gate || a->residual_out))
    return MOE_ERR_ARG;
  if (a->slot_of != nullptr ? (a->topk_weights == nullptr || a->topk < 1 || a->n_rows < 0)
                            : (a->topk_weights != nullptr || a->shared != nullptr))
    return MOE_ERR_ARG;
  if ((a->post_bias && !a->post_weight) || (a->pre_bias && !a->pre_weight)) return MOE_ERR_ARG;
  if (a->residual_out == nullptr && a->pre_weight == nullptr) return MOE_ERR_ARG;
  if ((a->pre_weight != nullptr) != (a->out != nullptr)) return MOE_ERR_ARG;
  if (a->residual == nullptr) return MOE_ERR_ARG;
  const long long H = a->H;
  if (a->ld_residual < H || (a->rows && a->ld_rows < H) || (a->shared && a->ld_shared < H) ||
      (a->residual_out && a->ld_residual_out < H) || (a->out && a->ld_out < H))
    return MOE_ERR_ARG;
  // whole vectors of eight elements: 16-byte bases (32 where the elements are fp32), row strides
  // of whole vectors (a gate vector per row too)
  const auto rows8 = [](const void* p, long long ld, int dtype) {
    const uintptr_t mask = dtype == MOE_DTYPE_F32 ? 31 : 15;
    return !p || ((reinterpret_cast<uintptr_t>(p) & mask) == 0 && ld % 8 == 0);
  };
  const int rt = a->residual_dtype, wt = a->weight_dtype, t = a->dtype;
  const bool vec = H % 8 == 0 && rows8(a->residual, a->ld_residual, rt) &&
                   rows8(a->rows, a->ld_rows, t) && rows8(a->shared, a->ld_shared, t) &&
                   rows8(a->residual_out, a->ld_residual_out, rt) && rows8(a->out, a->ld_out, t) &&
                   rows8(a->post_weight, 0, wt) && rows8(a->post_bias, 0, wt) &&
                   rows8(a->pre_weight, 0, wt) && rows8(a->pre_bias, 0, wt) &&
                   (a->gate == nullptr || a->gate_col == 0 || rows8(a->gate, a->gate_row, wt));
  return status(launch_block_norm(*a, vec, static_cast<cudaStream_t>(stream)));
}

moe_status moe_block_norm_set_wait_probe(unsigned long long ns) {
  if (ns > 1000000000ull) return MOE_ERR_ARG;
  set_norm_probe(ns);
  return MOE_OK;
}

moe_status moe_block_norm_get_device_error(void* stream, int* code) {
  if (code == nullptr) return MOE_ERR_ARG;
  const cudaError_t e = norm_device_error(code, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return status(e);
  return *code ? MOE_ERR_TIMEOUT : MOE_OK;
}

}  // extern "C"
