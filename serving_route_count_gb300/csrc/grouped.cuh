// grouped.cuh - parameters of the products grouped by expert (moe_grouped_run) that the kernels
// and the C ABI share.
#pragma once

#include "moe_common.cuh"

namespace moe {

// Scratch buffer of a plan: the error word, the tickets of the units that are cut along K ([pairs][2
// CTAs][2 accumulators]), then the partial sums.  What lies before those is zero between calls.
constexpr int kGtMaxPairs = 80;          // CTA pairs that the buffer serves
constexpr size_t kGtTicketsAt = 256, kGtPartAt = 4096;
static_assert(kGtTicketsAt + kGtMaxPairs * 4 * sizeof(int32_t) <= kGtPartAt, "tickets");

struct GroupedDims {
  int E, N, K, dtype, act, layout, max_rows;
  float limit, alpha, beta;
  unsigned long long probe_ns;         // test hook (0: off), see moe_grouped_set_wait_probe
};

struct GroupedCall {
  const void* x;
  long long ldx;
  int x_rows;
  const void* w;
  long long ldw;
  const int32_t* offsets;
  const int32_t* perm;      // or NULL
  int topk;
  void* out;
  long long ldo;
  int S;
  int32_t* err;             // device error word of the scratch buffer
};

// Values of one output row: N, or the N / 2 of a SwiGLU.
inline int grouped_cols(const GroupedDims& d) { return d.act ? d.N / 2 : d.N; }

}  // namespace moe
