// fp8.cuh - parameters of the 8-bit products with block scales (moe_fp8_run) and of the
// quantisation to that form (moe_fp8_quant), shared by the kernels and the C ABI.
#pragma once

#include "grouped.cuh"

namespace moe {

constexpr int kFp8Block = 128;           // values of a scale along K; rows too where it is a tile's
constexpr float kFp8Max = 448.f;         // largest e4m3 value

// A product of e4m3 operands: sizes and activation as of the 16-bit grouped products (GroupedDims; dtype is
// the output's), operands as there with one byte per element, and the scales.  offsets NULL: one matrix,
// whose rows are all S positions.
struct Fp8Call {
  GroupedCall c;
  const float* xs;          // [x_rows, KB], row stride ldxs
  long long ldxs;
  const float* ws;          // [E, tall, KB]
};

inline __host__ __device__ int fp8_blocks(int n) { return cdiv(n, kFp8Block); }
// Scale rows of one weight matrix: with a SwiGLU each half has tiles of its own.
inline __host__ __device__ int fp8_tall(const GroupedDims& d) {
  return d.act ? 2 * fp8_blocks(d.N / 2) : fp8_blocks(d.N);
}
// Scale row of weight row r.
inline __host__ __device__ int fp8_scale_row(const GroupedDims& d, int r) {
  if (!d.act) return r / kFp8Block;
  const int half = d.N / 2;
  return r < half ? r / kFp8Block : fp8_blocks(half) + (r - half) / kFp8Block;
}

}  // namespace moe
