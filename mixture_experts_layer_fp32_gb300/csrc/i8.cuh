// 8-bit integer products: what the narrow and the wide kernel share.
#pragma once

#include "common.cuh"
#include "sm100_ptx.cuh"

namespace moe {
namespace i8 {

// y[m, n] = (sum_k x[m, k] W[n, k]) x_scale[m] w_scale[n] + bias[n]
struct Args {
  int rows, N, K;
  const void* x;          // narrow: codes, or values that it quantises
  const float* x_scale;
  const int8_t* W;
  const float *w_scale, *bias;
  void* y;
  int out_f32;
  int splits;             // of K over blocks; > 1: whole sums into part
  int32_t* part;          // [split][rows][N]
  int* err;
};

// The sum is whole; it and the products with the scales are rounded to fp32, one
// rounding each, and the result once more to bf16.
__device__ __forceinline__ float scaled(int sum, float x_scale, float w_scale, float bias) {
  return __fmaf_rn(static_cast<float>(sum) * x_scale, w_scale, bias);
}

// More rows (i8_wide.cu): x as fp16 numbers, laid out by the launch before; the weights
// are read before that has ended.
int wide_splits(int64_t rows, int N, int K);
cudaError_t launch_wide(const Args& a, const __half* x, cudaStream_t s);

}  // namespace i8
}  // namespace moe
