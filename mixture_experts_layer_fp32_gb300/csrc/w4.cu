// Products with 4-bit weights (group scales) for few rows, and the routed
// SwiGLU experts built from them.
#include "w4.cuh"

namespace moe {
namespace {

// One warp: x[0..K) (a function of k) times row `row` of W.
template <typename X>
__device__ float dot_row(const W4& W, int64_t row, int K, int group, int lane, X x) {
  const int nb = w4_blocks(K), ng = K / group;
  const uint32_t* codes = reinterpret_cast<const uint32_t*>(W.codes) + row * nb * 16;
  float sum = 0.f;
  for (int w = lane; w < nb * 16; w += 32) {
    const int k = (w >> 4) * 128 + (w & 3) * 32 + ((w >> 2) & 3) * 8;
    if (k >= K) continue;
    const int64_t gi = row * ng + k / group;
    const float z = W.zeros ? static_cast<float>(W.zeros[gi]) : 8.f;
    const uint32_t v = codes[w];
    float part = 0.f;
    for (int i = 0; i < 8; ++i) {
      const int nib = i / 2 + 4 * (i & 1);
      part += (static_cast<float>((v >> (4 * nib)) & 15) - z) * x(k + i);
    }
    sum += part * __bfloat162float(W.scales[gi]);
  }
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
  return sum;
}

__global__ void linear_kernel(int64_t rows, int N, int K, int group, const __nv_bfloat16* x, W4 W,
                              void* y, int y_dtype) {
  const int lane = threadIdx.x & 31;
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * blockDim.x / 32;
  for (int64_t i = warp; i < rows * N; i += warps) {
    const int64_t r = i / N, n = i % N;
    const float v = dot_row(W, n, K, group, lane,
                            [&](int k) { return __bfloat162float(x[r * K + k]); });
    if (lane == 0) {
      if (y_dtype == MOE_F32) static_cast<float*>(y)[i] = v;
      else static_cast<__nv_bfloat16*>(y)[i] = __float2bfloat16_rn(v);
    }
  }
}

// hidden values of every pair, fp32
__global__ void experts_fc1_kernel(int P, int h, int f, int E, int k, int group,
                                   const __nv_bfloat16* x, const int32_t* idx,
                                   const uint8_t* keep, W4 W1, W4 W3, float* hid, int* err) {
  const int lane = threadIdx.x & 31;
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * blockDim.x / 32;
  for (int64_t i = warp; i < static_cast<int64_t>(P) * f; i += warps) {
    const int p = static_cast<int>(i / f), n = static_cast<int>(i % f);
    if (keep && !keep[p]) continue;
    const int e = idx[p];
    if (e < 0 || e >= E) {
      if (lane == 0) report_error(err, DEV_ERR_INDEX, e);
      continue;
    }
    const __nv_bfloat16* xt = x + static_cast<int64_t>(p / k) * h;
    auto get = [&](int c) { return __bfloat162float(xt[c]); };
    const float a = dot_row(W1, static_cast<int64_t>(e) * f + n, h, group, lane, get);
    const float b = dot_row(W3, static_cast<int64_t>(e) * f + n, h, group, lane, get);
    if (lane == 0) hid[i] = a / (1.f + expf(-a)) * b;
  }
}

__global__ void experts_fc2_kernel(int T, int h, int f, int E, int k, int group,
                                   const int32_t* idx, const float* prob, const uint8_t* keep,
                                   W4 W2, const float* hid, __nv_bfloat16* y) {
  const int lane = threadIdx.x & 31;
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * blockDim.x / 32;
  for (int64_t i = warp; i < static_cast<int64_t>(T) * h; i += warps) {
    const int t = static_cast<int>(i / h), n = static_cast<int>(i % h);
    float sum = 0.f;
    for (int j = 0; j < k; ++j) {
      const int p = t * k + j, e = idx[p];
      if ((keep && !keep[p]) || e < 0 || e >= E) continue;
      const float* hp = hid + static_cast<int64_t>(p) * f;
      sum += prob[p] * dot_row(W2, static_cast<int64_t>(e) * h + n, f, group, lane,
                               [&](int c) { return hp[c]; });
    }
    if (lane == 0) y[i] = __float2bfloat16_rn(sum);
  }
}

}  // namespace

size_t w4_linear_scratch(int64_t, int, int) { return 0; }

cudaError_t launch_w4_linear(int64_t rows, int N, int K, int group, const void* x, const W4& W,
                             void* y, int y_dtype, void*, cudaStream_t s) {
  linear_kernel<<<152 * 8, 256, 0, s>>>(rows, N, K, group, static_cast<const __nv_bfloat16*>(x),
                                        W, y, y_dtype);
  return cudaGetLastError();
}

size_t w4_experts_scratch(int T, int, int, int k, int f) {
  return static_cast<size_t>(T) * k * f * 4;
}

cudaError_t launch_w4_experts(int T, int h, int E, int k, int f, int group, const void* x,
                              const int32_t* topk_idx, const float* topk_prob,
                              const uint8_t* keep, const W4& W1, const W4& W3, const W4& W2,
                              void* y, void* scratch, int* err, cudaStream_t s) {
  float* hid = static_cast<float*>(scratch);
  experts_fc1_kernel<<<152 * 8, 256, 0, s>>>(T * k, h, f, E, k, group,
                                             static_cast<const __nv_bfloat16*>(x), topk_idx, keep,
                                             W1, W3, hid, err);
  experts_fc2_kernel<<<152 * 8, 256, 0, s>>>(T, h, f, E, k, group, topk_idx, topk_prob, keep, W2,
                                             hid, static_cast<__nv_bfloat16*>(y));
  return cudaGetLastError();
}

}  // namespace moe
