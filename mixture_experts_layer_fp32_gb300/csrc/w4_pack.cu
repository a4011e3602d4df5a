// 4-bit weights: quantisation from bf16 and packing of given codes.  Both run
// once, when a model is loaded.
#include "w4.cuh"

namespace moe {
namespace {

// One block: 32 output rows x one group of inputs of one expert, transposed
// through shared memory (W has the outputs contiguous, the codes the inputs).
constexpr int kQuantRows = 32;
__global__ void __launch_bounds__(256)
    w4_quantize_kernel(int K, int N, int group, const __nv_bfloat16* W, uint32_t* codes,
                       __nv_bfloat16* scales, uint8_t* zeros) {
  __shared__ float tile[128][kQuantRows + 1];
  __shared__ float scale[kQuantRows], zero[kQuantRows];
  const int n0 = blockIdx.x * kQuantRows, g = blockIdx.y;
  const int64_t e = blockIdx.z;
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const __nv_bfloat16* src = W + (e * K + static_cast<int64_t>(g) * group) * N + n0;
  for (int k = ty; k < group; k += 8)
    tile[k][tx] = __bfloat162float(src[static_cast<int64_t>(k) * N + tx]);
  __syncthreads();
  if (ty == 0) {
    float lo = 0.f, hi = 0.f;
    bool good = true;  // (the minimum and the maximum drop a NaN)
    for (int k = 0; k < group; ++k) {
      lo = fminf(lo, tile[k][tx]);
      hi = fmaxf(hi, tile[k][tx]);
      good &= isfinite(tile[k][tx]);
    }
    const float range = zeros ? (hi - lo) / 15.f : fmaxf(hi, -lo) / 7.f;
    const __nv_bfloat16 s16 = __float2bfloat16_rn(good ? range : __uint_as_float(0x7fffffffu));
    const float s = __bfloat162float(s16);
    float z = 8.f;
    if (zeros) z = s > 0.f ? fminf(fmaxf(rintf(-lo / s), 0.f), 15.f) : 0.f;
    scale[tx] = s;
    zero[tx] = z;
    const int64_t at = (e * N + n0 + tx) * (K / group) + g;
    scales[at] = s16;
    if (zeros) zeros[at] = static_cast<uint8_t>(z);
  }
  __syncthreads();
  const int nb = w4_blocks(K);
  for (int i = threadIdx.x; i < kQuantRows * group / 8; i += 256) {
    const int n = i / (group / 8), w = i % (group / 8);  // w: the word's place in k order
    const float s = scale[n], z = zero[n];
    uint32_t v = 0;
    for (int c = 0; c < 8; ++c) {
      const float q = s > 0.f ? rintf(tile[8 * w + c][n] / s) + z : z;
      v |= static_cast<uint32_t>(fminf(fmaxf(q, 0.f), 15.f)) << (4 * (c / 2 + 4 * (c & 1)));
    }
    const int k = g * group + 8 * w, kb = k & 127;
    codes[((e * N + n0 + n) * nb + k / 128) * 16 + ((kb >> 3) & 3) * 4 + (kb >> 5)] = v;
  }
}

__global__ void w4_pack_kernel(int64_t words, int K, const uint8_t* values, uint32_t* codes) {
  const int nb = w4_blocks(K);
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < words;
       i += step) {
    const int64_t row = i / (nb * 16);
    const int w = static_cast<int>(i % (nb * 16));
    const int k = (w >> 4) * 128 + (w & 3) * 32 + ((w >> 2) & 3) * 8;
    uint32_t v = 0;
    for (int c = 0; c < 8; ++c)
      if (k + c < K)
        v |= static_cast<uint32_t>(values[row * K + k + c] & 15) << (4 * (c / 2 + 4 * (c & 1)));
    codes[i] = v;
  }
}

}  // namespace

cudaError_t launch_w4_quantize(int E, int K, int N, int group, const void* W, uint8_t* codes,
                               void* scales, uint8_t* zeros, cudaStream_t s) {
  w4_quantize_kernel<<<dim3(N / kQuantRows, K / group, E), 256, 0, s>>>(
      K, N, group, static_cast<const __nv_bfloat16*>(W), reinterpret_cast<uint32_t*>(codes),
      static_cast<__nv_bfloat16*>(scales), zeros);
  return cudaGetLastError();
}

cudaError_t launch_w4_pack(int E, int N, int K, const uint8_t* values, uint8_t* codes,
                           cudaStream_t s) {
  const int64_t words = static_cast<int64_t>(E) * N * w4_blocks(K) * 16;
  const int64_t blocks = (words + 255) / 256;
  w4_pack_kernel<<<static_cast<unsigned>(blocks < 16384 ? blocks : 16384), 256, 0, s>>>(
      words, K, values, reinterpret_cast<uint32_t*>(codes));
  return cudaGetLastError();
}

}  // namespace moe
