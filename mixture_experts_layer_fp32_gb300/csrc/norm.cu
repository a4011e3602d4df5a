// Layer norm and RMS norm of z = residual + dropout(x), their backward pass
// with the reduction of the parameters' gradients, and the dropout with the
// residual sum on its own.
#include "common.cuh"
#include "philox.cuh"

namespace moe {
namespace {

__device__ __forceinline__ float load1(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float load1(const __nv_bfloat16* p, int64_t i) {
  return __bfloat162float(p[i]);
}
__device__ __forceinline__ void store1(float* p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, int64_t i, float v) {
  p[i] = __float2bfloat16_rn(v);
}
__device__ __forceinline__ float param1(const void* p, int is_bf16, int64_t i) {
  return is_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i])
                 : static_cast<const float*>(p)[i];
}

struct NormArgs {
  int64_t rows;
  int hidden, rms, param_bf16;
  float eps;
  Dropout drop;
  const uint64_t* rng;
};

__device__ __forceinline__ float drop1(const Dropout& d, const Philox& g, int64_t i, float v) {
  const uint4 w = philox_words(g, static_cast<uint64_t>(i) >> 2);
  const uint32_t j = static_cast<uint32_t>(i) & 3;
  const uint32_t u = j == 0 ? w.x : j == 1 ? w.y : j == 2 ? w.z : w.w;
  return u > d.limit ? v * d.scale : 0.f;
}

constexpr int kRowThreads = 256;

// the block's sums of a and b, in every thread; the order of the sums is fixed
__device__ __forceinline__ float2 block_sum(float a, float b, float2* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(~0u, a, o);
    b += __shfl_xor_sync(~0u, b, o);
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  float2 t = make_float2(0.f, 0.f);
  for (unsigned w = 0; w < blockDim.x / 32; ++w) {
    t.x += red[w].x;
    t.y += red[w].y;
  }
  return t;
}

// One block to a row, any width: the row is read once for the mean, once for
// the variance and once for the output.
template <typename T>
__global__ void __launch_bounds__(kRowThreads)
    norm_wide_kernel(NormArgs a, const T* x, const T* res, const void* weight, const void* bias,
                     T* z, T* y, float* mean, float* rstd) {
  __shared__ float2 red[kRowThreads / 32];
  const int H = a.hidden;
  const Philox g = a.drop.on ? philox_of(a.rng) : Philox{};
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const int64_t base = r * H;
    auto value = [&](int c) {
      float v = load1(x, base + c);
      if (a.drop.on) v = drop1(a.drop, g, base + c, v);
      return res ? load1(res, base + c) + v : v;
    };
    float m = 0.f;
    if (!a.rms) {
      float sum = 0.f;
      for (int c = threadIdx.x; c < H; c += kRowThreads) sum += value(c);
      m = block_sum(sum, 0.f, red).x / H;
    }
    float sq = 0.f;
    for (int c = threadIdx.x; c < H; c += kRowThreads) {
      const float d = value(c) - m;
      sq += d * d;
    }
    const float rs = 1.f / sqrtf(block_sum(sq, 0.f, red).x / H + a.eps);
    for (int c = threadIdx.x; c < H; c += kRowThreads) {
      const float v = value(c);
      float o = (v - m) * rs;
      if (weight) o *= param1(weight, a.param_bf16, c);
      if (bias) o += param1(bias, a.param_bf16, c);
      if (z) store1(z, base + c, v);
      store1(y, base + c, o);
    }
    if (threadIdx.x == 0) {
      if (mean && !a.rms) mean[r] = m;
      if (rstd) rstd[r] = rs;
    }
  }
}

// Block b takes the rows b, b + gridDim, ...; its sums for dweight and dbias
// stay in its own part[b], which norm_param_grads_kernel adds up.
template <typename T>
__global__ void __launch_bounds__(kRowThreads)
    norm_backward_wide_kernel(NormArgs a, const T* dy, const T* z, const void* weight,
                              const float* mean, const float* rstd, const T* dz, T* dx,
                              T* dbranch, float* part) {
  __shared__ float2 red[kRowThreads / 32];
  const int H = a.hidden;
  const Philox g = a.drop.on ? philox_of(a.rng) : Philox{};
  float* pw = part + static_cast<int64_t>(blockIdx.x) * 2 * H;
  float* pb = pw + H;
  bool first = true;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const int64_t base = r * H;
    const float m = a.rms ? 0.f : mean[r], rs = rstd[r];
    float s1 = 0.f, s2 = 0.f;
    for (int c = threadIdx.x; c < H; c += kRowThreads) {
      float d = load1(dy, base + c);
      if (weight) d *= param1(weight, a.param_bf16, c);
      s1 += d;
      s2 += d * (load1(z, base + c) - m) * rs;
    }
    const float2 t = block_sum(s1, s2, red);
    const float c1 = a.rms ? 0.f : t.x / H, c2 = t.y / H;
    for (int c = threadIdx.x; c < H; c += kRowThreads) {
      const float d = load1(dy, base + c), xh = (load1(z, base + c) - m) * rs;
      const float gw = weight ? d * param1(weight, a.param_bf16, c) : d;
      float o = rs * (gw - c1 - xh * c2);
      if (dz) o += load1(dz, base + c);
      store1(dx, base + c, o);
      if (dbranch)
        store1(dbranch, base + c, a.drop.on ? drop1(a.drop, g, base + c, o) : o);
      pw[c] = (first ? 0.f : pw[c]) + d * xh;
      pb[c] = (first ? 0.f : pb[c]) + d;
    }
    first = false;
  }
}

// dweight and dbias: the sums over the blocks' parts, in their order
__global__ void norm_param_grads_kernel(int parts, int H, const float* part, float* dweight,
                                        float* dbias) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= H) return;
  float w = 0.f, b = 0.f;
  for (int p = 0; p < parts; ++p) {
    w += part[static_cast<int64_t>(p) * 2 * H + c];
    b += part[static_cast<int64_t>(p) * 2 * H + H + c];
  }
  if (dweight) dweight[c] = w;
  if (dbias) dbias[c] = b;
}

template <typename T>
__global__ void dropout_add_kernel(int64_t n, Dropout d, const uint64_t* rng, const T* x,
                                   const T* res, T* y) {
  const Philox g = d.on ? philox_of(rng) : Philox{};
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += step) {
    float v = load1(x, i);
    if (d.on) v = drop1(d, g, i, v);
    store1(y, i, res ? load1(res, i) + v : v);
  }
}

NormArgs args_of(const moe_norm_config& c, const uint64_t* rng) {
  NormArgs a;
  a.rows = c.rows;
  a.hidden = c.hidden;
  a.rms = c.kind == MOE_NORM_RMS;
  a.param_bf16 = c.param_dtype == MOE_BF16;
  a.eps = c.eps;
  a.drop = dropout_of(c.dropout);
  a.rng = rng;
  return a;
}

template <typename T>
cudaError_t norm_typed(const moe_norm_config& c, const void* x, const void* residual,
                       const uint64_t* rng, const void* weight, const void* bias, void* z, void* y,
                       float* mean, float* rstd, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(c.rows < 65536 ? c.rows : 65536);
  norm_wide_kernel<T><<<grid, kRowThreads, 0, s>>>(
      args_of(c, rng), static_cast<const T*>(x), static_cast<const T*>(residual), weight, bias,
      static_cast<T*>(z), static_cast<T*>(y), mean, rstd);
  return cudaGetLastError();
}

template <typename T>
cudaError_t norm_backward_typed(const moe_norm_config& c, const void* dy, const void* z,
                                const void* weight, const float* mean, const float* rstd,
                                const void* dz, const uint64_t* rng, void* dx, void* dbranch,
                                float* part, cudaStream_t s) {
  NormArgs a = args_of(c, rng);
  if (dbranch == nullptr) a.drop.on = 0;
  norm_backward_wide_kernel<T><<<norm_backward_ctas(c), kRowThreads, 0, s>>>(
      a, static_cast<const T*>(dy), static_cast<const T*>(z), weight, mean, rstd,
      static_cast<const T*>(dz), static_cast<T*>(dx), static_cast<T*>(dbranch), part);
  return cudaGetLastError();
}

}  // namespace

int norm_backward_ctas(const moe_norm_config& c) {
  constexpr int kMost = 608;
  return static_cast<int>(c.rows < kMost ? c.rows : kMost);
}

cudaError_t launch_norm(const moe_norm_config& c, const void* x, const void* residual,
                        const uint64_t* rng, const void* weight, const void* bias, void* z,
                        void* y, float* mean, float* rstd, cudaStream_t s) {
  if (c.rows == 0) return cudaSuccess;
  return c.dtype == MOE_F32
             ? norm_typed<float>(c, x, residual, rng, weight, bias, z, y, mean, rstd, s)
             : norm_typed<__nv_bfloat16>(c, x, residual, rng, weight, bias, z, y, mean, rstd, s);
}

cudaError_t launch_norm_backward(const moe_norm_config& c, const void* dy, const void* z,
                                 const void* weight, const float* mean, const float* rstd,
                                 const void* dz, const uint64_t* rng, void* dx, void* dbranch,
                                 float* dweight, float* dbias, float* part, cudaStream_t s) {
  if (c.rows > 0) {
    const cudaError_t st =
        c.dtype == MOE_F32
            ? norm_backward_typed<float>(c, dy, z, weight, mean, rstd, dz, rng, dx, dbranch, part,
                                         s)
            : norm_backward_typed<__nv_bfloat16>(c, dy, z, weight, mean, rstd, dz, rng, dx,
                                                 dbranch, part, s);
    if (st != cudaSuccess) return st;
  }
  if (!dweight && !dbias) return cudaSuccess;
  norm_param_grads_kernel<<<(c.hidden + 255) / 256, 256, 0, s>>>(norm_backward_ctas(c), c.hidden,
                                                                 part, dweight, dbias);
  return cudaGetLastError();
}

cudaError_t launch_dropout_add(int64_t n, int dtype, double p, const uint64_t* rng, const void* x,
                               const void* residual, void* y, cudaStream_t s) {
  if (n == 0) return cudaSuccess;
  const Dropout d = dropout_of(p);
  const int64_t blocks = (n + 255) / 256;
  const unsigned grid = static_cast<unsigned>(blocks < 8192 ? blocks : 8192);
  if (dtype == MOE_F32)
    dropout_add_kernel<float><<<grid, 256, 0, s>>>(n, d, rng, static_cast<const float*>(x),
                                                   static_cast<const float*>(residual),
                                                   static_cast<float*>(y));
  else
    dropout_add_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(
        n, d, rng, static_cast<const __nv_bfloat16*>(x),
        static_cast<const __nv_bfloat16*>(residual), static_cast<__nv_bfloat16*>(y));
  return cudaGetLastError();
}

}  // namespace moe
