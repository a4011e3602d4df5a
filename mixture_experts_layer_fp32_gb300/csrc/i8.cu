// 8-bit integers: rows to codes with a scale each, and the product for few rows.
#include <type_traits>

#include "i8.cuh"

namespace moe {
namespace i8 {
namespace {

// ------------------------------------------------------------------ quantising
// A row's scale is its largest magnitude times fp32's 1 / 127, a code the nearest whole
// number of x over the scale, ties to even.  The quotient is estimated by a product with
// the reciprocal, within 2^-15 of it (127 times two roundings of 2^-24); where that could
// lie on the other side of a half, what is left of x (exact by fma: it has few bits)
// decides whether the neighbour is nearer.  A row's values stay in registers between the
// search and the codes as far as a block holds them (kHeld 16-byte pieces a thread).
// 8192 x 4096 bf16 take 41 us (with the remainder of every value 51; the bytes 15), fp32
// 30 (47; 25): a row's load, search and store follow one another.
constexpr int kQuantThreads = 256, kHeld = 4;

template <typename T>
struct Piece {
  static constexpr int n = 16 / sizeof(T);
  T v[n];
};
__device__ __forceinline__ float as_float(float v) { return v; }
__device__ __forceinline__ float as_float(__nv_bfloat16 v) { return __bfloat162float(v); }

__device__ __forceinline__ float code_of(float x, float scale, float inverse) {
  float q = rintf(x * inverse);
  const float twice = 2.f * fmaf(-q, scale, x);
  const bool odd = static_cast<int>(q) & 1;
  if (twice > scale || (twice == scale && odd)) q += 1.f;
  else if (-twice > scale || (-twice == scale && odd)) q -= 1.f;
  return fminf(fmaxf(q, -127.f), 127.f);
}

constexpr float kWhole = 12582912.f;  // 1.5 2^23: a small number added to it is rounded

// n codes in one store: halves of a sector would be filled up from memory.
template <int n>
__device__ __forceinline__ void store_codes(int8_t* at, const float (&q)[n]) {
  char v[n];
#pragma unroll
  for (int i = 0; i < n; ++i) v[i] = static_cast<char>(__float_as_int(q[i] + kWhole) & 0xff);
  using Word = typename std::conditional<n == 8, uint2, uint32_t>::type;
  Word w;
  memcpy(&w, v, n);
  *reinterpret_cast<Word*>(at) = w;
}
template <int n>
__device__ __forceinline__ void store_codes(__half* at, const float (&q)[n]) {
  __half2 v[n / 2];
#pragma unroll
  for (int i = 0; i < n / 2; ++i) v[i] = __floats2half2_rn(q[2 * i], q[2 * i + 1]);
  using Word = typename std::conditional<n == 8, uint4, uint2>::type;
  Word w;
  memcpy(&w, v, 2 * n);
  *reinterpret_cast<Word*>(at) = w;
}

template <typename T>
__device__ __forceinline__ Piece<T> read_piece(const T* at) {
  const uint4 q = *reinterpret_cast<const uint4*>(at);
  Piece<T> p;
  memcpy(&p, &q, 16);
  return p;
}

// The largest magnitude, and whether all are numbers.
struct Top {
  float most = 0.f;
  bool good = true;
  template <typename T>
  __device__ __forceinline__ void look(const Piece<T>& p) {
#pragma unroll
    for (int i = 0; i < Piece<T>::n; ++i) {
      const float v = fabsf(as_float(p.v[i]));
      most = fmaxf(most, v);
      good &= v < INFINITY;
    }
  }
  __device__ __forceinline__ void of_warp() {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(~0u, most, o));
    good = __all_sync(~0u, good);
  }
};

struct Coder {
  float scale, up, s, inverse;
  bool some, plain;
  __device__ __forceinline__ explicit Coder(const Top& top) {
    scale = top.good ? top.most * (1.f / 127.f) : NAN;
    // no reciprocal of a scale past 2^-126 is lost to overflow
    up = scale < 0x1p-100f ? 0x1p64f : 1.f;
    some = scale > 0.f;  // neither 0 nor NaN
    plain = some && up == 1.f;
    s = scale * up;
    inverse = some ? 1.f / s : 0.f;
  }
  template <typename T, typename Code>
  __device__ __forceinline__ void put(const Piece<T>& p, Code* out) const {
    float q[Piece<T>::n];
    bool sure = plain;
#pragma unroll
    for (int j = 0; j < Piece<T>::n; ++j) {
      const float t = as_float(p.v[j]) * inverse;
      q[j] = (t + kWhole) - kWhole;
      sure &= fabsf(t - q[j]) < 0.5f - 0x1p-14f;
    }
    if (!sure)
#pragma unroll
      for (int j = 0; j < Piece<T>::n; ++j)
        q[j] = some ? code_of(as_float(p.v[j]) * up, s, inverse) : 0.f;
    store_codes(out, q);
  }
};

template <typename T, typename Code>
__global__ void __launch_bounds__(kQuantThreads)
    quantize_kernel(int K, const T* x, Code* codes, float* scales) {
  constexpr int V = Piece<T>::n;
  __shared__ float tops[kQuantThreads / 32];
  const int64_t row = blockIdx.x;
  const T* xr = x + row * K;
  Code* out = codes + row * K;
  pdl_trigger();
  Piece<T> held[kHeld];
  Top top;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int k = (i * kQuantThreads + threadIdx.x) * V;
    if (k < K) held[i] = read_piece(xr + k);
  }
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if ((i * kQuantThreads + threadIdx.x) * V < K) top.look(held[i]);
  for (int k = (kHeld * kQuantThreads + threadIdx.x) * V; k < K; k += kQuantThreads * V)
    top.look(read_piece(xr + k));
  top.of_warp();
  if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top.most;
  top.good = __syncthreads_and(top.good);
#pragma unroll
  for (int w = 0; w < kQuantThreads / 32; ++w) top.most = fmaxf(top.most, tops[w]);
  const Coder coder(top);
  if (threadIdx.x == 0) scales[row] = coder.scale;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int k = (i * kQuantThreads + threadIdx.x) * V;
    if (k < K) coder.put(held[i], out + k);
  }
  for (int k = (kHeld * kQuantThreads + threadIdx.x) * V; k < K; k += kQuantThreads * V)
    coder.put(read_piece(xr + k), out + k);
}

template <typename T, typename Code>
cudaError_t quantize(int64_t rows, int K, const void* x, Code* codes, float* scales,
                     cudaStream_t s) {
  quantize_kernel<T, Code><<<static_cast<unsigned>(rows), kQuantThreads, 0, s>>>(
      K, static_cast<const T*>(x), codes, scales);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ few rows
// Sixteen outputs to a warp, 8 NT rows of x as the columns of the integer
// instruction m16n8k32, whose sums are whole.  64 inputs of a row of W are 16 bytes to
// each of four lanes: the inputs are permuted within 64, the same for x, so that both
// operands come straight from memory in 16-byte pieces.  A block's 8 warps share
// 8 / parts groups of 16 outputs, `parts` warps to the inputs of one.  What bounds it:
// memory, and beside it the integer instruction (4 rows by 65536 x 4096: 51 us, 5.3 TB/s,
// the tensor cores busy for 61% of it); one row by 4096 x 4096 (7.5 us, the bytes 2.5) a
// launch, the row's quantising in every block and one round of loads.
constexpr int kNarrowWarps = 8;
constexpr int kSteps = 4;  // of 64 inputs, in flight

__device__ __forceinline__ uint4 read_codes(const int8_t* p, bool there) {
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (there) v = __ldg(reinterpret_cast<const uint4*>(p));
  return v;
}
__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                       uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The rows' codes into shared memory (`pitch` bytes a row), scales beside them, by the
// whole block: 8 / 4 / 2 / 1 warps to a row of 1, 2, 4, 8.
template <typename T>
__device__ void quantize_here(const T* x, int rows, int K, int8_t* codes, int pitch,
                              float* scales) {
  constexpr int V = Piece<T>::n;
  __shared__ float tops[kNarrowWarps];
  __shared__ int goods[kNarrowWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int each = rows <= 1 ? 8 : rows <= 2 ? 4 : rows <= 4 ? 2 : 1;
  const int row = warp / each, part = warp % each, step = each * 32 * V;
  const T* xr = x + static_cast<int64_t>(row) * K;
  const int first = (part * 32 + lane) * V;
  Top top;
  if (row < rows) {
#pragma unroll 2
    for (int k = first; k < K; k += step) top.look(read_piece(xr + k));
    top.of_warp();
  }
  if (lane == 0) tops[warp] = top.most, goods[warp] = top.good;
  __syncthreads();
  if (row < rows) {
    for (int w = row * each; w < (row + 1) * each; ++w)
      top.most = fmaxf(top.most, tops[w]), top.good &= goods[w] != 0;
    const Coder coder(top);
    if (part == 0 && lane == 0) scales[row] = coder.scale;
#pragma unroll 1
    for (int k = first; k < K; k += step)
      coder.put(read_piece(xr + k), codes + static_cast<int64_t>(row) * pitch + k);
  }
  __syncthreads();
}

// X: what x is; codes, or values that the kernel quantises itself (up to 8 rows).
template <int NT, typename X>
__global__ void __launch_bounds__(kNarrowWarps * 32, 2)
    narrow_kernel(const __grid_constant__ Args a, int parts) {
  constexpr bool kHere = !std::is_same<X, int8_t>::value;
  extern __shared__ __align__(16) int8_t here[];
  __shared__ float here_scales[8];
  __shared__ int sums[kNarrowWarps][16 * 8 * NT];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int part = warp % parts, group = blockIdx.x * (kNarrowWarps / parts) + warp / parts;
  const int n0 = group * 16;
  const int rows = a.rows;
  int acc[NT][4];
#pragma unroll
  for (int c = 0; c < NT; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[c][i] = 0;
  const int steps = (a.K + 63) / 64;
  const int begin = steps * part / parts, end = steps * (part + 1) / parts;
  // outputs and rows past the last one repeat it; what they give is not stored
  const int8_t* w0 = a.W + static_cast<int64_t>(min(n0 + g, a.N - 1)) * a.K + t * 16;
  const int8_t* w1 = a.W + static_cast<int64_t>(min(n0 + g + 8, a.N - 1)) * a.K + t * 16;
  const int pitch = a.K + 64;  // neighbouring rows in other banks
  const int8_t* xs[NT];
#pragma unroll
  for (int c = 0; c < NT; ++c) {
    const int r = min(c * 8 + g, rows - 1);
    xs[c] = kHere ? here + r * pitch + t * 16
                  : static_cast<const int8_t*>(a.x) + static_cast<int64_t>(r) * a.K + t * 16;
  }
  uint4 w[2][kSteps][2];
  auto load = [&](int set, int step) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int k = (step + i) * 64;
      const bool there = step + i < end && k + t * 16 < a.K;
      w[set][i][0] = read_codes(w0 + k, there);
      w[set][i][1] = read_codes(w1 + k, there);
    }
  };
  load(0, begin);
  if constexpr (kHere)
    quantize_here(static_cast<const X*>(a.x), rows, a.K, here, pitch, here_scales);
  else
    pdl_wait();  // x
  auto use = [&](int set, int step) {
    uint4 x[NT][kSteps];
#pragma unroll
    for (int c = 0; c < NT; ++c)
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int k = (step + i) * 64;
        x[c][i] = make_uint4(0u, 0u, 0u, 0u);
        if (step + i < end && k + t * 16 < a.K)
          x[c][i] = *reinterpret_cast<const uint4*>(xs[c] + k);
      }
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
#pragma unroll
      for (int c = 0; c < NT; ++c) {
        const uint4 &p = w[set][i][0], &q = w[set][i][1], &v = x[c][i];
        mma_s8(acc[c], p.x, q.x, p.y, q.y, v.x, v.y);
        mma_s8(acc[c], p.z, q.z, p.w, q.w, v.z, v.w);
      }
  };
  for (int s = begin; s < end; s += 2 * kSteps) {
    load(1, s + kSteps);
    use(0, s);
    load(0, s + 2 * kSteps);
    use(1, s + kSteps);
  }
  // sums[warp][column][output]
#pragma unroll
  for (int c = 0; c < NT; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      sums[warp][(c * 8 + t * 2 + (i & 1)) * 16 + g + (i >> 1) * 8] = acc[c][i];
  __syncthreads();
  const int groups = kNarrowWarps / parts;
  for (int i = threadIdx.x; i < groups * rows * 16; i += kNarrowWarps * 32) {
    const int n = i & 15, at = i >> 4, gr = at % groups, m = at / groups;
    const int out = (blockIdx.x * groups + gr) * 16 + n;
    if (out >= a.N) continue;
    int sum = 0;
    for (int p = 0; p < parts; ++p) sum += sums[gr * parts + p][m * 16 + n];
    const float v = scaled(sum, kHere ? here_scales[m] : a.x_scale[m], a.w_scale[out], a.bias ? a.bias[out] : 0.f);
    const int64_t to = static_cast<int64_t>(m) * a.N + out;
    if (a.out_f32) static_cast<float*>(a.y)[to] = v;
    else static_cast<__nv_bfloat16*>(a.y)[to] = __float2bfloat16_rn(v);
  }
}

// X int8_t: the kernel reads weights before it waits for the launch before it, which
// therefore has to be this call's own quantising (itself begun after all that came
// earlier); after anything else it is launched as usual.
template <int NT, typename X>
cudaError_t narrow(const Args& a, bool after_own, cudaStream_t s) {
  // warps for 16 on each of 152 SMs, where the inputs allow it
  const int groups = (a.N + 15) / 16;
  int parts = 1;
  while (parts < kNarrowWarps && groups * parts < 2432 && a.K / (parts * 2) >= 256) parts *= 2;
  const int each = kNarrowWarps / parts;
  const dim3 grid((groups + each - 1) / each), block(kNarrowWarps * 32);
  if (after_own) return launch_dependent(narrow_kernel<NT, X>, grid, block, 0, s, a, parts);
  const size_t smem = std::is_same<X, int8_t>::value
                          ? 0 : static_cast<size_t>(a.rows) * (a.K + 64);
  narrow_kernel<NT, X><<<grid, block, smem, s>>>(a, parts);
  return cudaGetLastError();
}

// Whether the narrow kernel's blocks quantise x themselves: it spares a launch (1 x 4096
// bf16 by 4096 x 4096: 7.2 us on the device where two launches take 7.7, and 7.1 of the
// host's time where those take 8.5), but each of them reads all of it.
bool quantize_inside(int64_t rows, int K, int x_dtype) {
  return rows * K * (x_dtype == MOE_F32 ? 4 : 2) <= 32 * 1024;
}

// Codes as fp16 numbers, for the wide kernel.
__global__ void __launch_bounds__(256) halves_kernel(int64_t n, const int8_t* codes, __half* out) {
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 16;
  pdl_trigger();
  if (i >= n) return;  // n is a multiple of 16
  const int4 q = *reinterpret_cast<const int4*>(codes + i);
  int8_t c[16];
  memcpy(c, &q, 16);
  __half h[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) h[j] = __int2half_rn(c[j]);
  uint4 v[2];
  memcpy(v, h, 32);
  *reinterpret_cast<uint4*>(out + i) = v[0];
  *reinterpret_cast<uint4*>(out + i + 8) = v[1];
}

size_t up256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

}  // namespace
}  // namespace i8

cudaError_t launch_quantize_rows_i8(int64_t rows, int K, int dtype, const void* x, int8_t* codes,
                                    float* scales, cudaStream_t s) {
  return dtype == MOE_F32 ? i8::quantize<float>(rows, K, x, codes, scales, s)
                          : i8::quantize<__nv_bfloat16>(rows, K, x, codes, scales, s);
}

// Whether the narrow kernel takes it: up to 8 rows, and up to 16 where the weight is
// small, as the integer instruction is the bound with two sets of columns (16 rows of
// codes by 4096 x 4096: 8.3 us and 14.4 in the wide kernel, by 8192 x 4096 14.4 and 14.5;
// 13 rows by 14337 x 7168: 41 and 27).
static bool is_narrow(int64_t rows, int N, int K) {
  return rows <= 8 || (rows <= 16 && static_cast<int64_t>(N) * K <= 1 << 25);
}

// x as codes or fp16 numbers, its scales, partial sums.
struct LinearScratch {
  size_t scales, part, total;
};
static LinearScratch linear_scratch(int64_t rows, int N, int K) {
  LinearScratch L;
  L.scales = i8::up256(static_cast<size_t>(rows) * K * (is_narrow(rows, N, K) ? 1 : 2));
  L.part = L.scales + i8::up256(static_cast<size_t>(rows) * 4);
  const int splits = is_narrow(rows, N, K) ? 1 : i8::wide_splits(rows, N, K);
  L.total = L.part + (splits > 1 ? static_cast<size_t>(splits) * rows * N * 4 : 0);
  return L;
}
size_t i8_linear_scratch(int64_t rows, int N, int K) { return linear_scratch(rows, N, K).total; }

// What any call of up to so many rows needs: rows of as many columns (32, 64, or chunks of
// 128) are cut into as many parts, so the most of each are looked at; with 152 items or
// more, and so from 152 chunks on, nothing is cut.
size_t i8_linear_scratch_most(int64_t rows, int N, int K) {
  size_t most = i8_linear_scratch(rows, N, K);
  auto look = [&](int64_t r) {
    const size_t bytes = i8_linear_scratch(r < rows ? r : rows, N, K);
    most = bytes > most ? bytes : most;
  };
  look(8);
  look(16);
  look(32);
  look(64);
  for (int64_t r = 128; r < rows && r <= 152 * 128; r += 128) look(r);
  return most;
}

cudaError_t launch_linear_i8(int64_t rows, int N, int K, const void* x, int x_dtype,
                             const float* x_scale, const int8_t* W, const float* w_scale,
                             const float* bias, void* y, int y_dtype, void* scratch, int* err,
                             cudaStream_t s) {
  const LinearScratch L = linear_scratch(rows, N, K);
  char* at = static_cast<char*>(scratch);
  i8::Args a = {};
  a.rows = static_cast<int>(rows), a.N = N, a.K = K;
  a.W = W, a.w_scale = w_scale, a.bias = bias;
  a.y = y, a.out_f32 = y_dtype == MOE_F32;
  a.err = err;
  a.x_scale = x_scale;
  float* scales = reinterpret_cast<float*>(at + L.scales);
  const bool coded = x_dtype == MOE_I8;
  if (!coded) a.x_scale = scales;
  a.x = x;
  if (is_narrow(rows, N, K)) {
    if (!coded && rows <= 8 && i8::quantize_inside(rows, K, x_dtype))
      return x_dtype == MOE_F32 ? i8::narrow<1, float>(a, false, s)
                                : i8::narrow<1, __nv_bfloat16>(a, false, s);
    if (!coded) {
      int8_t* codes = reinterpret_cast<int8_t*>(at);
      const cudaError_t st = launch_quantize_rows_i8(rows, K, x_dtype, x, codes, scales, s);
      if (st != cudaSuccess) return st;
      a.x = codes;
    }
    return rows <= 8 ? i8::narrow<1, int8_t>(a, !coded, s) : i8::narrow<2, int8_t>(a, !coded, s);
  }
  __half* halves = reinterpret_cast<__half*>(at);
  cudaError_t st;
  if (coded) {
    const int64_t n = rows * K;
    i8::halves_kernel<<<static_cast<unsigned>((n / 16 + 255) / 256), 256, 0, s>>>(
        n, static_cast<const int8_t*>(x), halves);
    st = cudaGetLastError();
  } else if (x_dtype == MOE_F32) {
    st = i8::quantize<float>(rows, K, x, halves, scales, s);
  } else {
    st = i8::quantize<__nv_bfloat16>(rows, K, x, halves, scales, s);
  }
  if (st != cudaSuccess) return st;
  a.splits = i8::wide_splits(rows, N, K);
  a.part = reinterpret_cast<int32_t*>(at + L.part);
  return i8::launch_wide(a, halves, s);
}

}  // namespace moe
