// Products with 4-bit weights (group scales) for few rows, and the routed
// SwiGLU experts built from them: the launches around w4_kernel.cuh and w4_wide.cuh.
#include "w4_kernel.cuh"

namespace moe {
namespace {

using namespace w4;

__device__ __forceinline__ float4 load4(const float* p) {
  return *reinterpret_cast<const float4*>(p);
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 q = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(q.x << 16), __uint_as_float(q.x & 0xffff0000u),
                     __uint_as_float(q.y << 16), __uint_as_float(q.y & 0xffff0000u));
}

// the largest magnitude of four values and one so far; infinity for any that
// is none or not a number (fmaxf would drop it)
__device__ __forceinline__ float top_of(float top, float4 q) {
  const float m = fmaxf(fmaxf(fabsf(q.x), fabsf(q.y)), fmaxf(fabsf(q.z), fabsf(q.w)));
  const bool good = isfinite(q.x) && isfinite(q.y) && isfinite(q.z) && isfinite(q.w);
  return fmaxf(top, good ? m : __uint_as_float(0x7f800000u));
}

// Rows of x into fp16.  With 2^E the largest magnitude of a row (its exponent),
// x = 2^(E-14) (p0 + 2^-11 p1): p0 is the nearest fp16 number, p1 that of what
// is left.  The inputs 2, 3, 6 and 7 of eight are held over 16, so that fp16's last
// step, 2^-24, is 2^-20 of theirs: bf16 values down to 2^-27 of the row's largest
// are exact.  Inputs past K give zeros.  A row with an infinity or a NaN gives
// NaN.  A row to a block, which holds up to 16384 inputs from the search for the
// largest to the splitting (two blocks that each searched the whole row took
// 9.7 us for 128 rows of 14336 where one takes 7.5, both from cold caches); a warp has 128
// inputs, a block of the weights' layout, at a time.
// SORTED: row i is the token of the i-th pair in the plan's order.
constexpr int kSplitWarps = 16, kHeld = 8;
template <typename T, int CP, bool SORTED>
__global__ void __launch_bounds__(kSplitWarps * 32)
    w4_split_kernel(int K, int blocks, const T* x, __half* pieces, float* units, Args a) {
  __shared__ float tops[kSplitWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x;
  pdl_trigger();
  pdl_wait();
  int from = row;
  if constexpr (SORTED) {
    __shared__ Plan plan;
    make_plan(plan, a, kTallColumns);
    if (row >= plan.end[MOE_MAX_EXPERTS - 1]) return;  // dropped pairs
    from = plan.token[row];
  }
  const T* xr = x + static_cast<int64_t>(from) * K;
  float4 held[kHeld];
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int k = (i * kSplitWarps + warp) * 128 + lane * 4;
    held[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (k < K) held[i] = load4(xr + k);
  }
#pragma unroll
  for (int i = 0; i < kHeld; ++i) top = top_of(top, held[i]);
  for (int k = kHeld * kSplitWarps * 128 + threadIdx.x * 4; k < K; k += kSplitWarps * 128)
    top = top_of(top, load4(xr + k));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
  if (lane == 0) tops[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kSplitWarps; ++w) top = fmaxf(top, tops[w]);
  // the exponent field of 2^(E-14), within what its reciprocal can hold
  int e = static_cast<int>(__float_as_uint(top) >> 23) - 14;
  e = e < 1 ? 1 : e;
  const float inverse = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
  if (threadIdx.x == 0)
    units[row] = __uint_as_float(isfinite(top) ? static_cast<uint32_t>(e) << 23 : 0x7fffffffu);

  auto split = [&](int blk, float4 q) {
    float v[4] = {q.x * inverse, q.y * inverse, q.z * inverse, q.w * inverse};
#pragma unroll
    for (int p = 0; p < CP; ++p) {
      __half h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // the inputs 2, 3, 6 and 7 of eight meet codes that stand 4 bits higher
        const float up = i < 2 ? 1.f : 16.f;
        h[i] = __float2half_rn(v[i] * (1.f / up));
        const float had = __half2float(h[i]) * up;
        v[i] = (v[i] - had) * 2048.f;
      }
      __half2 out[2] = {__halves2half2(h[0], h[1]), __halves2half2(h[2], h[3])};
      *reinterpret_cast<uint2*>(pieces +
                                ((static_cast<int64_t>(row) * CP + p) * blocks + blk) * 128 +
                                lane * 4) = *reinterpret_cast<uint2*>(out);
    }
  };
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (i * kSplitWarps + warp < blocks) split(i * kSplitWarps + warp, held[i]);
  for (int blk = kHeld * kSplitWarps + warp; blk < blocks; blk += kSplitWarps) {
    const int k = blk * 128 + lane * 4;
    split(blk, k < K ? load4(xr + k) : make_float4(0.f, 0.f, 0.f, 0.f));
  }
}

size_t align256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

// Split rows in the scratch, with room for the block that the kernels read past
// the last one.
struct Split {
  __half* x;
  float* unit;
};
size_t split_bytes(size_t rows, int K, int pieces) {
  const size_t blocks = rows * w4_blocks(K);
  return align256((blocks * pieces + 1) * 256) + align256(rows * 4);
}
Split split_at(char* at, size_t rows, int K, int pieces) {
  const size_t blocks = rows * w4_blocks(K);
  Split p;
  p.x = reinterpret_cast<__half*>(at);
  p.unit = reinterpret_cast<float*>(at + align256((blocks * pieces + 1) * 256));
  return p;
}

// a: the pairs, if SORTED
template <typename T, int CP, bool SORTED>
cudaError_t launch_split(bool dependent, int rows, int K, const T* x, const Split& p,
                         const Args& a, cudaStream_t s) {
  const int blocks = w4_blocks(K);
  auto k = w4_split_kernel<T, CP, SORTED>;
  const dim3 grid(static_cast<unsigned>(rows)), block(kSplitWarps * 32);
  if (dependent)
    return launch_dependent(k, grid, block, 0, s, K, blocks, x, p.x, p.unit, a);
  k<<<grid, block, 0, s>>>(K, blocks, x, p.x, p.unit, a);
  return cudaGetLastError();
}

// y[t] = sum_j p[t, j] sum_s part[s][t, j], over the kept pairs
__global__ void __launch_bounds__(256)
    w4_combine_kernel(int T, int h, int k, int E, int splits, const float* part,
                      const int32_t* idx, const float* prob, const uint8_t* keep,
                      __nv_bfloat16* y) {
  const int per_row = h / 4;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= static_cast<int64_t>(T) * per_row) return;
  const int t = static_cast<int>(i / per_row), c = static_cast<int>(i % per_row) * 4;
  pdl_wait();
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < k; ++j) {
    const int pair = t * k + j, e = idx[pair];
    if ((keep && keep[pair] == 0) || e < 0 || e >= E) continue;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int q = 0; q < splits; ++q) {
      const float4 u = *reinterpret_cast<const float4*>(
          part + (static_cast<int64_t>(q) * T * k + pair) * h + c);
      v.x += u.x;
      v.y += u.y;
      v.z += u.z;
      v.w += u.w;
    }
    const float p = prob[pair];
    s[0] += p * v.x;
    s[1] += p * v.y;
    s[2] += p * v.z;
    s[3] += p * v.w;
  }
  __nv_bfloat162* out = reinterpret_cast<__nv_bfloat162*>(y + static_cast<int64_t>(t) * h + c);
  out[0] = __floats2bfloat162_rn(s[0], s[1]);
  out[1] = __floats2bfloat162_rn(s[2], s[3]);
}

// y = the sum of the parts of a split product
__global__ void __launch_bounds__(256)
    w4_join_kernel(int64_t n, int splits, const float* part, int out_f32, void* y) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= n) return;
  pdl_wait();
  float s = 0.f;
#pragma unroll 4
  for (int q = 0; q < splits; ++q) s += part[q * n + i];
  if (out_f32) static_cast<float*>(y)[i] = s;
  else static_cast<__nv_bfloat16*>(y)[i] = __float2bfloat16_rn(s);
}

struct LinearShape {
  int rows;  // of one launch
  Way way;
};
LinearShape linear_shape(int64_t rows, int N, int K) {
  LinearShape L;
  L.rows = static_cast<int>(rows < kMaxRows ? rows : kMaxRows);
  // a second launch adds the parts up: some 1.5 us, about 6 blocks of a warp
  L.way = way_of(LINEAR, L.rows, (L.rows + 63) / 64, N, w4_blocks(K), 6);
  return L;
}

struct ExpertsShape {
  int tokens, pairs;  // of one launch
  Way way1, way2;
};
ExpertsShape experts_shape(int T, int h, int E, int k, int f) {
  ExpertsShape S;
  const int most = kMaxRows / k;
  S.tokens = T < most ? T : most;
  S.pairs = S.tokens * k;
  // rows that an expert has at most, or with luck: the mean and two standard
  // deviations of a random routing
  const double mean = static_cast<double>(S.pairs) / E;
  const double luck = mean + 2.0 * __builtin_sqrt(mean) + 1.0;
  const int64_t rows = static_cast<int64_t>(luck < S.tokens ? luck : S.tokens);
  const int64_t hit = S.pairs < E ? S.pairs : E;
  S.way1 = way_of(FC1, rows, hit, f, w4_blocks(h), -1);
  S.way2 = way_of(FC2, rows, hit, h, w4_blocks(f), 0);
  return S;
}

}  // namespace

namespace w4 {

namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
bool map_3d(CUtensorMap* m, CUtensorMapDataType type, void* at, const cuuint64_t (&dims)[3],
            const cuuint64_t (&strides)[2], const cuuint32_t (&box)[3],
            CUtensorMapSwizzle swizzle) {
  static const EncodeTiledFn encode = []() -> EncodeTiledFn {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  const cuuint32_t unit[3] = {1, 1, 1};
  return encode != nullptr &&
         encode(m, type, 3, at, dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool map_codes(CUtensorMap* m, const uint8_t* codes, int64_t rows, int blocks, int box_rows,
               bool swapped) {
  return map_3d(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, const_cast<uint8_t*>(codes),
                {64, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(blocks)},
                {static_cast<cuuint64_t>(blocks) * 64, 64},
                {64, static_cast<cuuint32_t>(box_rows), swapped ? 2u : 4u},
                swapped ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_NONE);
}

bool map_x(CUtensorMap* m, const __half* x, int64_t columns, int blocks) {
  return map_3d(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, const_cast<__half*>(x),
                {64, static_cast<cuuint64_t>(columns), static_cast<cuuint64_t>(blocks) * 2},
                {static_cast<cuuint64_t>(blocks) * 256, 128}, {64, 8, 2},
                CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace w4

size_t w4_linear_scratch(int64_t rows, int N, int K) {
  const LinearShape L = linear_shape(rows, N, K);
  return split_bytes(L.rows, K, 1) +
         (L.way.splits == 1 ? 0 : static_cast<size_t>(L.way.splits) * L.rows * N * 4);
}

// Fewer rows are cut into more parts, so a call of them can need more.  A launch
// has kMaxRows rows at most: all of them are tried, some 10 us in all.
size_t w4_linear_scratch_most(int64_t rows, int N, int K) {
  size_t most = 0;
  for (int64_t r = 0; r <= rows && r <= kMaxRows; ++r) {
    const size_t bytes = w4_linear_scratch(r, N, K);
    most = bytes > most ? bytes : most;
  }
  return most;
}

cudaError_t launch_w4_linear(int64_t rows, int N, int K, int group, const void* x, const W4& W,
                             void* y, int y_dtype, void* scratch, int* err, cudaStream_t s) {
  const LinearShape L = linear_shape(rows, N, K);
  const Split xs = split_at(static_cast<char*>(scratch), L.rows, K, 1);
  float* part =
      reinterpret_cast<float*>(static_cast<char*>(scratch) + split_bytes(L.rows, K, 1));
  const int out_f32 = y_dtype == MOE_F32;
  for (int64_t r = 0; r < rows; r += L.rows) {
    const int m = static_cast<int>(rows - r < L.rows ? rows - r : L.rows);
    void* out = static_cast<char*>(y) + r * N * (out_f32 ? 4 : 2);
    Args a = {};
    cudaError_t st = launch_split<__nv_bfloat16, 1, false>(
        false, m, K, static_cast<const __nv_bfloat16*>(x) + r * K, xs, a, s);
    if (st != cudaSuccess) return st;
    a.x = xs.x;
    a.unit = xs.unit;
    a.rows = m;
    a.err = err;
    a.w0 = a.w1 = W;
    a.blocks = w4_blocks(K);
    a.groups = K / group;
    a.N = N;
    a.splits = L.way.splits;
    a.few = L.way.few;
    a.out = L.way.splits > 1 ? part : out;
    a.out_f32 = L.way.splits > 1 ? 1 : out_f32;
    st = launch_linear(group, K, L.way.wide, a, s);
    if (st != cudaSuccess) return st;
    if (L.way.splits > 1) {
      const int64_t n = static_cast<int64_t>(m) * N;
      st = launch_dependent(w4_join_kernel, dim3(static_cast<unsigned>((n + 255) / 256)),
                            dim3(256), 0, s, n, L.way.splits,
                            static_cast<const float*>(part), out_f32, out);
      if (st != cudaSuccess) return st;
    }
  }
  return cudaSuccess;
}

size_t w4_experts_scratch(int T, int h, int E, int k, int f) {
  const ExpertsShape S = experts_shape(T, h, E, k, f);
  return split_bytes(S.way1.wide ? S.pairs : S.tokens, h, 1) +
         align256(static_cast<size_t>(S.pairs) * f * 4) +
         split_bytes(S.pairs, f, 2) + static_cast<size_t>(S.way2.splits) * S.pairs * h * 4;
}

size_t w4_experts_scratch_most(int T, int h, int E, int k, int f) {
  size_t most = 0;
  for (int t = 0; t <= T && t <= kMaxRows / k; ++t) {
    const size_t bytes = w4_experts_scratch(t, h, E, k, f);
    most = bytes > most ? bytes : most;
  }
  return most;
}

cudaError_t launch_w4_experts(int T, int h, int E, int k, int f, int group, const void* x,
                              const int32_t* topk_idx, const float* topk_prob,
                              const uint8_t* keep, const W4& W1, const W4& W3, const W4& W2,
                              void* y, void* scratch, int* err, cudaStream_t s) {
  const ExpertsShape S = experts_shape(T, h, E, k, f);
  char* at = static_cast<char*>(scratch);
  const int x_rows = S.way1.wide ? S.pairs : S.tokens;
  const Split xs = split_at(at, x_rows, h, 1);
  at += split_bytes(x_rows, h, 1);
  float* hidden = reinterpret_cast<float*>(at);
  at += align256(static_cast<size_t>(S.pairs) * f * 4);
  const Split hs = split_at(at, S.pairs, f, 2);
  at += split_bytes(S.pairs, f, 2);
  float* part = reinterpret_cast<float*>(at);
  for (int t = 0; t < T; t += S.tokens) {
    const int n = T - t < S.tokens ? T - t : S.tokens;
    const int64_t first = static_cast<int64_t>(t) * k;
    Args a = {};
    a.idx = topk_idx + first;
    a.keep = keep ? keep + first : nullptr;
    a.pairs = n * k;
    a.E = E;
    a.topk = k;
    a.err = err;
    const __nv_bfloat16* in = static_cast<const __nv_bfloat16*>(x) + static_cast<int64_t>(t) * h;
    cudaError_t st =
        S.way1.wide ? launch_split<__nv_bfloat16, 1, true>(false, n * k, h, in, xs, a, s)
                    : launch_split<__nv_bfloat16, 1, false>(false, n, h, in, xs, a, s);
    if (st != cudaSuccess) return st;
    a.x = xs.x;
    a.unit = xs.unit;
    a.w0 = W1;
    a.w1 = W3;
    a.blocks = w4_blocks(h);
    a.groups = h / group;
    a.N = f;
    a.splits = 1;
    a.few = S.way1.few;
    a.out = hidden;
    st = launch_fc1(group, h, S.way1.wide, a, s);
    if (st != cudaSuccess) return st;
    // rows of dropped pairs hold nothing; nobody reads their pieces
    st = launch_split<float, 2, false>(true, n * k, f, hidden, hs, a, s);
    if (st != cudaSuccess) return st;
    a.x = hs.x;
    a.unit = hs.unit;
    a.w0 = a.w1 = W2;
    a.blocks = w4_blocks(f);
    a.groups = f / group;
    a.N = h;
    a.splits = S.way2.splits;
    a.few = S.way2.few;
    a.out = part;
    st = launch_fc2(group, f, S.way2.wide, a, s);
    if (st != cudaSuccess) return st;
    const int64_t vecs = static_cast<int64_t>(n) * (h / 4);
    st = launch_dependent(w4_combine_kernel, dim3(static_cast<unsigned>((vecs + 255) / 256)),
                          dim3(256), 0, s, n, h, k, E, S.way2.splits,
                          static_cast<const float*>(part), a.idx, topk_prob + first, a.keep,
                          static_cast<__nv_bfloat16*>(y) + static_cast<int64_t>(t) * h);
    if (st != cudaSuccess) return st;
  }
  return cudaSuccess;
}

}  // namespace moe
