// Layer norm and RMS norm of z = residual + dropout(x), their backward pass
// with the reduction of the parameters' gradients, and the dropout with the
// residual sum on its own.
#include <type_traits>

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
  const uint64_t ctr[1] = {static_cast<uint64_t>(i) >> 2};
  uint4 words[1];
  philox_words(g, ctr, words);
  const uint4 w = words[0];
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

// ---- rows of any width ----
//
// One block to a row, for widths past what the kernels below hold on the chip:
// the row is read once for the mean, once for the variance and once for the
// output.
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

// ---- rows that stay on the chip ----
//
// A row belongs to a group of warps that holds it in registers, VPT vectors of
// 16 bytes to a thread, from the first read to the last write, so every tensor
// moves once.  Vectors are cut from the whole tensor and not from the row:
// they are 16-byte aligned for every width, and a row of odd width starts and
// ends inside one.  Such an edge vector is read and written element by element.
// Which elements of a vector a column falls on (the row's phase) depends on
// the row number modulo the vector length; a block takes the rows of one
// residue, so its phase is fixed, its copy of the weights in shared memory is
// laid out for it, and in the backward pass a thread keeps the same columns.
//
// Measured, bf16 with fp32 parameters, bytes once in and once out: forward 8192 x
// 4096 27.5 us (4.9 TB/s, of 6.8 that a copy reaches), with dropout and residual
// 59.6 us (4.5 TB/s); backward 16384 x 4096 90 us (4.5 TB/s), with dropout 138 us
// (4.9 TB/s); fp32 forward 4096 x 4096 25.7 us (5.2), backward 8192 x 4096 70 us
// (5.7).  No unit is full in bf16 (with dropout the issue slots and the fp32 pipe
// 55-59%, the memory 52-72%): a row's reads, its parameters from shared memory, the
// generator's rounds (at least 80 cycles of an SM quarter for 128 elements) and its
// sums follow one another in the few warps that hold it.  Odd widths (8192 x 4099:
// 42 us, backward 86) pay for edge vectors and an odd number of warps.

template <typename T>
struct Lanes {
  static constexpr int V = 16 / static_cast<int>(sizeof(T));
};

// Two fp32 values in one instruction: the rows' arithmetic is bound by
// instructions issued, not by the fp32 units.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{.reg .b64 a, b, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; add.rn.f32x2 d, a, b; "
      "mov.b64 {%0, %1}, d;}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{.reg .b64 a, b, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mul.rn.f32x2 d, a, b; "
      "mov.b64 {%0, %1}, d;}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{.reg .b64 a, b, c, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mov.b64 c, {%6, %7}; "
      "fma.rn.f32x2 d, a, b, c; mov.b64 {%0, %1}, d;}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// a vector's values, in pairs
__device__ __forceinline__ void unpack(const uint4& q, float2 (&v)[2], const float*) {
  v[0] = make_float2(__uint_as_float(q.x), __uint_as_float(q.y));
  v[1] = make_float2(__uint_as_float(q.z), __uint_as_float(q.w));
}
__device__ __forceinline__ void unpack(const uint4& q, float2 (&v)[4], const __nv_bfloat16*) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ uint4 pack(const float2 (&v)[2], const float*) {
  return make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x),
                    __float_as_uint(v[1].y));
}
__device__ __forceinline__ uint4 pack(const float2 (&v)[4], const __nv_bfloat16*) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __float22bfloat162_rn(v[i]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The elements of an edge vector that lie in the row, one by one.  The reads
// stay a loop: only the tensor's last vector takes it.
__device__ __forceinline__ uint32_t bits_of(const float* p) { return __float_as_uint(*p); }
__device__ __forceinline__ uint32_t bits_of(const __nv_bfloat16* p) {
  return __bfloat16_as_ushort(*p);
}
__device__ __forceinline__ void put_bits(float* p, uint32_t b) { *p = __uint_as_float(b); }
__device__ __forceinline__ void put_bits(__nv_bfloat16* p, uint32_t b) {
  *p = __ushort_as_bfloat16(static_cast<unsigned short>(b));
}
template <typename T>
__device__ __forceinline__ uint4 load_edge(const T* row, int col, int H) {
  constexpr int V = Lanes<T>::V, B = 32 * 4 / V;  // bits of an element
  uint4 q = make_uint4(0, 0, 0, 0);
#pragma unroll 1
  for (int e = 0; e < V; ++e) {
    if (col + e < 0 || col + e >= H) continue;
    const uint32_t b = bits_of(row + col + e) << (e * B % 32);
    const int w = e * B / 32;
    q.x |= w == 0 ? b : 0;
    q.y |= w == 1 ? b : 0;
    q.z |= w == 2 ? b : 0;
    q.w |= w == 3 ? b : 0;
  }
  return q;
}
template <typename T>
__device__ __forceinline__ void store_edge(T* row, int col, int H, uint4 q) {
  constexpr int V = Lanes<T>::V, B = 32 * 4 / V;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const int w = e * B / 32;
    const uint32_t b = w == 0 ? q.x : w == 1 ? q.y : w == 2 ? q.z : q.w;
    if (col + e >= 0 && col + e < H) put_bits(row + col + e, b >> (e * B % 32));
  }
}

// The vector whose first element is column `col` of `row` (col may be negative
// or past the row in an edge vector).  An edge vector comes whole, foreign
// elements with it (mask_edge), but for the tensor's last one: `room` elements
// follow from the row's start on.
template <typename T, bool ALIGNED>
__device__ __forceinline__ uint4 load_vec(const T* row, int col, int H, int64_t room) {
  constexpr int V = Lanes<T>::V;
  if (col >= H) return make_uint4(0, 0, 0, 0);
  if (ALIGNED || col + V <= room) return *reinterpret_cast<const uint4*>(row + col);
  return load_edge(row, col, H);
}
// zeros for the elements outside of the row
template <int P>
__device__ __forceinline__ void mask_edge(float2 (&v)[P], int col, int H) {
  if (col >= 0 && col + 2 * P <= H) return;
#pragma unroll
  for (int e = 0; e < P; ++e) {
    if (col + 2 * e < 0 || col + 2 * e >= H) v[e].x = 0.f;
    if (col + 2 * e + 1 < 0 || col + 2 * e + 1 >= H) v[e].y = 0.f;
  }
}
template <typename T, bool ALIGNED>
__device__ __forceinline__ void store_vec(T* row, int col, int H,
                                          const float2 (&v)[Lanes<T>::V / 2]) {
  constexpr int V = Lanes<T>::V;
  if (col >= H) return;
  const uint4 q = pack(v, static_cast<const T*>(row));
  if (ALIGNED || (col >= 0 && col + V <= H)) *reinterpret_cast<uint4*>(row + col) = q;
  else store_edge(row, col, H, q);
}

// dropout of N vectors; vector n holds the flat elements first[n] .. first[n] + V - 1,
// first[n] % V == 0
template <int V, int N>
__device__ __forceinline__ void drop_vecs(const Dropout& d, const Philox& g,
                                          const int64_t (&first)[N], float2 (&v)[N][V / 2]) {
  constexpr int B = V / 4;  // generator blocks of a vector
  uint64_t ctr[N * B];
  uint4 w[N * B];
#pragma unroll
  for (int n = 0; n < N * B; ++n) ctr[n] = (static_cast<uint64_t>(first[n / B]) >> 2) + n % B;
  philox_words(g, ctr, w);
#pragma unroll
  for (int n = 0; n < N * B; ++n) {
    float2 &lo = v[n / B][n % B * 2], &hi = v[n / B][n % B * 2 + 1];
    lo = mul2(lo, both(d.scale));
    hi = mul2(hi, both(d.scale));
    lo.x = w[n].x > d.limit ? lo.x : 0.f;
    lo.y = w[n].y > d.limit ? lo.y : 0.f;
    hi.x = w[n].z > d.limit ? hi.x : 0.f;
    hi.y = w[n].w > d.limit ? hi.y : 0.f;
  }
}

// The row group of a thread.  group_warps warps hold one row; the groups of a
// block take rows of the block's residue in turn.
template <typename T, bool ALIGNED>
struct Group {
  int size, id, t, phase;
  int64_t row, step;
  __device__ Group(int group_warps, int H) {
    constexpr int V = Lanes<T>::V;
    size = group_warps * 32;
    id = threadIdx.x / size;
    t = threadIdx.x - id * size;
    const int groups = blockDim.x / size;
    step = static_cast<int64_t>(gridDim.x) * groups;
    if (ALIGNED) {
      phase = 0;
      row = static_cast<int64_t>(blockIdx.x) * groups + id;
    } else {  // gridDim.x is a multiple of V
      const int residue = blockIdx.x % V;
      phase = (residue * (H % V)) % V;
      row = residue + static_cast<int64_t>(V) * ((blockIdx.x / V) * groups + id);
    }
  }
  // first column of the thread's i-th vector
  __device__ int col(int i) const { return (i * size + t) * Lanes<T>::V - phase; }
};

// Sum over the group's threads in a fixed order, in every thread.  red:
// 2 x 32 values; calls alternate between its halves, which makes one barrier a
// call enough.
struct GroupSum {
  float2* red;
  int warps, base, half;
  __device__ GroupSum(float2* smem, int group_warps, int group)
      : red(smem), warps(group_warps), base(group * group_warps), half(0) {}

  __device__ static void shuffled(float2& v, int o) {
    v = add2(v, make_float2(__shfl_xor_sync(~0u, v.x, o), __shfl_xor_sync(~0u, v.y, o)));
  }
  __device__ static void shuffled(float& v, int o) { v += __shfl_xor_sync(~0u, v, o); }

  template <typename F>
  __device__ F operator()(F v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) shuffled(v, o);
    if (warps == 1) return v;
    const int lane = threadIdx.x & 31;
    F* buf = reinterpret_cast<F*>(red + half * 32);
    half ^= 1;
    if (lane == 0) buf[threadIdx.x >> 5] = v;
    // one barrier to a group of warps: the groups keep different rows
    asm volatile("bar.sync %0, %1;" ::"r"(1 + base / warps), "r"(warps * 32) : "memory");
    const int part = warps <= 8 ? lane & 7 : lane;  // every 8 lanes, or all 32
    v = F{};
    if (part < warps) v = buf[base + part];
    if (warps > 8) {
      shuffled(v, 16);
      shuffled(v, 8);
    }
    shuffled(v, 4);
    shuffled(v, 2);
    shuffled(v, 1);
    return v;
  }
};

// Where the value at phase + column of a parameter lies in shared memory.  A
// thread of bf16 rows reads eight values: the first halves of all threads' lie
// before the second halves, so that neighbours read neighbouring 16 bytes
// (8192 x 4096 bf16 33.2 -> 27.5 us: with the halves together, half of the banks
// waited).
template <int V>
__device__ __forceinline__ int place(int at, int padded) {
  if (V == 4) return at;
  return (at & 4 ? padded / 2 : 0) + (at >> 3) * 4 + (at & 3);
}

// A parameter's values at phase + column, zeros around them;
// without the parameter `none`.  A thread brings the columns that it will read,
// all its reads in flight at once; one group does it for the block.
template <typename T, int VPT, bool ALIGNED>
__device__ __forceinline__ void stage_param(float* dst, int padded, const void* p, int is_bf16,
                                            float none, const Group<T, ALIGNED>& g, int H) {
  constexpr int V = Lanes<T>::V;
  if (g.id != 0) return;
  float v[VPT][V];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = g.col(i);
#pragma unroll
    for (int e = 0; e < V; ++e) v[i][e] = c + e >= 0 && c + e < H ? none : 0.f;
    if (p == nullptr || c >= H) continue;
    if (ALIGNED && !is_bf16) {
#pragma unroll
      for (int e = 0; e < V; e += 4) {
        const float4 q = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + c + e);
        v[i][e] = q.x;
        v[i][e + 1] = q.y;
        v[i][e + 2] = q.z;
        v[i][e + 3] = q.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (c + e >= 0 && c + e < H) v[i][e] = param1(p, is_bf16, c + e);
    }
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int e = 0; e < V; e += 4)
      *reinterpret_cast<float4*>(dst + place<V>(g.col(i) + g.phase + e, padded)) =
          make_float4(v[i][e], v[i][e + 1], v[i][e + 2], v[i][e + 3]);
}

template <int V>
__device__ __forceinline__ void read_param(const float* src, int at, int padded,
                                           float2 (&v)[V / 2]) {
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    const float4 q = *reinterpret_cast<const float4*>(src + place<V>(at + 4 * i, padded));
    v[2 * i] = make_float2(q.x, q.y);
    v[2 * i + 1] = make_float2(q.z, q.w);
  }
}

// A row brought into L2 ahead of its reads, by one thread; the bytes around it
// that belong to its first and last 16 come too.  For the kernels that hold no
// row ahead (forward 1024 x 24568 bf16 35.2 -> 30.9 us, backward 4096 x 16384
// 160 -> 128 us); behind rows that are held it gains nothing.
template <typename T>
__device__ __forceinline__ void prefetch_row(const T* p, int64_t row, int64_t rows, int H) {
  if (row >= rows) return;
  constexpr int64_t size = sizeof(T), ones = 15;
  const int64_t from = row * H * size & ~ones, most = rows * H * size & ~ones;
  int64_t to = ((row + 1) * H * size + ones) & ~ones;
  to = to < most ? to : most;
  if (to > from)
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                     reinterpret_cast<const char*>(p) + from),
                 "r"(static_cast<uint32_t>(to - from))
                 : "memory");
}

template <typename T, int VPT, bool ALIGNED, bool DROP>
__global__ void __launch_bounds__(1024)
    norm_rows_kernel(NormArgs a, int group_warps, int padded, const T* x, const T* res,
                     const void* weight, const void* bias, T* z, T* y, float* mean, float* rstd) {
  constexpr int V = Lanes<T>::V, P = V / 2;
  extern __shared__ __align__(16) float params[];  // weight, bias: `padded` each
  __shared__ float2 red[64];
  const int H = a.hidden;
  const Group<T, ALIGNED> g(group_warps, H);
  GroupSum sum(red, group_warps, g.id);
  const Philox rng = DROP ? philox_of(a.rng) : Philox{};
  const float inv_h = 1.f / static_cast<float>(H);

  uint4 qx[VPT], qr[VPT];
  auto fetch = [&](uint4 (&q)[VPT], const T* p, int64_t r) {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      q[i] = load_vec<T, ALIGNED>(p + r * H, g.col(i), H, (a.rows - r) * H);
  };
  // one row ahead where the registers allow it
  constexpr bool AHEAD = VPT <= 2;
  if (AHEAD && g.row < a.rows) {
    fetch(qx, x, g.row);
    if (res) fetch(qr, res, g.row);
  }
  stage_param<T, VPT>(params, padded, weight, a.param_bf16, 1.f, g, H);
  stage_param<T, VPT>(params + padded, padded, bias, a.param_bf16, 0.f, g, H);
  __syncthreads();

  for (int64_t r = g.row; r < a.rows; r += g.step) {
    float2 v[VPT][P];
    if (!AHEAD) {
      fetch(qx, x, r);
      if (res) fetch(qr, res, r);
      if (g.t == 0) {
        prefetch_row(x, r + g.step, a.rows, H);
        if (res) prefetch_row(res, r + g.step, a.rows, H);
      }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) unpack(qx[i], v[i], x);
    // the next row's reads run under this row's work
    const bool more = AHEAD && r + g.step < a.rows;
    if (more) fetch(qx, x, r + g.step);
    if (DROP) {
      int64_t first[VPT];
#pragma unroll
      for (int i = 0; i < VPT; ++i) first[i] = r * H + g.col(i);
      drop_vecs<V>(a.drop, rng, first, v);
    }
    if (res) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        float2 w[P];
        unpack(qr[i], w, x);
#pragma unroll
        for (int e = 0; e < P; ++e) v[i][e] = add2(v[i][e], w[e]);
        if (z) store_vec<T, ALIGNED>(z + r * H, g.col(i), H, v[i]);
      }
    }
    if (more && res) fetch(qr, res, r + g.step);
    if (!ALIGNED) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) mask_edge(v[i], g.col(i), H);
    }
    float m = 0.f;
    if (!a.rms) {
      float2 s = both(0.f);
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < P; ++e) s = add2(s, v[i][e]);
      m = sum(s.x + s.y) * inv_h;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < P; ++e) v[i][e] = add2(v[i][e], both(-m));
      if (!ALIGNED) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) mask_edge(v[i], g.col(i), H);
      }
    }
    float2 sq = both(0.f);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = g.col(i);
      if (c >= H) continue;
#pragma unroll
      for (int e = 0; e < P; ++e) sq = fma2(v[i][e], v[i][e], sq);
    }
    const float rs = rsqrtf(sum(sq.x + sq.y) * inv_h + a.eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = g.col(i);
      if (c >= H) continue;
      float2 w[P], b[P];
      read_param<V>(params, c + g.phase, padded, w);
      read_param<V>(params + padded, c + g.phase, padded, b);
#pragma unroll
      for (int e = 0; e < P; ++e) b[e] = fma2(mul2(v[i][e], both(rs)), w[e], b[e]);
      store_vec<T, ALIGNED>(y + r * H, c, H, b);
    }
    if (g.t == 0) {
      if (mean && !a.rms) mean[r] = m;
      if (rstd) rstd[r] = rs;
    }
  }
}

// A thread's own vectors of the rows to come, copied to shared memory without
// registers.  Only the thread itself reads them, so no barrier is needed.
// Edge vectors are copied whole (their foreign elements are masked after) and
// the tensor's last vector as far as the tensor goes.
__device__ __forceinline__ void copy_vec(uint4* slot, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(slot))),
               "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// The sums for dweight and dbias stay in the thread's registers over all of its
// rows, are added up over the block's groups in order, and go to the block's
// part.  The row to come is read two rows ahead (STAGED).  Rows too wide for
// that keep the sums in shared memory and read a row when they come to it.
constexpr int kSlots = 3;
template <typename T, int VPT, bool ALIGNED, bool DROP, bool STAGED>
__global__ void __launch_bounds__(STAGED ? 512 : 640)
    norm_backward_rows_kernel(NormArgs a, int group_warps, int padded, const T* dy, const T* x,
                              const void* weight, const float* mean, const float* rstd,
                              const T* dz, T* dx, T* dbranch, float* part) {
  constexpr int V = Lanes<T>::V, P = V / 2;
  // weight [padded]; then the copied vectors (STAGED) or the two sums [padded]
  // each.  After the last row the staged sums take the place of all that.
  extern __shared__ __align__(16) float params[];
  __shared__ float2 red[64];
  const int H = a.hidden;
  const Group<T, ALIGNED> g(group_warps, H);
  GroupSum sum(red, group_warps, g.id);
  const Philox rng = DROP ? philox_of(a.rng) : Philox{};
  const float inv_h = 1.f / static_cast<float>(H);
  const int64_t total = a.rows * H;
  constexpr int S = STAGED ? VPT : 1;
  float2 sw[S][P], sb[S][P];
  float* sums = STAGED ? params : params + padded;
  uint4* slots = reinterpret_cast<uint4*>(params + padded) + threadIdx.x;
  auto slot = [&](int n, int tensor, int i) {
    return slots + ((n * 3 + tensor) * VPT + i) * blockDim.x;
  };
  auto fetch = [&](int64_t r, int n) {
    if (r < a.rows) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = g.col(i);
        if (c >= H) continue;
        const int64_t at = r * H + c;
        int bytes = 16;
        if (!ALIGNED && at + V > total) bytes = static_cast<int>(total - at) * sizeof(T);
        copy_vec(slot(n, 0, i), x + at, bytes);
        copy_vec(slot(n, 1, i), dy + at, bytes);
        if (dz) copy_vec(slot(n, 2, i), dz + at, bytes);
      }
    }
    copies_commit();
  };
  auto read = [&](const T* p, int64_t r, int n, int tensor, int i, float2(&v)[P]) {
    const int c = g.col(i);
    if (STAGED) {
      unpack(*slot(n, tensor, i), v, p);
    } else {
      unpack(load_vec<T, ALIGNED>(p + r * H, c, H, (a.rows - r) * H), v, p);
    }
    if (!ALIGNED) mask_edge(v, c, H);
  };
  if (STAGED) {
#pragma unroll
    for (int n = 0; n < kSlots - 1; ++n) fetch(g.row + n * g.step, n);
  }
  stage_param<T, VPT>(params, padded, weight, a.param_bf16, 1.f, g, H);
  if (!STAGED)
    for (int c = threadIdx.x; c < 2 * padded; c += blockDim.x) sums[c] = 0.f;
#pragma unroll
  for (int i = 0; i < S; ++i)
#pragma unroll
    for (int e = 0; e < P; ++e) sw[i][e] = sb[i][e] = both(0.f);
  float m_next = 0.f, rs_next = 0.f;
  if (g.row < a.rows) {
    if (!a.rms) m_next = mean[g.row];
    rs_next = rstd[g.row];
  }
  __syncthreads();

  int n = 0;  // the slot of row r
  for (int64_t r = g.row; r < a.rows; r += g.step) {
    const float m = m_next, rs = rs_next;
    if (r + g.step < a.rows) {
      if (!a.rms) m_next = mean[r + g.step];
      rs_next = rstd[r + g.step];
    }
    if (STAGED) {
      fetch(r + (kSlots - 1) * g.step, n == 0 ? kSlots - 1 : n - 1);
      copies_wait<kSlots - 1>();
    } else if (g.t == 0) {
      prefetch_row(x, r + g.step, a.rows, H);
      prefetch_row(dy, r + g.step, a.rows, H);
      if (dz) prefetch_row(dz, r + g.step, a.rows, H);
    }
    float2 s1 = both(0.f), s2 = both(0.f);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = g.col(i);
      if (c >= H) continue;
      float2 vx[P], vd[P], w[P];
      read(x, r, n, 0, i, vx);
      read(dy, r, n, 1, i, vd);
      read_param<V>(params, c + g.phase, padded, w);
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const float2 gw = mul2(vd[e], w[e]);
        s1 = add2(s1, gw);
        s2 = fma2(gw, mul2(add2(vx[e], both(-m)), both(rs)), s2);
      }
    }
    const float2 s = sum(make_float2(s1.x + s1.y, s2.x + s2.y));
    const float c1 = a.rms ? 0.f : s.x * inv_h, c2 = s.y * inv_h;
    float2 o[VPT][P];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = g.col(i);
#pragma unroll
      for (int e = 0; e < P; ++e) o[i][e] = both(0.f);
      if (c >= H) continue;
      float2 vx[P], vd[P], w[P], tw[P], tb[P];
      if (dz) read(dz, r, n, 2, i, o[i]);
      read(x, r, n, 0, i, vx);
      read(dy, r, n, 1, i, vd);
      read_param<V>(params, c + g.phase, padded, w);
      if (!STAGED) {
        read_param<V>(sums, c + g.phase, padded, tw);
        read_param<V>(sums + padded, c + g.phase, padded, tb);
      }
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const float2 xh = mul2(add2(vx[e], both(-m)), both(rs));
        const float2 core = fma2(xh, both(-c2), fma2(vd[e], w[e], both(-c1)));
        o[i][e] = fma2(core, both(rs), o[i][e]);
        if (STAGED) {
          sw[i][e] = fma2(vd[e], xh, sw[i][e]);
          sb[i][e] = add2(vd[e], sb[i][e]);
        } else {
          tw[e] = fma2(vd[e], xh, tw[e]);
          tb[e] = add2(vd[e], tb[e]);
        }
      }
      if (!STAGED) {
#pragma unroll
        for (int e = 0; e < P; e += 2) {
          const int at = place<V>(c + g.phase + 2 * e, padded);
          *reinterpret_cast<float4*>(sums + at) =
              make_float4(tw[e].x, tw[e].y, tw[e + 1].x, tw[e + 1].y);
          *reinterpret_cast<float4*>(sums + padded + at) =
              make_float4(tb[e].x, tb[e].y, tb[e + 1].x, tb[e + 1].y);
        }
      }
      store_vec<T, ALIGNED>(dx + r * H, c, H, o[i]);
      if (dbranch && (!DROP || !STAGED)) {
        if (DROP) {
          const int64_t first[1] = {r * H + c};
          float2(&one)[1][P] = *reinterpret_cast<float2(*)[1][P]>(&o[i]);
          drop_vecs<V>(a.drop, rng, first, one);
        }
        store_vec<T, ALIGNED>(dbranch + r * H, c, H, o[i]);
      }
    }
    if (DROP && STAGED) {
      int64_t first[VPT];
#pragma unroll
      for (int i = 0; i < VPT; ++i) first[i] = r * H + g.col(i);
      drop_vecs<V>(a.drop, rng, first, o);
#pragma unroll
      for (int i = 0; i < VPT; ++i) store_vec<T, ALIGNED>(dbranch + r * H, g.col(i), H, o[i]);
    }
    n = n == kSlots - 1 ? 0 : n + 1;
  }

  if (STAGED) copies_wait<0>();
  __syncthreads();
  if (STAGED) {
    const int groups = blockDim.x / g.size;
    for (int k = 0; k < groups; ++k) {
      if (g.id == k) {
#pragma unroll
        for (int i = 0; i < S; ++i) {
          const int at = g.col(i) + g.phase;
          if (at >= padded) continue;
#pragma unroll
          for (int e = 0; e < P; ++e) {
            float2* pw = reinterpret_cast<float2*>(sums + place<V>(at + 2 * e, padded));
            float2* pb = pw + padded / 2;
            *pw = k == 0 ? sw[i][e] : add2(*pw, sw[i][e]);
            *pb = k == 0 ? sb[i][e] : add2(*pb, sb[i][e]);
          }
        }
      }
      __syncthreads();
    }
  }
  float* out = part + static_cast<int64_t>(blockIdx.x) * 2 * H;
  for (int c = threadIdx.x; c < H; c += blockDim.x) {
    const int at = place<V>(c + g.phase, padded);
    out[c] = sums[at];
    out[H + c] = sums[padded + at];
  }
}

// dweight and dbias: the sums over the blocks' parts, in a fixed order.  One
// block to 32 columns of one of the two; warp w takes the parts w, w + 16, ...
constexpr int kGradWarps = 16;
__global__ void __launch_bounds__(kGradWarps * 32)
    norm_param_grads_kernel(int parts, int H, const float* part, float* dweight, float* dbias) {
  __shared__ float buf[kGradWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float* out = blockIdx.y == 0 ? dweight : dbias;
  pdl_wait();
  float s = 0.f;
  if (c < H && out) {
    const float* p = part + static_cast<int64_t>(blockIdx.y) * H + c;
#pragma unroll 10
    for (int i = warp; i < parts; i += kGradWarps) s += p[static_cast<int64_t>(i) * 2 * H];
  }
  buf[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < H && out) {
    s = 0.f;
#pragma unroll
    for (int w = 0; w < kGradWarps; ++w) s += buf[w][lane];
    out[c] = s;
  }
}

// Flat vectors of 16 bytes, two to a thread at a time so that their reads and
// their generator rounds overlap; the last elements of a length that is no
// multiple of the vector's go one by one.  8192 x 4096 bf16 with a residual:
// 36 us (5.6 TB/s); half of it is the generator's, under the memory's time.
template <typename T, bool DROP>
__global__ void __launch_bounds__(256)
    dropout_add_kernel(int64_t n, Dropout d, const uint64_t* rng, const T* x, const T* res, T* y) {
  constexpr int V = Lanes<T>::V;
  const Philox g = DROP ? philox_of(rng) : Philox{};
  const int64_t vecs = n / V;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  const int64_t me = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const uint4 *xv = reinterpret_cast<const uint4*>(x), *rv = reinterpret_cast<const uint4*>(res);
  uint4* yv = reinterpret_cast<uint4*>(y);
  for (int64_t q = me; q < vecs; q += 2 * step) {
    const bool two = q + step < vecs;
    const int64_t p[2] = {q, two ? q + step : q}, at[2] = {p[0] * V, p[1] * V};
    uint4 qx[2], qr[2];
    float2 v[2][V / 2], w[V / 2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      qx[i] = xv[p[i]];
      if (res) qr[i] = rv[p[i]];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) unpack(qx[i], v[i], x);
    if (DROP) drop_vecs<V>(d, g, at, v);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (res) {
        unpack(qr[i], w, x);
#pragma unroll
        for (int e = 0; e < V / 2; ++e) v[i][e] = add2(v[i][e], w[e]);
      }
      if (i == 0 || two) yv[p[i]] = pack(v[i], x);
    }
  }
  const int64_t i = vecs * V + me;
  if (i < n) {
    const float v = DROP ? drop1(d, g, i, load1(x, i)) : load1(x, i);
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

constexpr int kSms = 152;
constexpr size_t kMostSmem = 216 * 1024;

// How rows are laid over threads.  vectors: 16-byte vectors that a row can
// touch; group_warps warps x vpt vectors hold them.
struct Shape {
  int vpt = 0;  // 0: too wide for the chip, the wide kernel
  int group_warps = 0, groups = 1, padded = 0, threads = 0;
  bool aligned = true, staged = false;
  unsigned grid = 0;
};

void shape_common(Shape& s, const moe_norm_config& c, int vectors, int V) {
  s.group_warps = (vectors + s.vpt * 32 - 1) / (s.vpt * 32);
  s.groups = s.group_warps >= 8 ? 1 : 8 / s.group_warps;
  if (c.rows < static_cast<int64_t>(kSms) * s.groups) s.groups = 1;
  s.threads = s.group_warps * s.groups * 32;
  s.padded = s.group_warps * 32 * s.vpt * V;
}

// One wave of blocks, per_sm to an SM as far as shared memory allows; for odd
// widths whole sets of residues.
void shape_grid(Shape& s, const moe_norm_config& c, int V, int per_sm, size_t smem) {
  const int fit = static_cast<int>(kMostSmem / smem);
  if (per_sm > fit) per_sm = fit;
  const int64_t most = static_cast<int64_t>(kSms) * (per_sm < 1 ? 1 : per_sm);
  int64_t grid = (c.rows + s.groups - 1) / s.groups, top = most;
  if (!s.aligned) {
    grid = ((c.rows + V - 1) / V + s.groups - 1) / s.groups * V;
    top = most / V * V;
  }
  s.grid = static_cast<unsigned>(grid < top ? grid : top);
}

// vectors that a row of any phase can touch
int row_vectors(const moe_norm_config& c, int V) {
  return c.hidden % V == 0 ? c.hidden / V : (c.hidden + 2 * V - 2) / V;
}

// Two vectors to a thread: with one, more threads wait at each row's sums
// (8192 x 4096 bf16 27.5 us, one 36.1; 100 x 8192 4.0, one 4.6).  One for a few
// short rows, where all threads are few (100 x 2048 bf16 2.98 us, two 3.16) and
// for rows that one warp holds.  More where 1024 threads with two do not hold a
// row, without a row ahead in registers (1024 x 24568 bf16 30.9 us; the wide
// kernel 104).
Shape forward_shape(const moe_norm_config& c) {
  Shape s;
  const int V = c.dtype == MOE_F32 ? 4 : 8;
  if (c.hidden > 32768) return s;
  const int vectors = row_vectors(c, V);
  s.aligned = c.hidden % V == 0;
  if (vectors <= 32 || (c.rows <= kSms && vectors <= 256)) s.vpt = 1;
  else if (vectors <= 2048) s.vpt = 2;
  else if (V == 8 && vectors <= 3072) s.vpt = 3;
  else if (V == 4 && vectors <= 4096) s.vpt = 4;
  else if (V == 4 && vectors <= 5120) s.vpt = 5;
  else return s;
  shape_common(s, c, vectors, V);
  shape_grid(s, c, V, 1024 / s.threads, 2 * static_cast<size_t>(s.padded) * 4);
  return s;
}

size_t backward_smem(const Shape& s) {
  const size_t padded = static_cast<size_t>(s.padded) * 4;
  if (!s.staged) return 3 * padded;
  const size_t rows = padded + static_cast<size_t>(kSlots) * 3 * s.threads * s.vpt * 16;
  return rows > 2 * padded ? rows : 2 * padded;
}

// Staged up to what 16 warps hold with two vectors to a thread (16384 x 4096 bf16
// 90 us, 109 with the sums in shared memory and rows read as they come; 8192 x
// 8192 90 and 120; the wide kernel takes 355 and more).  Past that the sums need
// the shared memory (4096 x 16384 bf16 124 us; 735 in the wide kernel), and as
// many warps as hold the row with two to four vectors to a thread hide the reads
// best (7455 x 9001 bf16, two vectors 161 us, four 273).
Shape backward_shape(const moe_norm_config& c) {
  Shape s;
  const int V = c.dtype == MOE_F32 ? 4 : 8;
  if (c.hidden > 32768) return s;
  const int vectors = row_vectors(c, V);
  s.aligned = c.hidden % V == 0;
  s.vpt = vectors <= 32 ? 1 : 2;
  s.staged = vectors <= s.vpt * 32 * 16;
  if (!s.staged) {
    s.vpt = (vectors + 32 * 20 - 1) / (32 * 20);  // 2, 3, 4 or 8
    if (s.vpt > 4 && V == 4) s.vpt = 8;
  }
  if (s.vpt > 8 || (s.vpt > 4 && V == 8) || vectors > s.vpt * 32 * 20) {
    s.vpt = 0;
    return s;
  }
  shape_common(s, c, vectors, V);
  const size_t smem = backward_smem(s);
  if (smem > kMostSmem) {
    s.vpt = 0;
    return s;
  }
  shape_grid(s, c, V, 512 / s.threads, smem);
  return s;
}

// f with the values of the flags as types
template <typename F>
auto with_bool(bool b, F&& f) {
  return b ? f(std::true_type{}) : f(std::false_type{});
}

// 48 KB need no leave, but the kernels' own variables are among them.
template <auto KERNEL>
cudaError_t allow_smem(size_t bytes) {
  return bytes <= 47 * 1024 ? cudaSuccess : allow_most_smem<KERNEL>();
}

template <typename T>
cudaError_t norm_typed(const moe_norm_config& c, const void* x, const void* residual,
                       const uint64_t* rng, const void* weight, const void* bias, void* z, void* y,
                       float* mean, float* rstd, cudaStream_t s) {
  const NormArgs a = args_of(c, rng);
  const T *xt = static_cast<const T*>(x), *rt = static_cast<const T*>(residual);
  T *zt = static_cast<T*>(z), *yt = static_cast<T*>(y);
  const Shape p = forward_shape(c);
  auto launch = [&](auto vpt) -> cudaError_t {
    return with_bool(p.aligned, [&](auto aligned) {
      return with_bool(a.drop.on, [&](auto drop) -> cudaError_t {
        constexpr auto k = norm_rows_kernel<T, decltype(vpt)::value, decltype(aligned)::value,
                                            decltype(drop)::value>;
        const size_t smem = 2 * static_cast<size_t>(p.padded) * 4;
        const cudaError_t st = allow_smem<k>(smem);
        if (st != cudaSuccess) return st;
        k<<<p.grid, p.threads, smem, s>>>(a, p.group_warps, p.padded, xt, rt, weight, bias, zt, yt,
                                          mean, rstd);
        return cudaGetLastError();
      });
    });
  };
  switch (p.vpt) {
    case 1: return launch(std::integral_constant<int, 1>{});
    case 2: return launch(std::integral_constant<int, 2>{});
    case 3:
      if constexpr (sizeof(T) == 2) return launch(std::integral_constant<int, 3>{});
      break;
    case 4:
      if constexpr (sizeof(T) == 4) return launch(std::integral_constant<int, 4>{});
      break;
    case 5:
      if constexpr (sizeof(T) == 4) return launch(std::integral_constant<int, 5>{});
  }
  const unsigned grid = static_cast<unsigned>(c.rows < 65536 ? c.rows : 65536);
  norm_wide_kernel<T><<<grid, kRowThreads, 0, s>>>(a, xt, rt, weight, bias, zt, yt, mean, rstd);
  return cudaGetLastError();
}

template <typename T>
cudaError_t norm_backward_typed(const moe_norm_config& c, const void* dy, const void* z,
                                const void* weight, const float* mean, const float* rstd,
                                const void* dz, const uint64_t* rng, void* dx, void* dbranch,
                                float* part, cudaStream_t s) {
  NormArgs a = args_of(c, rng);
  if (dbranch == nullptr) a.drop.on = 0;
  const T *dyt = static_cast<const T*>(dy), *zt = static_cast<const T*>(z),
          *dzt = static_cast<const T*>(dz);
  T *dxt = static_cast<T*>(dx), *dbt = static_cast<T*>(dbranch);
  const Shape p = backward_shape(c);
  auto launch = [&](auto vpt, auto staged) -> cudaError_t {
    return with_bool(p.aligned, [&](auto aligned) {
      return with_bool(a.drop.on, [&](auto drop) -> cudaError_t {
        constexpr auto k =
            norm_backward_rows_kernel<T, decltype(vpt)::value, decltype(aligned)::value,
                                      decltype(drop)::value, decltype(staged)::value>;
        const size_t smem = backward_smem(p);
        const cudaError_t st = allow_smem<k>(smem);
        if (st != cudaSuccess) return st;
        k<<<p.grid, p.threads, smem, s>>>(a, p.group_warps, p.padded, dyt, zt, weight, mean, rstd,
                                          dzt, dxt, dbt, part);
        return cudaGetLastError();
      });
    });
  };
  if (p.vpt != 0 && p.staged) {
    if (p.vpt == 1) return launch(std::integral_constant<int, 1>{}, std::true_type{});
    return launch(std::integral_constant<int, 2>{}, std::true_type{});
  }
  if (p.vpt == 2) return launch(std::integral_constant<int, 2>{}, std::false_type{});
  if (p.vpt == 3) return launch(std::integral_constant<int, 3>{}, std::false_type{});
  if (p.vpt == 4) return launch(std::integral_constant<int, 4>{}, std::false_type{});
  if constexpr (sizeof(T) == 4)
    if (p.vpt == 8) return launch(std::integral_constant<int, 8>{}, std::false_type{});
  norm_backward_wide_kernel<T><<<norm_backward_ctas(c), kRowThreads, 0, s>>>(
      a, dyt, zt, weight, mean, rstd, dzt, dxt, dbt, part);
  return cudaGetLastError();
}

}  // namespace

int norm_backward_ctas(const moe_norm_config& c) {
  if (c.rows == 0) return 0;
  const Shape p = backward_shape(c);
  if (p.vpt != 0) return static_cast<int>(p.grid);
  return static_cast<int>(c.rows < 4 * kSms ? c.rows : 4 * kSms);
}

// The blocks grow with the rows but for one step down: from 152 times the groups of
// a block on, a block has several groups (shape_common).
int norm_backward_ctas_most(const moe_norm_config& c) {
  moe_norm_config d = c;
  int most = 0;
  for (const int dtype : {MOE_F32, MOE_BF16}) {
    d.dtype = dtype;
    for (const int64_t groups : {2, 4, 8, 0}) {
      const int64_t before = kSms * groups - 1;
      d.rows = groups != 0 && before < c.rows ? before : c.rows;
      const int ctas = norm_backward_ctas(d);
      most = ctas > most ? ctas : most;
    }
  }
  return most;
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
  return launch_dependent(norm_param_grads_kernel, dim3((c.hidden + 31) / 32, 2),
                          dim3(kGradWarps * 32), 0, s, norm_backward_ctas(c), c.hidden,
                          static_cast<const float*>(part), dweight, dbias);
}

template <typename T>
cudaError_t dropout_add_typed(int64_t n, const Dropout& d, const uint64_t* rng, const void* x,
                              const void* residual, void* y, cudaStream_t s) {
  const int64_t blocks = (n / Lanes<T>::V + 256) / 256;
  const unsigned grid = static_cast<unsigned>(blocks < kSms * 8 ? blocks : kSms * 8);
  auto k = d.on ? dropout_add_kernel<T, true> : dropout_add_kernel<T, false>;
  k<<<grid, 256, 0, s>>>(n, d, rng, static_cast<const T*>(x), static_cast<const T*>(residual),
                         static_cast<T*>(y));
  return cudaGetLastError();
}

cudaError_t launch_dropout_add(int64_t n, int dtype, double p, const uint64_t* rng, const void* x,
                               const void* residual, void* y, cudaStream_t s) {
  if (n == 0) return cudaSuccess;
  const Dropout d = dropout_of(p);
  return dtype == MOE_F32 ? dropout_add_typed<float>(n, d, rng, x, residual, y, s)
                          : dropout_add_typed<__nv_bfloat16>(n, d, rng, x, residual, y, s);
}

}  // namespace moe
