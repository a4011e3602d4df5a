// The next token of each row of logits from a given random number: temperature,
// top-k, top-p, min-p.
//
// With m the row's largest logit, token i has the weight w_i = exp((l_i - m) / t),
// held as a whole number of 2^-40: sums of them do not depend on their order, so
// every split of a row gives the same token.  Tokens are ordered by logit, equal
// ones by index (the lower first); the kept ones are the first n of that order,
// bounded by top-k, then by top-p of the mass that top-k left, and those with w_i >=
// min_p.  The token is the lowest index whose running sum of kept weights exceeds u
// times their total.
//
// A row belongs to a cluster of up to 16 blocks, which hold it in their shared memory
// from its only read to the end (rows too long for that, or too many, are read again from
// L2).  With a top-k of up to 1200 (or with 2048 tokens in all) the largest logits of the
// threads' tokens give a threshold above which there are that many and few more; those
// are gathered and sorted by one block, which draws the token.  Otherwise one pass counts
// tokens and adds weights up in 1024 bins of 1/32 of a nat below the largest; the bin that
// a border falls into is gathered and sorted, by its exact order (a bin with more than
// 2048 tokens is first narrowed down by further passes over ever finer ranges of that
// order).
//
// What bounds it: a row's latency (load, passes with cluster barriers, sorts), not memory.
// One row of 128000 fp32 takes 25 us with a top-p, 15 with a top-k of 50 beside it, 27 with
// one of 1000, 5 greedy (its bytes at the copy rate 0.1); 64 of 151936 bf16 with a top-k, top-p
// and min-p 23 (bytes 3).  Without a top-k the 64 take longer, as all tokens are weighed:
// 48 with a temperature alone, 57 with a min-p (a pass of weights, then one warp that goes
// over its run again for the token), and 103 to 110 with a top-p (four additions in shared
// memory a token, the border's bin searched for in further passes; integer instructions
// mostly, 58% of the issue slots).
#include <float.h>
#include <math.h>

#include "common.cuh"
#include "sm100_ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
static_assert(kWarps == 32, "a warp looks at all warps' sums");
constexpr int kBins = 1024, kList = 2 * kThreads;
// The top-k that is looked for among the threads' largest logits.  With n threads that hold
// 3 k or more tokens at random, the k-th largest of those n has about -n ln(1 - k / n) <=
// 1.22 k tokens above it, a few more for the bin that it falls into: of 1200, 1460 and
// what the bin adds (up to 2048 are listed, else the row goes the general way after all).
// Gathered and the general way, top-k 50 / 600 / 900 / 1200 / 1600 with a top-p, 1 x 128000
// of spread 2.5: 14.6 / 21 / 24 / 29 / 35 us and 29 / 30 / 30 / 31 / 29 (of spread 1: 15 /
// 23 / 24 / 34 / 35 and 30 / 31 / 30 / 31 / 33; 12 x 151936: 16 / 24 / 25 / 31 / 36 and 42).
constexpr int kLikely = 1200;
constexpr float kBinsPerNat = 32.f;
constexpr float kOne = 1099511627776.f;  // 2^40
constexpr int kMaxBlocks = 16;           // of a cluster
constexpr size_t kMaxData = 152 * 1024;  // bytes of a block's part of a row
constexpr int kFewest = 2048;            // tokens of a block, where a row is split
constexpr int kSumBy32 = 4095;           // tokens of a thread whose halves add up in 32 bits

typedef unsigned long long u64;

struct Args {
  int64_t rows, V;
  int part;          // tokens of a block
  bool held;         // in shared memory
  const void* logits;
  const float* u;
  SampleChoices c;
  int32_t* tokens;
  float* prob;
};

struct Result {       // of a search, written by block 0 to every block
  u64 last;           // the order of the last token kept
  u64 mass;           // of the kept ones
};

struct Shared {
  uint32_t count[kBins];   // this block's
  u64 mass[kBins];
  uint32_t counts[kBins];  // the row's
  u64 masses[kBins];
  u64 list[kList];         // block 0's
  union {
    struct {
      u64 sums[kList];     // running sums of its weights
      u64 own[kList];      // what this block adds to it
    };
    struct {
      uint32_t pieces[3][kBins];    // of the masses while they are added up, 15 bits each
      uint32_t fine_counts[kBins];  // the row's, of a narrowed range
      u64 fine_masses[kBins];
    };
  };
  uint32_t listed, owned, base;
  u64 warp_sum[kWarps];
  uint32_t warp_count[kWarps];
  float warp_max[kWarps];
  // what the blocks tell one another, an entry each
  float max_of[kMaxBlocks];
  u64 sum_of[kMaxBlocks];
  u64 low_of[kMaxBlocks], high_of[kMaxBlocks];
  uint32_t first_of[kMaxBlocks];
  Result result;
  // of a scan over the bins
  int bin;
  uint32_t count_above;
  u64 mass_above;
};

constexpr size_t kShared = (sizeof(Shared) + 15) / 16 * 16;
static_assert(kShared + kMaxData <= 227 * 1024, "shared memory");

// ------------------------------------------------------------------ other blocks
__device__ __forceinline__ uint32_t there(const void* p, int rank) {
  return ptx::mapa_shared(ptx::smem_u32(p), rank);
}
__device__ __forceinline__ void put(uint32_t at, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ void put(uint32_t at, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(v) : "memory");
}
__device__ __forceinline__ void put(uint32_t at, float v) { put(at, __float_as_uint(v)); }
__device__ __forceinline__ uint32_t get32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ u64 get64(uint32_t at) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t add32(uint32_t at, uint32_t v) {
  uint32_t old;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(at), "r"(v) : "memory");
  return old;
}

__device__ __forceinline__ void sync_cluster() {
  __syncwarp();
  ptx::cluster_sync();
}

// A logit's place in the order: larger, earlier.  NaN and -infinity have none (0).
__device__ __forceinline__ uint32_t key_of(float l) {
  if (!(l > -INFINITY)) return 0u;
  uint32_t b = __float_as_uint(l);
  if (b == 0x80000000u) b = 0u;  // -0 is 0
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key & 0x7fffffffu : ~key);
}
// the same with the index: no two tokens of a row are equal
__device__ __forceinline__ u64 order_of(uint32_t key, uint32_t i) {
  return static_cast<u64>(key) << 32 | (0xffffffffu - i);
}

struct Scale {
  float max, inverse;  // 1 / t
  __device__ __forceinline__ float below(float l) const {  // in nats, >= 0
    return l == max ? 0.f : (max - l) * inverse;
  }
  __device__ __forceinline__ float weight(float l) const { return expf(-below(l)); }
};
// w 2^40 for 0 <= w <= 1 as a whole number: its upper part, 2^20 at most, and 20 bits
// (rounded, so 2^20 at most too)
__device__ __forceinline__ void whole(float w, uint32_t& hi, uint32_t& lo) {
  const float v = w * 0x1p20f;  // exact
  hi = __float2uint_rd(v);
  lo = __float2uint_rn((v - __uint2float_rn(hi)) * 0x1p20f);
}
__device__ __forceinline__ u64 whole(float w) {
  uint32_t hi, lo;
  whole(w, hi, lo);
  return (static_cast<u64>(hi) << 20) + lo;
}
// A bin's mass from this block: whole numbers of 41 bits in pieces of 15, whose sums
// over 2^17 tokens stay in 32 bits, since the 64-bit addition in shared memory is a
// loop.
__device__ __forceinline__ void add_mass(Shared& s, int bin, u64 w, bool pieces) {
  if (!pieces) {
    atomicAdd(&s.mass[bin], w);
    return;
  }
  const uint32_t low = static_cast<uint32_t>(w), lo = low & 0x7fffu, mid = low >> 15 & 0x7fffu;
  const uint32_t hi = static_cast<uint32_t>(w >> 30);
  if (lo) atomicAdd(&s.pieces[0][bin], lo);
  if (mid) atomicAdd(&s.pieces[1][bin], mid);
  if (hi) atomicAdd(&s.pieces[2][bin], hi);
}
__device__ void clear_bins(Shared& s) {
  __syncthreads();
  for (int i = threadIdx.x; i < kBins; i += kThreads) {
    s.count[i] = 0, s.mass[i] = 0;
    s.pieces[0][i] = s.pieces[1][i] = s.pieces[2][i] = 0;
  }
  __syncthreads();
}
__device__ void join_pieces(Shared& s) {
  __syncthreads();
  for (int i = threadIdx.x; i < kBins; i += kThreads)
    s.mass[i] += s.pieces[0][i] + (static_cast<u64>(s.pieces[1][i]) << 15) +
                 (static_cast<u64>(s.pieces[2][i]) << 30);
}
__device__ __forceinline__ int bin_of(float below) {
  return static_cast<int>(fminf(below * kBinsPerNat, static_cast<float>(kBins - 1)));
}

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

__device__ __forceinline__ u64 warp_total(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// The blocks' bins added up, in every block.
template <bool MASS>
__device__ void merge(Shared& s, int rank, int blocks, uint32_t* counts, u64* masses) {
  sync_cluster();
  const int each = kBins / blocks;
  for (int i = rank * each + threadIdx.x; i < (rank + 1) * each; i += kThreads) {
    // all blocks' at a time, so that their latencies are one
    uint32_t cs[kMaxBlocks], c = 0;
    u64 ms[kMaxBlocks], m = 0;
#pragma unroll
    for (int b = 0; b < kMaxBlocks; ++b) {
      cs[b] = b < blocks ? get32(there(&s.count[i], b)) : 0u;
      ms[b] = MASS && b < blocks ? get64(there(&s.mass[i], b)) : 0ull;
    }
#pragma unroll
    for (int b = 0; b < kMaxBlocks; ++b) c += cs[b], m += ms[b];
    for (int b = 0; b < blocks; ++b) {
      put(there(&counts[i], b), c);
      if (MASS) put(there(&masses[i], b), m);
    }
  }
  sync_cluster();
}

// The sums of the warps before this one, from s.warp_sum.
__device__ __forceinline__ u64 sums_before(const Shared& s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  return warp_total(lane < warp ? s.warp_sum[lane] : 0);
}

// The first of n entries (n <= 2048, 2 to a thread) at which the running sum of
// `value` reaches `want` (a count or a mass), or the last one of all: its number, and
// the sums before it, into s.  Called by the whole block.
template <typename Count, typename Mass, typename Reached>
__device__ void first_reached(Shared& s, int n, Count count, Mass mass, Reached reached) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i0 = threadIdx.x * 2;
  uint32_t c[2];
  u64 m[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    c[j] = i0 + j < n ? count(i0 + j) : 0u;
    m[j] = i0 + j < n ? mass(i0 + j) : 0ull;
  }
  uint32_t cs = c[0] + c[1];
  u64 ms = m[0] + m[1];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t co = __shfl_up_sync(~0u, cs, o);
    const u64 mo = __shfl_up_sync(~0u, ms, o);
    if (lane >= o) cs += co, ms += mo;
  }
  if (lane == 31) s.warp_count[warp] = cs, s.warp_sum[warp] = ms;
  if (threadIdx.x == 0) s.bin = n - 1;
  __syncthreads();
  cs += __reduce_add_sync(~0u, lane < warp ? s.warp_count[lane] : 0u);
  ms += sums_before(s);
  cs -= c[0] + c[1], ms -= m[0] + m[1];  // before this thread's two
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if (i0 + j < n && reached(cs + c[j], ms + m[j]) && !(reached(cs, ms))) s.bin = i0 + j;
    cs += c[j], ms += m[j];
  }
  __syncthreads();
  // the sums before it: its own thread knows them
  const int at = s.bin;
  if (at >= i0 && at < i0 + 2) {
    s.count_above = cs - c[1] - (at == i0 ? c[0] : 0u);
    s.mass_above = ms - m[1] - (at == i0 ? m[0] : 0ull);
  }
  __syncthreads();
}

// list[0 .. n) in descending order (bitonic; n a power of two from 64 on, kList at most):
// two entries to a thread, 64 to a warp, which orders those among itself.
__device__ void sort_descending(u64* list, int n) {
  const int lane = threadIdx.x & 31, first = (threadIdx.x >> 5) * 64 + lane;
  const bool active = first < n;
  u64 v[2] = {0, 0};
  __syncthreads();
  if (active) v[0] = list[first], v[1] = list[first + 32];
  auto keep = [](u64 mine, u64 other, bool larger) { return (mine > other) == larger ? mine : other; };
#pragma unroll 1
  for (int size = 2; size <= n; size *= 2) {
#pragma unroll 1
    for (int step = size / 2; step >= 64; step /= 2) {
      __syncthreads();
      if (active) list[first] = v[0], list[first + 32] = v[1];
      __syncthreads();
      if (active)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int e = first + j * 32;
          v[j] = keep(v[j], list[e ^ step], ((e & size) == 0) == ((e & step) == 0));
        }
    }
    if (!active) continue;
    if (size >= 64) {
      const bool down = (first & size) == 0;
      const u64 a = v[0], b = v[1];
      v[0] = keep(a, b, down), v[1] = keep(b, a, !down);
    }
#pragma unroll 1
    for (int step = min(size / 2, 16); step > 0; step /= 2)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int e = first + j * 32;
        const u64 other = __shfl_xor_sync(~0u, v[j], step);
        v[j] = keep(v[j], other, ((e & size) == 0) == ((e & step) == 0));
      }
  }
  __syncthreads();
  if (active) list[first] = v[0], list[first + 32] = v[1];
  __syncthreads();
}
__device__ __forceinline__ int sorted_size(int n) {
  int size = 64;
  while (size < n) size *= 2;
  return size;
}

// sums[i] = value(0) + .. + value(i), i < n <= kList
template <typename Value>
__device__ void running_sums(Shared& s, int n, Value value) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i0 = threadIdx.x * 2;
  const u64 a = i0 < n ? value(i0) : 0, b = i0 + 1 < n ? value(i0 + 1) : 0;
  u64 sum = a + b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 v = __shfl_up_sync(~0u, sum, o);
    if (lane >= o) sum += v;
  }
  if (lane == 31) s.warp_sum[warp] = sum;
  __syncthreads();
  sum += sums_before(s);
  if (i0 < n) s.sums[i0] = sum - b;
  if (i0 + 1 < n) s.sums[i0 + 1] = sum;
  __syncthreads();
}
// the first i < n at which sums[i] is past a border, or n
template <typename Past>
__device__ int first_past(Shared& s, int n, Past past) {
  if (threadIdx.x == 0) s.bin = n;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kList / kThreads; ++j) {
    const int i = threadIdx.x + j * kThreads;
    if (i < n && past(s.sums[i]) && (i == 0 || !past(s.sums[i - 1]))) s.bin = i;
  }
  __syncthreads();
  const int at = s.bin;
  __syncthreads();
  return at;
}

template <typename T>
struct Row {
  const T* at;      // this block's part, in shared memory or not
  int n;            // tokens of it
  int first;        // the first one's index in the row
  // a warp has a run of them, a token to a lane
  __device__ __forceinline__ int run() const { return (n + kWarps * 32 - 1) / (kWarps * 32) * 32; }
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int end = min(n, (warp + 1) * run());
#pragma unroll 4
    for (int i = warp * run() + lane; i < end; i += 32) f(to_float(at[i]), first + i);
  }
};

// The orders of the tokens of at least `least` for which `in` holds, into block 0's
// list; s.listed, there, says how many there are (0 before, which a cluster barrier has
// made known).  Four tokens of a lane are looked at
// together, as mostly none is wanted.
template <typename T, typename In>
__device__ void gather(Shared& s, const Row<T>& row, int blocks, float least, In in) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) s.owned = 0;
  __syncthreads();
  const int run = row.run(), end = min(row.n, (warp + 1) * run);
  for (int i0 = warp * run + lane; i0 < (warp + 1) * run; i0 += 128) {
    float l[4];
    bool any = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      l[j] = i0 + j * 32 < end ? to_float(row.at[i0 + j * 32]) : -INFINITY;
      any |= l[j] >= least;
    }
    if (!any) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = row.first + i0 + j * 32;
      if (l[j] >= least && in(l[j], i)) {
        const uint32_t at = atomicAdd(&s.owned, 1u);
        if (at < kList) s.own[at] = order_of(key_of(l[j]), i);
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) s.base = add32(there(&s.listed, 0), s.owned);
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < s.owned && s.base + i < kList; i += kThreads)
    put(there(&s.list[s.base + i], 0), s.own[i]);
  sync_cluster();
}

// Which of the tokens with orders in [low, high) is the one at which the running sum
// reaches what is wanted, counting from the sums `above` those.
template <typename T, typename In, typename Reached>
__device__ Result search(Shared& s, const Row<T>& row, int rank, int blocks, bool pieces,
                         const Scale& scale,
                         uint32_t n, uint32_t count_above, u64 mass_above, In in,
                         Reached reached) {
  u64 low = 0, high = ~0ull;  // of the tokens that are `in`
  if (n > kList) {
    u64 lo = ~0ull, hi = 0;
    row.each([&](float l, int i) {
      if (in(l)) {
        const u64 o = order_of(key_of(l), i);
        lo = min(lo, o), hi = max(hi, o);
      }
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      lo = min(lo, __shfl_xor_sync(~0u, lo, o));
      hi = max(hi, __shfl_xor_sync(~0u, hi, o));
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s.list[threadIdx.x >> 5] = lo, s.list[kWarps + (threadIdx.x >> 5)] = hi;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < kWarps; ++w) lo = min(lo, s.list[w]), hi = max(hi, s.list[kWarps + w]);
      for (int b = 0; b < blocks; ++b) {
        put(there(&s.low_of[rank], b), lo);
        put(there(&s.high_of[rank], b), hi);
      }
    }
    sync_cluster();
    low = ~0ull, high = 0;
    for (int b = 0; b < blocks; ++b) low = min(low, s.low_of[b]), high = max(high, s.high_of[b]);
    while (n > kList) {
      // 1024 equal ranges of [low, high], the highest first
      int shift = 0;
      while (((high - low) >> shift) >= kBins) ++shift;
      clear_bins(s);
      row.each([&](float l, int i) {
        if (!in(l)) return;
        const u64 o = order_of(key_of(l), i);
        if (o < low || o > high) return;
        const int b = static_cast<int>((high - o) >> shift);
        atomicAdd(&s.count[b], 1u);
        add_mass(s, b, whole(scale.weight(l)), pieces);
      });
      join_pieces(s);
      merge<true>(s, rank, blocks, s.fine_counts, s.fine_masses);
      first_reached(
          s, kBins, [&](int i) { return s.fine_counts[i]; },
          [&](int i) { return s.fine_masses[i]; },
          [&](uint32_t c, u64 m) { return reached(count_above + c, mass_above + m); });
      count_above += s.count_above, mass_above += s.mass_above;
      n = s.fine_counts[s.bin];
      const u64 top = high - (static_cast<u64>(s.bin) << shift);
      const u64 width = (u64{1} << shift) - 1;
      low = top - low > width ? top - width : low;
      high = top;
      __syncthreads();
    }
  }
  // the rest into block 0's list
  gather(s, row, blocks, -FLT_MAX, [&](float l, int i) {
    if (!in(l)) return false;
    const u64 o = order_of(key_of(l), i);
    return o >= low && o <= high;
  });
  if (rank == 0) {
    const int got = min(static_cast<int>(s.listed), kList), size = sorted_size(got);
    __syncthreads();
    if (threadIdx.x == 0) s.listed = 0;
    for (int i = got + threadIdx.x; i < size; i += kThreads) s.list[i] = 0;
    sort_descending(s.list, size);
    auto mass = [&](int i) { return whole(scale.weight(logit_of(static_cast<uint32_t>(s.list[i] >> 32)))); };
    first_reached(
        s, got, [&](int) { return 1u; }, mass,
        [&](uint32_t c, u64 m) { return reached(count_above + c, mass_above + m); });
    if (threadIdx.x == 0) {
      const u64 last = s.list[s.bin], sum = mass_above + s.mass_above + mass(s.bin);
      for (int b = 0; b < blocks; ++b) {
        put(there(&s.result.last, b), last);
        put(there(&s.result.mass, b), sum);
      }
    }
  }
  sync_cluster();
  const Result r = s.result;
  __syncthreads();
  return r;
}

// Block 0: the token, if the gathered ones are enough.  The list has all tokens from some
// logit on, or all there are.
__device__ bool draw_likely(Shared& s, const Args& a, int64_t r, const Scale& scale, int k,
                            float top_p, float min_p, float u) {
  const bool all = a.V <= kList;
  const uint32_t listed = s.listed;
  __syncthreads();
  if (threadIdx.x == 0) s.listed = 0;
  if (listed > kList || (!all && k > 0 && listed < static_cast<uint32_t>(k))) return false;
  int n = static_cast<int>(listed);
  auto weight = [&](uint32_t key) { return scale.weight(logit_of(key)); };
  int size = sorted_size(n);
  for (int i = n + threadIdx.x; i < size; i += kThreads) s.list[i] = 0;
  sort_descending(s.list, size);
  if (k > 0) n = min(n, k);
  if (top_p < 1.f) {
    running_sums(s, n, [&](int i) { return whole(weight(static_cast<uint32_t>(s.list[i] >> 32))); });
    const double want =
        static_cast<double>(fmaxf(top_p, 0.f)) * static_cast<double>(s.sums[n - 1]);
    n = min(n, first_past(s, n, [&](u64 m) { return static_cast<double>(m) >= want; }) + 1);
  }
  // in index order: the list anew with the index in front
  u64 mine[kList / kThreads];
#pragma unroll
  for (int j = 0; j < kList / kThreads; ++j) {
    const int i = j * kThreads + threadIdx.x;
    mine[j] = i < n ? s.list[i] << 32 | s.list[i] >> 32 : 0;
  }
  __syncthreads();
  size = sorted_size(n);
#pragma unroll
  for (int j = 0; j < kList / kThreads; ++j)
    if (j * kThreads + static_cast<int>(threadIdx.x) < size) s.list[j * kThreads + threadIdx.x] = mine[j];
  sort_descending(s.list, size);
  running_sums(s, n, [&](int i) {
    const float w = weight(static_cast<uint32_t>(s.list[i]));
    return w >= min_p ? whole(w) : u64{0};
  });
  const u64 total = s.sums[n - 1];
  const double at = static_cast<double>(u) * static_cast<double>(total);
  const int i = first_past(s, n, [&](u64 m) { return static_cast<double>(m) > at; });
  if (threadIdx.x == 0) {
    a.tokens[r] = static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(s.list[i] >> 32));
    if (a.prob)
      a.prob[r] = static_cast<float>(static_cast<double>(weight(static_cast<uint32_t>(s.list[i]))) *
                                     kOne / static_cast<double>(total));
  }
  return true;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(const __grid_constant__ Args a) {
  extern __shared__ __align__(16) char smem[];
  Shared& s = *reinterpret_cast<Shared*>(smem);
  char* data = smem + kShared;
  const int blocks = gridDim.x, rank = blockIdx.x;  // the cluster is a row of the grid
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t r = blockIdx.y + static_cast<int64_t>(blockIdx.z) * 65535;
  if (r >= a.rows) return;  // the whole cluster
  // Another block's shared memory is there once that block has begun: waited for before
  // the first store into it.
  ptx::cluster_arrive();
  Row<T> row;
  const int64_t begin = min(a.V, static_cast<int64_t>(rank) * a.part);
  row.first = static_cast<int>(begin);
  row.n = static_cast<int>(min(a.V, begin + a.part) - begin);
  const T* src = static_cast<const T*>(a.logits) + r * a.V + begin;
  row.at = src;
  if (a.held && row.n > 0) {
    // 16-byte pieces of the whole tensor; its own last piece, where it is none, by token
    const uint64_t at = static_cast<uint64_t>(r * a.V + begin) * sizeof(T);
    const uint64_t end = at + static_cast<uint64_t>(row.n) * sizeof(T);
    const uint64_t all = static_cast<uint64_t>(a.rows) * a.V * sizeof(T);
    const uint64_t from = at & ~uint64_t{15}, to = min((end + 15) & ~uint64_t{15}, all & ~uint64_t{15});
    const char* base = static_cast<const char*>(a.logits);
    for (uint64_t p = from + threadIdx.x * 16; p < to; p += kThreads * 16)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                       ptx::smem_u32(data + (p - from))),
                   "l"(base + p)
                   : "memory");
    for (uint64_t p = max(to, at) + threadIdx.x * sizeof(T); p < end; p += kThreads * sizeof(T))
      *reinterpret_cast<T*>(data + (p - from)) = *reinterpret_cast<const T*>(base + p);
    asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
    row.at = reinterpret_cast<const T*>(data + (at - from));
  }
  float t = a.c.temperature_of ? a.c.temperature_of[r] : a.c.temperature;
  int k = a.c.top_k_of ? a.c.top_k_of[r] : a.c.top_k;
  const float top_p = a.c.top_p_of ? a.c.top_p_of[r] : a.c.top_p;
  float min_p = a.c.min_p_of ? a.c.min_p_of[r] : a.c.min_p;
  const float u = fminf(fmaxf(a.u[r], 0.f), 0x1.fffffep-1f);  // NaN: 0
  min_p = min_p > 0.f ? fminf(min_p, 1.f) : 0.f;
  if (k >= a.V) k = 0;
  if (threadIdx.x == 0) s.listed = 0;
  __syncthreads();

  // the largest logit
  float top = -INFINITY;
  row.each([&](float l, int) { top = fmaxf(top, l); });  // NaN: none
  const float mine = top;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
  if (lane == 0) s.warp_max[warp] = top;
  __syncthreads();
  ptx::cluster_wait();
  if (warp == 0) {
    top = s.warp_max[lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    if (lane < blocks) put(there(&s.max_of[rank], lane), top);
  }
  sync_cluster();
  Scale scale;
  scale.max = s.max_of[0];
  for (int b = 1; b < blocks; ++b) scale.max = fmaxf(scale.max, s.max_of[b]);
  // past 1e30 all finite logits of any use weigh the same
  scale.inverse = 1.f / fminf(t, 1e30f);

  const bool none = scale.max == -INFINITY;
  const bool greedy = !(t > 0.f) || k == 1;
  if (none || greedy) {
    uint32_t best = 0xffffffffu;
    if (!none)
      row.each([&](float l, int i) {
        if (l == scale.max) best = min(best, static_cast<uint32_t>(i));
      });
    best = __reduce_min_sync(~0u, best);
    if (lane == 0) s.warp_count[warp] = best;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 0; w < kWarps; ++w) best = min(best, s.warp_count[w]);
      put(there(&s.first_of[rank], 0), best);
    }
    sync_cluster();
    if (rank == 0 && threadIdx.x == 0) {
      for (int b = 0; b < blocks; ++b) best = min(best, s.first_of[b]);
      a.tokens[r] = static_cast<int32_t>(best);  // none: -1
      if (a.prob) a.prob[r] = none ? 0.f : 1.f;
    }
    return;
  }

  u64 last = 0;  // orders from there on are kept
  const bool by_p = top_p < 1.f;
  if (k > 0 || by_p) {
    const bool pieces = a.part <= 1 << 17;
    // Few tokens, or a top-k: those that it can be about are gathered at once.
    // (the threshold is one of the threads' largest logits: of three times as many threads)
    if (a.V <= kList || (k > 0 && k <= min(kLikely, blocks * kThreads / 3))) {
      float least = -FLT_MAX;
      if (a.V > kList) {
        for (int i = threadIdx.x; i < kBins; i += kThreads) s.count[i] = 0;
        __syncthreads();
        if (mine > -INFINITY) atomicAdd(&s.count[bin_of(scale.below(mine))], 1u);
        merge<false>(s, rank, blocks, s.counts, s.masses);
        const uint32_t want = k;
        first_reached(
            s, kBins, [&](int i) { return s.counts[i]; }, [](int) { return u64{0}; },
            [=](uint32_t c, u64) { return c >= want; });
        // the bin's lower end; any threshold would do, the same in every block
        least = scale.max - static_cast<float>(s.bin + 1) / (kBinsPerNat * scale.inverse);
      }
      gather(s, row, blocks, least, [](float, int) { return true; });
      if (rank == 0) {
        const bool drawn = draw_likely(s, a, r, scale, k, top_p, min_p, u);
        if (threadIdx.x < blocks) put(there(&s.first_of[0], threadIdx.x), drawn ? 1u : 0u);
      }
      sync_cluster();
      if (s.first_of[0]) return;
    }

    clear_bins(s);
    row.each([&](float l, int) {
      if (!(l > -INFINITY)) return;
      const float below = scale.below(l);
      const int b = bin_of(below);
      atomicAdd(&s.count[b], 1u);
      if (by_p) add_mass(s, b, whole(expf(-below)), pieces);
    });
    join_pieces(s);
    merge<true>(s, rank, blocks, s.counts, s.masses);
    auto in_bin = [&](int bin) {
      return [=](float l) { return l > -INFINITY && bin_of(scale.below(l)) == bin; };
    };
    auto find = [&](auto reached) {
      first_reached(
          s, kBins, [&](int i) { return s.counts[i]; }, [&](int i) { return s.masses[i]; }, reached);
      const int bin = s.bin;
      const uint32_t ca = s.count_above, n = s.counts[bin];
      const u64 ma = s.mass_above;
      __syncthreads();
      return search(s, row, rank, blocks, pieces, scale, n, ca, ma, in_bin(bin), reached);
    };
    // all of them, where top-k leaves them
    u64 mass = 0;
    uint32_t tokens = 0;
    for (int i = threadIdx.x; i < kBins; i += kThreads) tokens += s.counts[i], mass += s.masses[i];
    mass = warp_total(mass);
    tokens = __reduce_add_sync(~0u, tokens);
    if (lane == 0) s.warp_sum[warp] = mass, s.warp_count[warp] = tokens;
    __syncthreads();
    mass = warp_total(s.warp_sum[lane]);
    tokens = __reduce_add_sync(~0u, s.warp_count[lane]);
    __syncthreads();
    if (k > 0 && static_cast<uint32_t>(k) < tokens) {
      const uint32_t want = k;
      const Result f = find([=](uint32_t c, u64) { return c >= want; });
      last = f.last;
      mass = f.mass;
    }
    if (by_p) {
      const double want = static_cast<double>(fmaxf(top_p, 0.f)) * static_cast<double>(mass);
      const Result f = find([=](uint32_t c, u64 m) { return c > 0 && static_cast<double>(m) >= want; });
      last = max(last, f.last);
    }
  }

  // the kept weights
  auto kept = [&](float l, int i, float& w) {
    const uint32_t key = key_of(l);
    if (key == 0u || order_of(key, i) < last) return u64{0};
    w = scale.weight(l);
    return w >= min_p ? whole(w) : u64{0};
  };
  u64 sum = 0;
  float w;
  if (last == 0 && min_p <= 0.f && a.part <= kThreads * kSumBy32) {
    // all of them, a thread's halves apart: 2^20 each at most
    static_assert(static_cast<u64>(kSumBy32) << 20 < u64{1} << 32, "sums of halves");
    uint32_t his = 0, los = 0;
    row.each([&](float l, int) {
      uint32_t hi, lo;
      whole(l > -INFINITY ? scale.weight(l) : 0.f, hi, lo);
      his += hi, los += lo;
    });
    sum = (static_cast<u64>(his) << 20) + los;
  } else {
    row.each([&](float l, int i) { sum += kept(l, i, w); });
  }
  sum = warp_total(sum);
  if (lane == 0) s.warp_sum[warp] = sum;
  __syncthreads();
  if (warp == 0) {
    sum = warp_total(s.warp_sum[lane]);
    if (lane < blocks) put(there(&s.sum_of[rank], lane), sum);
  }
  sync_cluster();
  u64 before = 0, total = 0;
  for (int b = 0; b < blocks; ++b) {
    if (b < rank) before += s.sum_of[b];
    total += s.sum_of[b];
  }
  const double at = static_cast<double>(u) * static_cast<double>(total);
  auto past = [&](u64 v) { return static_cast<double>(v) > at; };
  before += sums_before(s);
  if (past(before) || !past(before + s.warp_sum[warp])) return;
  // this warp's run has the token
  const int run = row.run();
  const int end = min(row.n, (warp + 1) * run);
  for (int i0 = warp * run; i0 < end; i0 += 32) {
    const int i = i0 + lane;
    u64 mine = 0;
    if (i < end) mine = kept(to_float(row.at[i]), row.first + i, w);
    u64 incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 v = __shfl_up_sync(~0u, incl, o);
      if (lane >= o) incl += v;
    }
    const uint32_t hit = __ballot_sync(~0u, past(before + incl));
    if (hit) {
      if (lane == __ffs(hit) - 1) {
        a.tokens[r] = row.first + i;
        if (a.prob) a.prob[r] = static_cast<float>(static_cast<double>(w) * kOne / static_cast<double>(total));
      }
      return;
    }
    before += __shfl_sync(~0u, incl, 31);
  }
}

// How many clusters of 2, 4, 8 and 16 blocks the device runs at a time (0 for sizes that
// it does not take), a block to an SM; looked up once for a kernel and device.
struct AtOnce {
  std::atomic<bool> known;
  std::atomic<int> clusters[4];
};
template <auto KERNEL>
cudaError_t clusters_at_once(const AtOnce** out) {
  static AtOnce devices[64];
  int device = 0;
  cudaError_t st = cudaGetDevice(&device);
  if (st != cudaSuccess) return st;
  AtOnce& d = devices[device & 63];
  if (!d.known.load(std::memory_order_acquire)) {
    st = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (st != cudaSuccess) return st;
    for (int i = 0; i < 4; ++i) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(2 << i);
      cfg.blockDim = dim3(kThreads);
      cfg.dynamicSmemBytes = kShared + kMaxData;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = 2 << i;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, KERNEL, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        n = 0;
      }
      d.clusters[i].store(n, std::memory_order_relaxed);
    }
    d.known.store(true, std::memory_order_release);
  }
  *out = &d;
  return cudaSuccess;
}

template <typename T>
cudaError_t launch(Args& a, cudaStream_t s) {
  cudaError_t st = allow_most_smem<sample_kernel<T>>();
  if (st != cudaSuccess) return st;
  const AtOnce* at_once = nullptr;
  st = clusters_at_once<sample_kernel<T>>(&at_once);
  if (st != cudaSuccess) return st;
  // More blocks to a row as long as there is work for each and all rows run at once: 16 x
  // 151936 fp32, top-k 50, in fours 20.6 us, in eights (not all at once) 34.8; 12 x 151936
  // bf16, top-p, in eights 42 and in fours 64; one row of 128000 in sixteens 27, in eights 33.
  // Rows that do not fit into shared memory so are read again from L2: 64 x 151936 fp32 in
  // twos 24.7 us with top-k 50 and 131 with top-p, held by fours in two rounds 39 and 117.
  int blocks = 1;
  for (int i = 0; i < 4; ++i) {
    const int next = 2 << i;
    if (a.V / next < kFewest || a.rows > at_once->clusters[i].load(std::memory_order_relaxed)) break;
    blocks = next;
  }
  a.part = static_cast<int>((a.V + blocks - 1) / blocks);
  const size_t bytes = static_cast<size_t>(a.part) * sizeof(T) + 32;
  a.held = bytes <= kMaxData;
  cudaLaunchConfig_t cfg = {};
  const unsigned ys = static_cast<unsigned>(a.rows < 65535 ? a.rows : 65535);
  cfg.gridDim = dim3(blocks, ys, static_cast<unsigned>((a.rows + 65534) / 65535));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kShared + (a.held ? bytes : 0);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = blocks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sample_kernel<T>, static_cast<const Args>(a));
}

}  // namespace

cudaError_t launch_sample(int64_t rows, int V, int dtype, const void* logits, const float* u,
                          const SampleChoices& c, int32_t* tokens, float* prob, cudaStream_t s) {
  Args a;
  a.rows = rows, a.V = V;
  a.logits = logits, a.u = u, a.c = c, a.tokens = tokens, a.prob = prob;
  return dtype == MOE_F32 ? launch<float>(a, s) : launch<__nv_bfloat16>(a, s);
}

}  // namespace moe
