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
// A row belongs to a cluster of up to 8 blocks, which hold it in their shared memory
// from its only read to the end (rows too long for that are read again from L2).
// Instead of a sort, one pass counts tokens and adds weights up in 1024 bins of 1/32
// of a nat below the largest; only the bin that a border falls into is gathered and
// sorted, by its exact order (a bin with more than 1024 tokens is first narrowed
// down by further passes over ever finer ranges of that order).  What bounds it: a
// row's latency (load, five to seven passes with a cluster barrier each), not
// memory.
#include <math.h>

#include "common.cuh"
#include "sm100_ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 1024, kList = 1024;
constexpr float kBinsPerNat = 32.f;
constexpr float kOne = 1099511627776.f;  // 2^40
constexpr int kMaxBlocks = 8;            // of a cluster
constexpr size_t kMaxData = 176 * 1024;  // bytes of a block's part of a row
constexpr int kFewest = 2048;            // tokens of a block, where a row is split

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
  uint32_t fine_counts[kBins];  // the row's, of a narrowed range
  u64 fine_masses[kBins];
  u64 list[kList];         // block 0's
  uint32_t listed;
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
  float max, t;
  __device__ __forceinline__ float below(float l) const {  // in nats, >= 0
    return l == max ? 0.f : (max - l) / t;
  }
  __device__ __forceinline__ float weight(float l) const { return expf(-below(l)); }
};
__device__ __forceinline__ u64 whole(float w) { return __float2ull_rn(w * kOne); }
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
__device__ void merge(Shared& s, int rank, int blocks, uint32_t* counts, u64* masses) {
  sync_cluster();
  const int each = kBins / blocks;
  for (int i = rank * each + threadIdx.x; i < (rank + 1) * each; i += kThreads) {
    uint32_t c = 0;
    u64 m = 0;
    for (int b = 0; b < blocks; ++b) {
      c += get32(there(&s.count[i], b));
      m += get64(there(&s.mass[i], b));
    }
    for (int b = 0; b < blocks; ++b) {
      put(there(&counts[i], b), c);
      put(there(&masses[i], b), m);
    }
  }
  sync_cluster();
}

// The first of n entries (n <= 1024, 2 to a thread) at which the running sum of
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
  uint32_t cb = 0;
  u64 mb = 0;
  for (int w = 0; w < warp; ++w) cb += s.warp_count[w], mb += s.warp_sum[w];
  cs += cb, ms += mb;
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

// list[0 .. n) in descending order, n a power of two
__device__ void sort_descending(u64* list, int n) {
  for (int size = 2; size <= n; size *= 2)
    for (int step = size / 2; step > 0; step /= 2) {
      __syncthreads();
      for (int i = threadIdx.x; i < n / 2; i += kThreads) {
        const int a = 2 * i - (i & (step - 1)), b = a + step;
        const bool down = (a & size) == 0;
        const u64 x = list[a], y = list[b];
        if ((x < y) == down) list[a] = y, list[b] = x;
      }
    }
  __syncthreads();
}

template <typename T>
struct Row {
  const T* at;      // this block's part, in shared memory or not
  int n;            // tokens of it
  int first;        // the first one's index in the row
  // a warp has a run of them, a token to a lane
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int run = (n + kWarps * 32 - 1) / (kWarps * 32) * 32;
    const int end = min(n, (warp + 1) * run);
#pragma unroll 4
    for (int i = warp * run + lane; i < end; i += 32) f(to_float(at[i]), first + i);
  }
};

// Which of the tokens with orders in [low, high) is the one at which the running sum
// reaches what is wanted, counting from the sums `above` those.
template <typename T, typename In, typename Reached>
__device__ Result search(Shared& s, const Row<T>& row, int rank, int blocks, const Scale& scale,
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
      __syncthreads();
      for (int i = threadIdx.x; i < kBins; i += kThreads) s.count[i] = 0, s.mass[i] = 0;
      __syncthreads();
      row.each([&](float l, int i) {
        if (!in(l)) return;
        const u64 o = order_of(key_of(l), i);
        if (o < low || o > high) return;
        const int b = static_cast<int>((high - o) >> shift);
        atomicAdd(&s.count[b], 1u);
        atomicAdd(&s.mass[b], whole(scale.weight(l)));
      });
      merge(s, rank, blocks, s.fine_counts, s.fine_masses);
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
  if (threadIdx.x == 0) s.listed = 0;
  sync_cluster();
  row.each([&](float l, int i) {
    if (!in(l)) return;
    const u64 o = order_of(key_of(l), i);
    if (o < low || o > high) return;
    const uint32_t at = add32(there(&s.listed, 0), 1u);
    if (at < kList) put(there(&s.list[min(at, static_cast<uint32_t>(kList - 1))], 0), o);
  });
  sync_cluster();
  if (rank == 0) {
    const int got = min(static_cast<int>(s.listed), kList);
    int size = 32;
    while (size < got) size *= 2;
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

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(const __grid_constant__ Args a) {
  extern __shared__ __align__(16) char data[];
  __shared__ Shared s;
  const int blocks = gridDim.x, rank = blockIdx.x;  // the cluster is a row of the grid
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t r = blockIdx.y + static_cast<int64_t>(blockIdx.z) * 65535;
  if (r >= a.rows) return;  // the whole cluster
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
  __syncthreads();

  // the largest logit
  float top = -INFINITY;
  row.each([&](float l, int) { top = fmaxf(top, l); });  // NaN: none
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
  if (lane == 0) s.warp_max[warp] = top;
  __syncthreads();
  if (threadIdx.x < blocks) {
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s.warp_max[w]);
    put(there(&s.max_of[rank], threadIdx.x), top);
  }
  sync_cluster();
  Scale scale;
  scale.max = s.max_of[0];
  for (int b = 1; b < blocks; ++b) scale.max = fmaxf(scale.max, s.max_of[b]);
  scale.t = t;

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
    for (int i = threadIdx.x; i < kBins; i += kThreads) s.count[i] = 0, s.mass[i] = 0;
    __syncthreads();
    row.each([&](float l, int) {
      if (!(l > -INFINITY)) return;
      const float below = scale.below(l);
      const int b = bin_of(below);
      atomicAdd(&s.count[b], 1u);
      if (by_p) atomicAdd(&s.mass[b], whole(expf(-below)));
    });
    merge(s, rank, blocks, s.counts, s.masses);
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
      return search(s, row, rank, blocks, scale, n, ca, ma, in_bin(bin), reached);
    };
    // all of them, where top-k leaves them
    u64 mass = 0;
    uint32_t tokens = 0;
    for (int i = threadIdx.x; i < kBins; i += kThreads) tokens += s.counts[i], mass += s.masses[i];
    mass = warp_total(mass);
    tokens = __reduce_add_sync(~0u, tokens);
    if (lane == 0) s.warp_sum[warp] = mass, s.warp_count[warp] = tokens;
    __syncthreads();
    mass = 0, tokens = 0;
    for (int w = 0; w < kWarps; ++w) mass += s.warp_sum[w], tokens += s.warp_count[w];
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
  row.each([&](float l, int i) { sum += kept(l, i, w); });
  sum = warp_total(sum);
  if (lane == 0) s.warp_sum[warp] = sum;
  __syncthreads();
  if (threadIdx.x < blocks) {
    sum = 0;
    for (int v = 0; v < kWarps; ++v) sum += s.warp_sum[v];
    put(there(&s.sum_of[rank], threadIdx.x), sum);
  }
  sync_cluster();
  u64 before = 0, total = 0;
  for (int b = 0; b < blocks; ++b) {
    if (b < rank) before += s.sum_of[b];
    total += s.sum_of[b];
  }
  const double at = static_cast<double>(u) * static_cast<double>(total);
  auto past = [&](u64 v) { return static_cast<double>(v) > at; };
  for (int v = 0; v < warp; ++v) before += s.warp_sum[v];
  if (past(before) || !past(before + s.warp_sum[warp])) return;
  // this warp's run has the token
  const int run = (row.n + kWarps * 32 - 1) / (kWarps * 32) * 32;
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

template <typename T>
cudaError_t launch(Args& a, cudaStream_t s) {
  cudaError_t st = allow_most_smem<sample_kernel<T>>();
  if (st != cudaSuccess) return st;
  int blocks = 1;
  // more blocks to a row as long as there is work for each and room for all
  while (blocks < kMaxBlocks && (a.V + blocks - 1) / blocks >= 2 * kFewest &&
         (a.rows * blocks * 2 <= 2 * 304 ||
          (a.V + blocks - 1) / blocks * sizeof(T) + 32 > kMaxData))
    blocks *= 2;
  a.part = static_cast<int>((a.V + blocks - 1) / blocks);
  const size_t bytes = static_cast<size_t>(a.part) * sizeof(T) + 32;
  a.held = bytes <= kMaxData;
  cudaLaunchConfig_t cfg = {};
  const unsigned ys = static_cast<unsigned>(a.rows < 65535 ? a.rows : 65535);
  cfg.gridDim = dim3(blocks, ys, static_cast<unsigned>((a.rows + 65534) / 65535));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = a.held ? bytes : 0;
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
