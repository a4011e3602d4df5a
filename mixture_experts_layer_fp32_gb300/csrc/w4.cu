// Products with 4-bit weights (group scales) for few rows, and the routed
// SwiGLU experts built from them.
//
// y = x W^T with few rows of x reads every weight once and is bound by that
// stream, so the kernel is built around it: blocks of 16 output rows x 128
// inputs (1 KB of codes) go to a warp, which copies the blocks to come into
// its own ring in shared memory (cp.async, no registers, no barriers) across
// item boundaries, and multiplies with mma.sync m16n8k16: the codes become
// whole bf16 numbers (exact: code - zero), the x rows are the 8 columns, a
// group's sum stays in fp32 and is scaled in fp32.  The code layout (moe.h)
// puts a lane's four words of a block next to each other, each covering one
// group of 32 with the three other lanes of its row.
//
// tcgen05 wants both operands of a 128-row tile in shared memory or TMEM as
// bf16, four times the bytes of the codes; with one to a few columns that
// traffic, not the multiplication, would be the bound.
#include "w4.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;      // of a block; they split an item's inputs
constexpr int kSlots = 6;      // ring of a warp, in blocks of 16 x 128 codes
constexpr int kMaxPairs = 1024;  // (token, slot) pairs of one launch
constexpr int kSms = 152;

// one block's bytes in the ring: codes, scales (16 bytes a row), zeros (8 a row)
constexpr int kCodeBytes = 1024, kScaleBytes = 16 * 16, kZeroBytes = 16 * 8;
constexpr int kSlotBytes = kCodeBytes + kScaleBytes + kZeroBytes;

enum { LINEAR = 0, FC1 = 1, FC2 = 2 };

struct Args {
  const __nv_bfloat16* x;  // LINEAR: [rows, K]; FC1: [T, K]; FC2: [pairs, 2, K], the two parts
  W4 w0, w1;               // FC1: W1 and W3 (rows g and g + 8 of a tile); else w0 alone
  int64_t scale_bytes;     // of one weight's scales
  int K, blocks, groups;   // inputs, blocks and groups of a row
  int N, tiles;            // outputs of an expert, its tiles
  int splits;              // parts of a row that are items of their own
  int rows;                // LINEAR: rows of x
  int out_f32;             // LINEAR
  void* out;               // LINEAR: y or partial sums; FC1: hidden parts; FC2: partial sums
  // experts
  const int32_t* idx;
  const uint8_t* keep;
  int pairs, E, topk;
  int* err;
};

__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, int bytes16) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes16)
               : "memory");
}
__device__ __forceinline__ void copy_async4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Codes m and m + 4 of a word as bf16 pair code - zero, exact: 128 + code is
// the bf16 number 0x4300 | code.  zero128: the pair of 128 + zero.
__device__ __forceinline__ uint32_t pair_of(uint32_t word, int m, uint32_t zero128) {
  const uint32_t v = ((word >> (4 * m)) & 0x000f000fu) | 0x43004300u;
  uint32_t d;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(v), "r"(zero128));
  return d;
}

// The pairs of a launch sorted by expert, in shared memory; every block works
// it out for itself, which is cheaper than a launch.
struct Plan {
  uint16_t pair[kMaxPairs];       // pairs by expert, ascending within one
  uint16_t count[MOE_MAX_EXPERTS];
  uint16_t first[MOE_MAX_EXPERTS];
  uint16_t warp_count[kWarps][MOE_MAX_EXPERTS];
  // chunks of at most 8 NT rows of one expert
  uint16_t chunk_expert[kMaxPairs];
  uint16_t chunk_row[kMaxPairs];
  int scan[kWarps][2];
  int chunks;
};

__device__ void make_plan(Plan& p, const Args& a, int chunk_rows) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < kWarps * MOE_MAX_EXPERTS; i += kWarps * 32)
    (&p.warp_count[0][0])[i] = 0;
  __syncthreads();
  // a warp takes up to four chunks of 32 pairs, one after another: ranks by
  // pair order within the warp
  constexpr int kRounds = kMaxPairs / (kWarps * 32);
  const int rounds = (a.pairs + kWarps * 32 - 1) / (kWarps * 32);
  int expert[kRounds], rank[kRounds];
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    expert[r] = -1;
    if (r >= rounds) continue;
    const int i = (warp * rounds + r) * 32 + lane;
    int e = -1;
    if (i < a.pairs && !(a.keep && a.keep[i] == 0)) {
      e = a.idx[i];
      if (e < 0 || e >= a.E) {
        if (blockIdx.x == 0) report_error(a.err, DEV_ERR_INDEX, e);
        e = -1;
      }
    }
    const unsigned same = __match_any_sync(~0u, e);
    const int before = __popc(same & ((1u << lane) - 1));
    int base = 0;
    if (e >= 0) base = p.warp_count[warp][e];
    __syncwarp();
    if (e >= 0 && before == 0) p.warp_count[warp][e] = base + __popc(same);
    __syncwarp();
    expert[r] = e;
    rank[r] = base + before;
  }
  __syncthreads();
  // thread e: expert e's count, then the scans of the counts and of the chunks
  static_assert(kWarps * 32 == MOE_MAX_EXPERTS, "one thread to an expert");
  int n = 0;
  for (int w = 0; w < kWarps; ++w) {
    const int c = p.warp_count[w][tid];
    p.warp_count[w][tid] = n;
    n += c;
  }
  const int chunks = (n + chunk_rows - 1) / chunk_rows;
  int sn = n, sc = chunks;
  for (int o = 1; o < 32; o <<= 1) {
    const int un = __shfl_up_sync(~0u, sn, o), uc = __shfl_up_sync(~0u, sc, o);
    if (lane >= o) {
      sn += un;
      sc += uc;
    }
  }
  if (lane == 31) {
    p.scan[warp][0] = sn;
    p.scan[warp][1] = sc;
  }
  __syncthreads();
  for (int w = 0; w < warp; ++w) {
    sn += p.scan[w][0];
    sc += p.scan[w][1];
  }
  p.count[tid] = n;
  p.first[tid] = sn - n;
  for (int c = 0; c < chunks; ++c) {
    p.chunk_expert[sc - chunks + c] = tid;
    p.chunk_row[sc - chunks + c] = sn - n + c * chunk_rows;
  }
  if (tid == kWarps * 32 - 1) p.chunks = sc;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kRounds; ++r)
    if (expert[r] >= 0)
      p.pair[p.first[expert[r]] + p.warp_count[warp][expert[r]] + rank[r]] =
          (warp * rounds + r) * 32 + lane;
  __syncthreads();
}

// An item: the rows of one chunk x one tile of outputs x one part of the inputs.
struct Item {
  int chunk, tile, lo, hi;  // blocks [lo, hi) of the row
};
__device__ __forceinline__ Item item_of(const Args& a, int v) {
  Item it;
  int s = 0;
  if (a.splits > 1) {
    s = v % a.splits;
    v /= a.splits;
  }
  it.chunk = v / a.tiles;
  it.tile = v - it.chunk * a.tiles;
  it.lo = a.blocks * s / a.splits;
  it.hi = a.blocks * (s + 1) / a.splits;
  return it;
}
// first block of a warp: the start moves with the item so that rows whose
// blocks do not divide evenly burden the warps in turn
__device__ __forceinline__ int first_block(const Item& it, int v, int warp) {
  return it.lo + ((warp + v) & (kWarps - 1));
}

template <int MODE, int G32, int NT>
__global__ void __launch_bounds__(kWarps * 32, 2) w4_kernel(Args a) {
  constexpr int GPB = 4 / G32;        // groups of a block
  constexpr int kChunkRows = MODE == FC2 ? 4 * NT : 8 * NT;
  extern __shared__ __align__(16) uint8_t smem[];
  float* red = reinterpret_cast<float*>(smem + kWarps * kSlots * kSlotBytes);  // 2 buffers
  Plan& plan = *reinterpret_cast<Plan*>(red + 2 * kWarps * NT * 128);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;

  int chunks;
  if (MODE == LINEAR) {
    chunks = (a.rows + kChunkRows - 1) / kChunkRows;
  } else {
    if (MODE == FC1) pdl_trigger();
    make_plan(plan, a, kChunkRows);
    chunks = plan.chunks;
  }
  const int items = chunks * a.tiles * a.splits;

  // ---- the stream of blocks, kSlots - 1 ahead of their use ----
  uint8_t* ring = smem + warp * kSlots * kSlotBytes;
  const uint32_t ring_at = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  int pv = blockIdx.x, pkb = 0, phi = 0, pslot = 0;
  int64_t prow0 = 0, prow1 = 0;
  auto rows_of_item = [&](const Item& it, int64_t& r0, int64_t& r1) {
    const int64_t e = MODE == LINEAR ? 0 : plan.chunk_expert[it.chunk];
    if (MODE == FC1) {
      r0 = r1 = e * a.N + it.tile * 8 + g;
    } else {  // outputs past the last one repeat it; they are not stored
      const int n0 = it.tile * 16 + g, n1 = n0 + 8;
      r0 = e * a.N + (n0 < a.N ? n0 : a.N - 1);
      r1 = e * a.N + (n1 < a.N ? n1 : a.N - 1);
    }
  };
  auto enter = [&]() {  // the producer's next item that has blocks for this warp
    while (pv < items) {
      const Item it = item_of(a, pv);
      pkb = first_block(it, pv, warp);
      phi = it.hi;
      if (pkb < phi) {
        rows_of_item(it, prow0, prow1);
        return;
      }
      pv += gridDim.x;
    }
  };
  const W4& w1 = MODE == FC1 ? a.w1 : a.w0;
  auto copy_scales = [&](const W4& w, int64_t row, uint32_t dst) {
    // the four lanes of a row bring the aligned 4-byte words around its values
    const int64_t at = (row * a.groups + pkb * GPB) * 2, word = (at & ~int64_t{3}) + 4 * t;
    if (word < at + 2 * GPB && word < a.scale_bytes) {
      const int64_t left = a.scale_bytes - word;
      copy_async4(dst + 4 * t, reinterpret_cast<const uint8_t*>(w.scales) + word,
                  left < 4 ? static_cast<int>(left) : 4);
    }
  };
  auto copy_zeros = [&](const W4& w, int64_t row, uint32_t dst) {
    const int64_t at = row * a.groups + pkb * GPB, word = (at & ~int64_t{3}) + 4 * t;
    if (t < 2 && word < at + GPB && word < a.scale_bytes / 2) {
      const int64_t left = a.scale_bytes / 2 - word;
      copy_async4(dst + 4 * t, w.zeros + word, left < 4 ? static_cast<int>(left) : 4);
    }
  };
  auto produce = [&]() {
    if (pv < items) {
      const uint32_t dst = ring_at + pslot * kSlotBytes;
      copy_async(dst + lane * 16, a.w0.codes + (prow0 * a.blocks + pkb) * 64 + t * 16, 16);
      copy_async(dst + 512 + lane * 16, w1.codes + (prow1 * a.blocks + pkb) * 64 + t * 16, 16);
      copy_scales(a.w0, prow0, dst + kCodeBytes + g * 16);
      copy_scales(w1, prow1, dst + kCodeBytes + 128 + g * 16);
      if (a.w0.zeros) {
        copy_zeros(a.w0, prow0, dst + kCodeBytes + kScaleBytes + g * 8);
        copy_zeros(w1, prow1, dst + kCodeBytes + kScaleBytes + 64 + g * 8);
      }
      pkb += kWarps;
      if (pkb >= phi) {
        pv += gridDim.x;
        enter();
      }
    }
    copies_commit();
    pslot = pslot + 1 == kSlots ? 0 : pslot + 1;
  };
  enter();
#pragma unroll 1
  for (int i = 0; i < kSlots - 1; ++i) produce();
  if (MODE == FC2) pdl_wait();  // the hidden values of FC1

  int slot = 0, buf = 0;
  for (int v = blockIdx.x; v < items; v += gridDim.x) {
    const Item it = item_of(a, v);
    int64_t row0, row1;
    rows_of_item(it, row0, row1);
    int row_first, row_count;  // of the chunk, in sorted order (LINEAR: in x)
    if (MODE == LINEAR) {
      row_first = it.chunk * kChunkRows;
      row_count = min(kChunkRows, a.rows - row_first);
    } else {
      const int e = plan.chunk_expert[it.chunk];
      row_first = plan.chunk_row[it.chunk];
      row_count = min(kChunkRows, plan.first[e] + plan.count[e] - row_first);
    }
    // column g of tile n: a row of x (FC2: one part of a row of hidden values)
    const __nv_bfloat16* xp[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int col = n * 8 + g, r = MODE == FC2 ? col >> 1 : col;
      xp[n] = nullptr;
      if (r < row_count) {
        int64_t at = row_first + r;
        if (MODE == FC1) at = plan.pair[row_first + r] / a.topk;
        if (MODE == FC2) at = 2 * at + (col & 1);
        xp[n] = a.x + at * a.K + 8 * t;
      }
    }
    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[n][c] = 0.f;

    for (int kb = first_block(it, v, warp); kb < it.hi; kb += kWarps) {
      __syncwarp();  // every lane is done with the slot that is filled next
      produce();
      copies_wait<kSlots - 1>();
      __syncwarp();  // and sees the others' copies
      const uint8_t* src = ring + slot * kSlotBytes;
      const uint4 q0 = *reinterpret_cast<const uint4*>(src + lane * 16);
      const uint4 q1 = *reinterpret_cast<const uint4*>(src + 512 + lane * 16);
      const uint32_t c0[4] = {q0.x, q0.y, q0.z, q0.w}, c1[4] = {q1.x, q1.y, q1.z, q1.w};
      const int g0 = static_cast<int>((row0 * a.groups + kb * GPB) & 3);
      const int g1 = static_cast<int>((row1 * a.groups + kb * GPB) & 3);
      const __nv_bfloat16* s0 =
          reinterpret_cast<const __nv_bfloat16*>(src + kCodeBytes + g * 16) + (g0 & 1);
      const __nv_bfloat16* s1 =
          reinterpret_cast<const __nv_bfloat16*>(src + kCodeBytes + 128 + g * 16) + (g1 & 1);
      const uint8_t* z0 = src + kCodeBytes + kScaleBytes + g * 8 + g0;
      const uint8_t* z1 = src + kCodeBytes + kScaleBytes + 64 + g * 8 + g1;
      float sum[NT][4];
      uint32_t zero0 = 0x43084308u, zero1 = 0x43084308u;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j % G32 == 0) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) sum[n][c] = 0.f;
          if (a.w0.zeros) {
            zero0 = 0x43004300u + z0[j / G32] * 0x00010001u;
            zero1 = 0x43004300u + z1[j / G32] * 0x00010001u;
          }
        }
        const bool in = kb * 128 + 32 * j < a.K;
        uint4 b[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          b[n] = make_uint4(0, 0, 0, 0);
          if (xp[n] && in) b[n] = *reinterpret_cast<const uint4*>(xp[n] + kb * 128 + 32 * j);
        }
        uint32_t f0[4], f1[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          f0[m] = pair_of(c0[j], m, zero0);
          f1[m] = pair_of(c1[j], m, zero1);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma(sum[n], f0[0], f1[0], f0[1], f1[1], b[n].x, b[n].y);
          mma(sum[n], f0[2], f1[2], f0[3], f1[3], b[n].z, b[n].w);
        }
        if (j % G32 == G32 - 1) {
          const float w = in ? __bfloat162float(s0[j / G32]) : 0.f;
          const float u = in ? __bfloat162float(s1[j / G32]) : 0.f;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            acc[n][0] += w * sum[n][0];
            acc[n][1] += w * sum[n][1];
            acc[n][2] += u * sum[n][2];
            acc[n][3] += u * sum[n][3];
          }
        }
      }
      slot = slot + 1 == kSlots ? 0 : slot + 1;
    }

    // ---- the warps' sums, added in order ----
    float* mine = red + (buf * kWarps + warp) * NT * 128;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 4; ++c) mine[(n * 4 + c) * 32 + lane] = acc[n][c];
    __syncthreads();
    const float* all = red + buf * kWarps * NT * 128;
    auto total = [&](int n, int c, int l) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += all[(w * NT + n) * 128 + c * 32 + l];
      return s;
    };
    buf ^= 1;
    if (MODE == FC1) {
      // W1's row is g, W3's g + 8: their sums of column 2t + c are c and c + 2
      for (int i = threadIdx.x; i < NT * 64; i += kWarps * 32) {
        const int n = i >> 6, c = (i >> 5) & 1, l = i & 31, r = n * 8 + 2 * (l & 3) + c;
        if (r >= row_count) continue;
        const float p = total(n, c, l), q = total(n, c + 2, l);
        const float hid = p / (1.f + expf(-p)) * q;
        // two bf16 whose sum is within 2^-17 of the value: one of them would be
        // the largest error of the layer
        const __nv_bfloat16 hi = __float2bfloat16_rn(hid);
        const float rest = isinf(__bfloat162float(hi)) ? 0.f : hid - __bfloat162float(hi);
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) +
                             static_cast<int64_t>(row_first + r) * 2 * a.N + it.tile * 8 + (l >> 2);
        out[0] = hi;
        out[a.N] = __float2bfloat16_rn(rest);
      }
    } else if (MODE == FC2) {
      // columns 2i and 2i + 1 are the two parts of row i
      const int s = a.splits > 1 ? v % a.splits : 0;
      for (int i = threadIdx.x; i < NT * 64; i += kWarps * 32) {
        const int n = i >> 6, half = (i >> 5) & 1, l = i & 31, r = n * 4 + (l & 3);
        const int o = it.tile * 16 + half * 8 + (l >> 2);
        if (r >= row_count || o >= a.N) continue;
        const int pair = plan.pair[row_first + r];
        static_cast<float*>(a.out)[(static_cast<int64_t>(s) * a.pairs + pair) * a.N + o] =
            total(n, 2 * half, l) + total(n, 2 * half + 1, l);
      }
    } else {
      const int s = a.splits > 1 ? v % a.splits : 0;
      for (int i = threadIdx.x; i < NT * 128; i += kWarps * 32) {
        const int n = i >> 7, c = (i >> 5) & 3, l = i & 31, r = n * 8 + 2 * (l & 3) + (c & 1);
        const int o = it.tile * 16 + (c >> 1) * 8 + (l >> 2);
        if (r >= row_count || o >= a.N) continue;
        const float y = total(n, c, l);
        const int64_t at = (static_cast<int64_t>(s) * a.rows + row_first + r) * a.N + o;
        if (a.out_f32) static_cast<float*>(a.out)[at] = y;
        else static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(y);
      }
    }
  }
  copies_wait<0>();
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
  for (int q = 0; q < splits; ++q) s += part[q * n + i];
  if (out_f32) static_cast<float*>(y)[i] = s;
  else static_cast<__nv_bfloat16*>(y)[i] = __float2bfloat16_rn(s);
}

template <int MODE, int G32, int NT>
cudaError_t launch_one(const Args& a, bool dependent, cudaStream_t s) {
  auto k = w4_kernel<MODE, G32, NT>;
  const size_t smem = kWarps * kSlots * kSlotBytes + 2 * kWarps * NT * 128 * sizeof(float) +
                      (MODE == LINEAR ? 0 : sizeof(Plan));
  const cudaError_t st =
      cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (st != cudaSuccess) return st;
  int64_t items = static_cast<int64_t>(a.tiles) * a.splits;
  if (MODE == LINEAR) items *= (a.rows + 8 * NT - 1) / (8 * NT);
  else items *= a.pairs;
  const unsigned grid = static_cast<unsigned>(items < 2 * kSms ? items : 2 * kSms);
  if (dependent) return launch_dependent(k, dim3(grid), dim3(kWarps * 32), smem, s, a);
  k<<<grid, kWarps * 32, smem, s>>>(a);
  return cudaGetLastError();
}

template <int MODE, int NT>
cudaError_t launch_group(int group, const Args& a, bool dependent, cudaStream_t s) {
  switch (group) {
    case 32: return launch_one<MODE, 1, NT>(a, dependent, s);
    case 64: return launch_one<MODE, 2, NT>(a, dependent, s);
    default: return launch_one<MODE, 4, NT>(a, dependent, s);
  }
}

// `columns`: those that an expert fills on average; tiles of 8 of them
template <int MODE>
cudaError_t launch_mode(int group, int64_t columns, const Args& a, bool dependent,
                        cudaStream_t s) {
  if (columns <= 8) return launch_group<MODE, 1>(group, a, dependent, s);
  if (columns <= 16) return launch_group<MODE, 2>(group, a, dependent, s);
  return launch_group<MODE, 4>(group, a, dependent, s);
}

int tiles_of(int N) { return (N + 15) / 16; }

// A row's inputs are split over items where the whole rows are too few items
// to fill the card evenly: about `want` items, parts of 8 blocks at least.
int splits_of(int64_t items, int blocks, int want) {
  int s = 1;
  while (s < 4 && items * s < want && blocks / (2 * s) >= kWarps) s *= 2;
  return s;
}

int linear_splits(int64_t rows, int N, int K) {
  const int64_t chunks = (rows + 31) / 32;
  return splits_of(chunks * tiles_of(N), w4_blocks(K), kSms);
}

// tokens of one launch of the experts
int tokens_per_launch(int k) { return kMaxPairs / k; }

int fc2_splits(int pairs, int E, int h, int f) {
  return splits_of(static_cast<int64_t>(pairs < E ? pairs : E) * tiles_of(h), w4_blocks(f),
                   8 * kSms);
}

size_t align256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

}  // namespace

size_t w4_linear_scratch(int64_t rows, int N, int K) {
  const int s = linear_splits(rows, N, K);
  return s == 1 ? 0 : static_cast<size_t>(s) * rows * N * 4;
}

cudaError_t launch_w4_linear(int64_t rows, int N, int K, int group, const void* x, const W4& W,
                             void* y, int y_dtype, void* scratch, cudaStream_t s) {
  Args a = {};
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.w0 = W;
  a.K = K;
  a.blocks = w4_blocks(K);
  a.groups = K / group;
  a.scale_bytes = static_cast<int64_t>(N) * a.groups * 2;
  a.N = N;
  a.tiles = tiles_of(N);
  a.splits = linear_splits(rows, N, K);
  const bool split = a.splits > 1;
  const int out_f32 = y_dtype == MOE_F32;
  // rows in launches whose items fit 32 bits
  const int64_t most = ((int64_t{1} << 30) / (static_cast<int64_t>(a.tiles) * a.splits) + 1) * 8;
  for (int64_t r = 0; r < rows; r += most) {
    const int64_t m = rows - r < most ? rows - r : most;
    a.rows = static_cast<int>(m);
    a.x = static_cast<const __nv_bfloat16*>(x) + r * K;
    void* out = static_cast<char*>(y) + r * N * (out_f32 ? 4 : 2);
    a.out = split ? scratch : out;
    a.out_f32 = split ? 1 : out_f32;
    cudaError_t st = launch_mode<LINEAR>(group, m, a, false, s);
    if (st != cudaSuccess) return st;
    if (split) {
      const int64_t n = m * N;
      st = launch_dependent(w4_join_kernel, dim3(static_cast<unsigned>((n + 255) / 256)),
                            dim3(256), 0, s, n, a.splits, static_cast<const float*>(scratch),
                            out_f32, out);
      if (st != cudaSuccess) return st;
    }
  }
  return cudaSuccess;
}

size_t w4_experts_scratch(int T, int h, int E, int k, int f) {
  const int t = tokens_per_launch(k), n = T < t ? T : t;
  const size_t pairs = static_cast<size_t>(n) * k;
  return align256(pairs * f * 4) + 4 * pairs * h * 4;
}

cudaError_t launch_w4_experts(int T, int h, int E, int k, int f, int group, const void* x,
                              const int32_t* topk_idx, const float* topk_prob,
                              const uint8_t* keep, const W4& W1, const W4& W3, const W4& W2,
                              void* y, void* scratch, int* err, cudaStream_t s) {
  const int most = tokens_per_launch(k);
  for (int t = 0; t < T; t += most) {
    const int n = T - t < most ? T - t : most, pairs = n * k;
    void* hidden = scratch;
    float* part = reinterpret_cast<float*>(static_cast<char*>(scratch) +
                                           align256(static_cast<size_t>(pairs) * f * 4));
    Args a = {};
    a.idx = topk_idx + static_cast<int64_t>(t) * k;
    a.keep = keep ? keep + static_cast<int64_t>(t) * k : nullptr;
    a.pairs = pairs;
    a.E = E;
    a.topk = k;
    a.err = err;
    const int64_t each = (pairs + E - 1) / E;  // rows of an expert, on average
    a.x = static_cast<const __nv_bfloat16*>(x) + static_cast<int64_t>(t) * h;
    a.w0 = W1;
    a.w1 = W3;
    a.K = h;
    a.blocks = w4_blocks(h);
    a.groups = h / group;
    a.scale_bytes = static_cast<int64_t>(E) * f * a.groups * 2;
    a.N = f;
    a.tiles = f / 8;
    a.splits = 1;
    a.out = hidden;
    cudaError_t st = launch_mode<FC1>(group, each, a, false, s);
    if (st != cudaSuccess) return st;
    a.x = static_cast<const __nv_bfloat16*>(hidden);
    a.w0 = W2;
    a.w1 = W2;
    a.K = f;
    a.blocks = w4_blocks(f);
    a.groups = f / group;
    a.scale_bytes = static_cast<int64_t>(E) * h * a.groups * 2;
    a.N = h;
    a.tiles = tiles_of(h);
    a.splits = fc2_splits(pairs, E, h, f);
    a.out = part;
    st = launch_mode<FC2>(group, 2 * each, a, true, s);
    if (st != cudaSuccess) return st;
    const int64_t vecs = static_cast<int64_t>(n) * (h / 4);
    st = launch_dependent(w4_combine_kernel, dim3(static_cast<unsigned>((vecs + 255) / 256)),
                          dim3(256), 0, s, n, h, k, E, a.splits, static_cast<const float*>(part),
                          a.idx, topk_prob + static_cast<int64_t>(t) * k, a.keep,
                          static_cast<__nv_bfloat16*>(y) + static_cast<int64_t>(t) * h);
    if (st != cudaSuccess) return st;
  }
  return cudaSuccess;
}

}  // namespace moe
