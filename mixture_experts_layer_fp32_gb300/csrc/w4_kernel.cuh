// The products with 4-bit weights and the 4-bit experts: the kernel for the
// fewest rows, and how a product is shared out between kernels, parts and warps.
//
// y = x W^T with few rows of x reads every weight once and should be bound by
// that stream.  What stands in the way is the work per code.  The fp16 number
// with the bits 0x640q is 1024 + q, and 0x64q0 is 1024 + 16 q, so a word of 8
// codes becomes four pairs of numbers by four masks with an or (one instruction:
// as two, the experts of one token took 53.7 us for 46.8) and one shift, and four
// subtractions of 1024 + z and 1024 + 16 z make q - z and 16 (q - z) of them, the
// A registers of mma.sync m16n8k16.  Every second pair of inputs has the 16 taken
// out of x beforehand.
//
// The subtractions could be spared: 0x000q is the subnormal q 2^-24, and a zero
// point's share is z times the sum of x.  But the tensor cores add products up
// under the largest exponent, and behave as if a subnormal's were 2^-14: up to 10
// bits of the small products beside a large one were lost (rows with values 1000
// times the others came out 1e-5 off in the mean, 1e-7 now; the hidden values'
// product 3e-6, and 2e-7 now), while the time is the same.
//
// The rows of x are brought to fp16 once (w4_split_kernel): with a power of two
// for each row a bf16 number is exact (down to 2^-27 of its row's largest), and an
// fp32 hidden value is two fp16 numbers, a column each, exact to 2^-22.  The
// products are exact and their sums are fp32.
//
// (E4M3 operands would need two masks and one shift, but mma.sync of that type
// costs this machine several instructions: 194 were issued for a block of
// 16 x 128 codes.)
//
// Measured, with the rows' split and the combine (rate of the codes and scales):
// a row of 4096 x 4096 6.0 us; 8 rows of 57344 x 4096 25.0 us (4.9 TB/s); the
// experts of one token (2 of 8 of 4096 x 14336) 43.7 us (4.2 TB/s), of 16 tokens
// (8 of 128 of 4096 x 1536) 164 us (5.0 TB/s, 74% of what a copy reaches).  No unit
// is full: the issue slots are used to 36-58%, the shared memory to 42-60%, the
// tensor pipe to 14-28%; a warp's reads, masks and products follow one another,
// the memory waits at the ends of items, and a second block to an SM does not fit
// the registers.  Two chains of products in a warp, or a warp's stages next to its
// neighbours' instead of in runs, made no difference.
#pragma once

#include "roles.cuh"
#include "sm100_ptx.cuh"
#include "w4.cuh"

namespace moe {
namespace w4 {

using namespace roles;

constexpr int kWarps = 8;        // that work out the plan
constexpr int kNarrowWarps = 16; // of a block of the narrow kernel, one to an SM
constexpr int kMaxRows = 1024;   // rows of x, or (token, slot) pairs, of one launch
constexpr int kSms = 152;

enum { LINEAR = 0, FC1 = 1, FC2 = 2 };

// fp16 numbers to a value of x.
__host__ __device__ constexpr int pieces_of(int mode) { return mode == FC2 ? 2 : 1; }

struct Args {
  // The split rows, of tokens in the narrow FC1, of the pairs sorted by expert in
  // the wide one: fp16 [x_rows][pieces][blocks * 128], the inputs 2, 3, 6 and 7
  // of eight over 16; and each row's unit
  const __half* x;
  const float* unit;
  W4 w0, w1;              // FC1: W1 and W3 (rows g and g + 8 of a tile); else w0 twice
  int blocks, groups;     // of 128 inputs; groups of a row
  int N, tiles;           // outputs of an expert, its tiles
  int splits;             // parts of a row's inputs, items of their own
  int split_units, split_rest;  // stages of 4 blocks / splits, and the remainder
  int wk;                 // narrow: warps that share an item's inputs: a power of two
  int each, each_rest;    // their units, in a part of split_units and of one more
  int chunk_rows;         // rows of x of a chunk
  bool few;               // wide: chunks of 32 columns
  int x_pitch;            // narrow: bytes of a column of x in shared memory
  int rows;               // LINEAR: rows of x
  int out_f32;            // LINEAR
  void* out;              // LINEAR: y or partial sums; FC1: hidden values; FC2: partial sums
  // experts
  const int32_t* idx;
  const uint8_t* keep;
  int pairs, E, topk;
  int* err;
};

__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t at) {
  uint4 q;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
               : "r"(at)
               : "memory");
  return q;
}

// c += A B, or c = A B
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// The pairs of a launch sorted by expert, in shared memory; every block works
// it out for itself, which is cheaper than a launch.
struct Plan {
  uint16_t pair[kMaxRows];   // pairs by expert, ascending within one
  uint16_t token[kMaxRows];  // their tokens
  uint16_t end[MOE_MAX_EXPERTS];
  uint16_t first[MOE_MAX_EXPERTS];
  uint16_t warp_count[kWarps][MOE_MAX_EXPERTS];
  // chunks of rows of one expert
  uint16_t chunk_expert[kMaxRows];
  uint16_t chunk_row[kMaxRows];
  int scan[kWarps][2];
  int chunks;
};

__device__ inline void make_plan(Plan& p, const Args& a, int chunk_rows) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool works = warp < kWarps;
  for (int i = tid; i < kWarps * MOE_MAX_EXPERTS; i += blockDim.x) (&p.warp_count[0][0])[i] = 0;
  __syncthreads();
  // a warp takes up to four times 32 pairs, one after another: ranks by pair
  // order within the warp
  constexpr int kRounds = kMaxRows / (kWarps * 32);
  const int rounds = (a.pairs + kWarps * 32 - 1) / (kWarps * 32);
  int expert[kRounds], rank[kRounds];
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    expert[r] = -1;
    rank[r] = 0;
    if (r >= rounds || !works) continue;
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
  for (int w = 0; works && w < kWarps; ++w) {
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
  if (works && lane == 31) {
    p.scan[warp][0] = sn;
    p.scan[warp][1] = sc;
  }
  __syncthreads();
  if (works) {
    for (int w = 0; w < warp; ++w) {
      sn += p.scan[w][0];
      sc += p.scan[w][1];
    }
    p.end[tid] = sn;
    p.first[tid] = sn - n;
    for (int c = 0; c < chunks; ++c) {
      p.chunk_expert[sc - chunks + c] = tid;
      p.chunk_row[sc - chunks + c] = sn - n + c * chunk_rows;
    }
    if (tid == kWarps * 32 - 1) p.chunks = sc;
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kRounds; ++r)
    if (expert[r] >= 0) {
      const int at = p.first[expert[r]] + p.warp_count[warp][expert[r]] + rank[r];
      const int pair = (warp * rounds + r) * 32 + lane;
      p.pair[at] = pair;
      p.token[at] = pair / a.topk;
    }
  __syncthreads();
}

// Where a group of warps (wide: a block) stands in its list of items: the rows of one chunk x
// one part of the inputs x one tile of outputs, tiles first, so that neighbours
// read the same x.  A group takes every step-th.
struct Item {
  int chunk, part, tile;
  __device__ Item(int first, const Args& a) {
    tile = first % a.tiles;
    first /= a.tiles;
    part = first % a.splits;
    chunk = first / a.splits;
  }
  __device__ void next(int step, const Args& a) {
    tile += step;
    carry(a);
  }
  __device__ void carry(const Args& a) {
    while (tile >= a.tiles) {
      tile -= a.tiles;
      if (++part == a.splits) {
        part = 0;
        ++chunk;
      }
    }
  }
};

// Stores of the sums: two outputs, `low` of row g and `high` of row g + 8 of a
// tile that begins at output o (FC1: the two halves of feature o), of row r of
// the chunk.
template <int MODE>
__device__ __forceinline__ void put(const Args& a, const Plan& plan, int part, int row_first, int r,
                                    int o, float low, float high) {
  const float unit =
      a.unit[MODE == FC1 ? static_cast<int>(plan.token[row_first + r]) : row_first + r];
  low *= unit;
  high *= unit;
  if (MODE == FC1) {
    static_cast<float*>(a.out)[static_cast<int64_t>(row_first + r) * a.N + o] =
        low / (1.f + expf(-low)) * high;
  } else if (MODE == FC2) {
    float* out = static_cast<float*>(a.out) +
                 (static_cast<int64_t>(part) * a.pairs + plan.pair[row_first + r]) * a.N + o;
    out[0] = low;
    out[8] = high;
  } else {
    const int64_t at = (static_cast<int64_t>(part) * a.rows + row_first + r) * a.N + o;
    if (a.out_f32) {
      float* out = static_cast<float*>(a.out) + at;
      if (o < a.N) out[0] = low;
      if (o + 8 < a.N) out[8] = high;
    } else {
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + at;
      if (o < a.N) out[0] = __float2bfloat16_rn(low);
      if (o + 8 < a.N) out[8] = __float2bfloat16_rn(high);
    }
  }
}

// A row's scales and zeros of one block of inputs.
template <int GPB>
struct Scales {
  uint32_t s[(GPB + 1) / 2], z;
};
// at: the first value's place; valid: values of the row from there on
template <int GPB, bool ZEROS, bool TAIL>
__device__ __forceinline__ void load_scales(Scales<GPB>& v, const unsigned short* s,
                                            const uint8_t* z, int valid) {
  if (!TAIL) {
    if (GPB == 1) {
      v.s[0] = __ldg(s);
    } else if (GPB == 2) {
      v.s[0] = __ldg(reinterpret_cast<const uint32_t*>(s));
    } else {
      const uint2 q = __ldg(reinterpret_cast<const uint2*>(s));
      v.s[0] = q.x;
      v.s[(GPB + 1) / 2 - 1] = q.y;
    }
    if (ZEROS) {
      if (GPB == 1) v.z = __ldg(z);
      else if (GPB == 2) v.z = __ldg(reinterpret_cast<const unsigned short*>(z));
      else v.z = __ldg(reinterpret_cast<const uint32_t*>(z));
    }
  } else {  // rows of any alignment; past the row's last group: 0
#pragma unroll
    for (int q = 0; q < (GPB + 1) / 2; ++q) v.s[q] = 0;
    v.z = 0;
#pragma unroll
    for (int q = 0; q < GPB; ++q) {
      if (q >= valid) continue;
      v.s[q / 2] |= static_cast<uint32_t>(__ldg(s + q)) << (16 * (q & 1));
      if (ZEROS) v.z |= static_cast<uint32_t>(__ldg(z + q)) << (8 * q);
    }
  }
}
template <int GPB>
__device__ __forceinline__ float scale_of(const Scales<GPB>& v, int q) {
  return __uint_as_float(q & 1 ? v.s[q / 2] & 0xffff0000u : v.s[q / 2] << 16);
}
template <int GPB, bool ZEROS>
__device__ __forceinline__ uint32_t zero_of(const Scales<GPB>& v, int q) {
  return ZEROS ? (v.z >> (8 * q)) & 15u : 8u;
}
template <int GPB, bool ZEROS>
__device__ __forceinline__ Scales<GPB> scales_from(const Scales<GPB>& v, int lane) {
  Scales<GPB> r;
#pragma unroll
  for (int q = 0; q < (GPB + 1) / 2; ++q) r.s[q] = __shfl_sync(~0u, v.s[q], lane);
  r.z = ZEROS ? __shfl_sync(~0u, v.z, lane) : 0;
  return r;
}
// Codes as fp16 pairs: of a word's inputs 0 1, 2 3, 4 5, 6 7 the numbers 1024 + q,
// 1024 + 16 q, 1024 + q, 1024 + 16 q; less the same of the zero point, which is
// exact (whole numbers below 2048).
__device__ __forceinline__ uint32_t less(uint32_t a, uint32_t b) {
  const __half2 d = __hsub2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&d);
}
struct ZeroPair {
  uint32_t one, sixteen;
};
__device__ __forceinline__ ZeroPair zero_pair(uint32_t z) {
  return {0x64006400u + z * 0x00010001u, 0x64006400u + z * 0x00100010u};
}
// (word & MASK) | base in one instruction, which takes one constant: base is held
template <uint32_t MASK>
__device__ __forceinline__ uint32_t masked(uint32_t word, uint32_t base) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(word), "n"(MASK), "r"(base));
  return d;
}
__device__ __forceinline__ uint32_t held_1024() {
  uint32_t v;
  asm("mov.b32 %0, 0x64006400;" : "=r"(v));
  return v;
}
__device__ __forceinline__ void pairs_of(uint32_t word, uint32_t base, const ZeroPair& z,
                                         uint32_t (&p)[4]) {
  const uint32_t high = word >> 8;
  p[0] = less(masked<0x000f000fu>(word, base), z.one);
  p[1] = less(masked<0x00f000f0u>(word, base), z.sixteen);
  p[2] = less(masked<0x000f000fu>(high, base), z.one);
  p[3] = less(masked<0x00f000f0u>(high, base), z.sixteen);
}

// Up to 8 columns (8 rows of x; FC2: 4) to a chunk.  A tile is 16 outputs (FC1:
// 8 features, W1's rows and W3's); wk warps share its inputs, each a run of
// stages of four blocks.  Codes come by TMA, one stage ahead and across the ends
// of items, into a ring of the warp's own: one instruction for 4 KB.  A block
// takes consecutive items, so that it has few changes of the chunk or the part;
// at each it brings the chunk's x (of the part's inputs) into shared memory.
// Reading x through L1 instead cost a third of the time: L1 answers in order,
// and a read that would hit waits behind every one that misses.
//
// A wait that runs out reports it and the warp goes on with what is there, so that
// nobody waits for it, but copies nothing more; the block ends after its copies.
constexpr int kNarrowX = 66 * 1024;  // bytes of x, at most

template <int MODE, int G32, bool ZEROS, bool TAIL>
__global__ void __launch_bounds__(kNarrowWarps * 32, 1) w4_narrow_kernel(
    const __grid_constant__ CUtensorMap map0, const __grid_constant__ CUtensorMap map1, Args a) {
  constexpr int GPB = 4 / G32;         // groups of a block
  constexpr int CP = pieces_of(MODE);  // columns of a row
  constexpr int XR = 2 / CP;           // rows of x in a lane's two columns
  constexpr int SB = 4;                // blocks of a stage
  constexpr int kStage = SB * 1024;
  constexpr int kTile = MODE == FC1 ? 8 : 16;
  constexpr int kRed = 2 * XR * 32;
  constexpr int W = kNarrowWarps;
  extern __shared__ __align__(128) uint8_t smem[];
  float* red = reinterpret_cast<float*>(smem + W * 2 * kStage);  // 2 buffers
  uint8_t* x_at = reinterpret_cast<uint8_t*>(red + 2 * W * kRed);
  Plan& plan = *reinterpret_cast<Plan*>(x_at + kNarrowX);
  __shared__ uint64_t bars[W][2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int wk = a.wk, group = warp / wk, w_in = warp & (wk - 1), step = W / wk;
  pdl_trigger();

  int chunks;
  if (MODE == LINEAR) {
    chunks = (a.rows + a.chunk_rows - 1) / a.chunk_rows;
  } else {
    make_plan(plan, a, a.chunk_rows);
    chunks = plan.chunks;
  }
  // this block's items
  const int64_t items = static_cast<int64_t>(chunks) * a.splits * a.tiles;
  const int begin = static_cast<int>(items * blockIdx.x / gridDim.x);
  const int end = static_cast<int>(items * (blockIdx.x + 1) / gridDim.x);
  const uint32_t ring = ptx::smem_u32(smem) + warp * 2 * kStage;
  const uint32_t bar = ptx::smem_u32(&bars[warp][0]);
  if (lane == 0) {
    ptx::mbar_init(bar, 1);
    ptx::mbar_init(bar + 8, 1);
    ptx::fence_mbar_init();
  }
  __syncwarp();

  // ---- codes and scales, a stage ahead ----
  int next = begin + group;  // the item of the stage to come
  Item it(next, a);
  int stage = 0, left = 0;  // its number in the row; the item's stages from there on
  uint32_t row = 0;         // the tile's first output
  // lane t of a row (g, g + 8) reads the scales of the stage's block t; the row's
  // lanes have them from each other by shuffles
  const unsigned short *ps0, *ps1;
  const uint8_t *pz0, *pz1;
  Scales<GPB> scale0, scale1;
  auto enter = [&]() {
    if (next >= end) return;
    const bool rest = it.part < a.split_rest;
    const int each = rest ? a.each_rest : a.each;
    stage = it.part * a.split_units + min(it.part, a.split_rest) + w_in * each;
    left = min(each, a.split_units + rest - w_in * each);
    const uint32_t e = MODE == LINEAR ? 0 : plan.chunk_expert[it.chunk];
    row = e * a.N + static_cast<uint32_t>(it.tile) * kTile;
    int r0 = g, r1 = MODE == FC1 ? g : g + 8;
    if (MODE == LINEAR) {  // outputs past the last one take its scales and are not stored
      r0 = min(r0, a.N - 1 - it.tile * kTile);
      r1 = min(r1, a.N - 1 - it.tile * kTile);
    }
    const uint64_t at = static_cast<uint64_t>(row) * a.groups + (stage * SB + t) * GPB;
    ps0 = reinterpret_cast<const unsigned short*>(a.w0.scales) + at + r0 * a.groups;
    ps1 = reinterpret_cast<const unsigned short*>(a.w1.scales) + at + r1 * a.groups;
    if (ZEROS) {
      pz0 = a.w0.zeros + at + r0 * a.groups;
      pz1 = a.w1.zeros + at + r1 * a.groups;
    }
  };
  int fill = 0;
  bool lost = false;  // a wait ran out
  auto fetch = [&]() {
    if (next >= end) return;
    __syncwarp();  // every lane has read what the slot held
    if (lane == 0 && !lost) {
      const uint32_t dst = ring + fill * kStage, b = bar + fill * 8;
      ptx::mbar_arrive_expect_tx(b, kStage);
      // blocks past the row's end come as zeros
      ptx::tma_load_3d(dst, &map0, 0, static_cast<int>(row), stage * SB, b);
      if (MODE == FC1)
        ptx::tma_load_3d(dst + kStage / 2, &map1, 0, static_cast<int>(row), stage * SB, b);
    }
    const int valid = a.groups - (stage * SB + t) * GPB;  // groups from the lane's block on
    if (valid > 0) {
      load_scales<GPB, ZEROS, TAIL>(scale0, ps0, pz0, valid);
      load_scales<GPB, ZEROS, TAIL>(scale1, ps1, pz1, valid);
    }
    if (--left > 0) {
      ++stage;
      ps0 += SB * GPB;
      ps1 += SB * GPB;
      if (ZEROS) {
        pz0 += SB * GPB;
        pz1 += SB * GPB;
      }
    } else {
      next += step;
      it.next(step, a);
      enter();
    }
    fill ^= 1;
  };
  enter();
  int at_hand = next;  // the item of the stage at hand
  Item now = it;
  int stage_now = stage, left_now = left;
  fetch();
  pdl_wait();  // the split rows

  const uint32_t base = held_1024();
  int use = 0, phase = 0, buf = 0;  // the slot at hand and its barrier's phase
  const int x_row = a.blocks * (128 * CP);
  const uint32_t xs = ptx::smem_u32(x_at);
  Item epoch(begin, a);
  for (int from = begin; from < end;) {
    const int to = min(end, from + a.tiles - epoch.tile);  // the epoch's items
    int row_first, row_count;  // of the chunk, in sorted order (LINEAR: in x)
    if (MODE == LINEAR) {
      row_first = epoch.chunk * a.chunk_rows;
      row_count = min(a.chunk_rows, a.rows - row_first);
    } else {
      row_first = plan.chunk_row[epoch.chunk];
      row_count = min(a.chunk_rows, plan.end[plan.chunk_expert[epoch.chunk]] - row_first);
    }
    const int first = epoch.part * a.split_units + min(epoch.part, a.split_rest);  // stage
    const int stages = a.split_units + (epoch.part < a.split_rest);
    const int blocks_in = min(stages * SB, a.blocks - first * SB);
    // ---- the epoch's x: column c is piece c % CP of row c / CP ----
    __syncthreads();
    {
      auto row_of = [&](int r) {
        return MODE == FC1 ? static_cast<int>(plan.token[row_first + r]) : row_first + r;
      };
      // 16 warps: 16 / columns of them to a column
      const int columns = row_count * CP, share = W / columns;
      if (warp < columns * share) {
        const int c = warp / share;
        const __half* p = a.x + static_cast<int64_t>(row_of(c / CP)) * x_row +
                          (CP == 2 ? (c & 1) * (x_row / 2) : 0) + first * (SB * 128);
        for (int i = warp % share * 32 + lane; i < blocks_in * 16; i += share * 32)
          copy_async(xs + c * a.x_pitch + i * 16, p + i * 8);
      }
      copies_commit();
      copies_wait<0>();
    }
    __syncthreads();
    // columns past the chunk's repeat its first and are not stored; a lane's sums
    // are of the columns 2t, 2t + 1
    const uint32_t x_lane = xs + (g < row_count * CP ? g : 0) * a.x_pitch + t * 16;

    while (at_hand < to) {
      float acc[2][XR];  // of the outputs g and g + 8
#pragma unroll
      for (int i = 0; i < XR; ++i) acc[0][i] = acc[1][i] = 0.f;
      auto block = [&](uint32_t src, uint32_t xb, const Scales<GPB>& st0,
                       const Scales<GPB>& st1, int b) {
        constexpr uint32_t kBlock = MODE == FC1 ? 512 : 1024;
        constexpr uint32_t kSecond = MODE == FC1 ? kStage / 2 : 512;
        const uint4 q0 = lds16(src + b * kBlock), q1 = lds16(src + b * kBlock + kSecond);
        const uint32_t c0[4] = {q0.x, q0.y, q0.z, q0.w}, c1[4] = {q1.x, q1.y, q1.z, q1.w};
        const Scales<GPB> s0 = scales_from<GPB, ZEROS>(st0, (lane & ~3) + b);
        const Scales<GPB> s1 = scales_from<GPB, ZEROS>(st1, (lane & ~3) + b);
#pragma unroll
        for (int q = 0; q < GPB; ++q) {
          const ZeroPair z0 = zero_pair(zero_of<GPB, ZEROS>(s0, q));
          const ZeroPair z1 = zero_pair(zero_of<GPB, ZEROS>(s1, q));
          float sum[4];
#pragma unroll
          for (int j = q * G32; j < (q + 1) * G32; ++j) {
            uint32_t p0[4], p1[4];
            pairs_of(c0[j], base, z0, p0);
            pairs_of(c1[j], base, z1, p1);
            const uint4 x = lds16(xb + b * 256 + j * 64);
            if (j == q * G32) mma_first(sum, p0[0], p1[0], p0[1], p1[1], x.x, x.y);
            else mma(sum, p0[0], p1[0], p0[1], p1[1], x.x, x.y);
            mma(sum, p0[2], p1[2], p0[3], p1[3], x.z, x.w);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float s = scale_of(i ? s1 : s0, q);
            if (CP == 2) {  // the second piece is in 2^-11 of the first's unit
              acc[i][0] += s * (sum[2 * i] + 0.00048828125f * sum[2 * i + 1]);
            } else {
              acc[i][0] += s * sum[2 * i];
              acc[i][XR - 1] += s * sum[2 * i + 1];
            }
          }
        }
      };

      const Item mine = now;
      for (bool more = true; more;) {
        const Scales<GPB> st0 = scale0, st1 = scale1;
        const int blocks = min(SB, a.blocks - stage_now * SB);
        const int k = (stage_now - first) * SB;  // its first block in the epoch's x
        more = left_now > 1;
        at_hand = next;
        now = it;
        stage_now = stage;
        left_now = left;
        const bool ahead = next < end;  // a copy into the other slot
        fetch();
        if (!lost && !arrives(bar + use * 8, phase)) {
          lost = true;
          report_error(a.err, DEV_ERR_TIMEOUT, static_cast<int>(blockIdx.x));
          if (lane == 0) {  // whose copies they are
            arrives(bar + use * 8, phase);
            if (ahead) arrives(bar + (use ^ 1) * 8, phase ^ use);
          }
        }
        const uint32_t src = ring + use * kStage + lane * 16, xb = x_lane + k * 256;
        if (blocks == SB) {
#pragma unroll
          for (int b = 0; b < SB; ++b) block(src, xb, st0, st1, b);
        } else {
#pragma unroll 1
          for (int b = 0; b < blocks; ++b) block(src, xb, st0, st1, b);
        }
        phase ^= use;
        use ^= 1;
      }

      // ---- the warps' sums, added in order ----
      float* all = red + (group * 2 + buf) * wk * kRed;
#pragma unroll
      for (int i = 0; i < XR; ++i) {
        all[w_in * kRed + i * 64 + lane] = acc[0][i];
        all[w_in * kRed + i * 64 + 32 + lane] = acc[1][i];
      }
      if (wk == 1) __syncwarp();
      else asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(wk * 32) : "memory");
      for (int i = w_in * 32 + lane; i < XR * 32; i += wk * 32) {
        const int l = i & 31, c = i >> 5, r = XR * (l & 3) + c;
        if (r >= row_count) continue;
        const float* p = all + c * 64 + l;
        float low = 0.f, high = 0.f;
        for (int w = 0; w < wk; ++w) {
          low += p[w * kRed];
          high += p[w * kRed + 32];
        }
        put<MODE>(a, plan, mine.part, row_first, r, mine.tile * kTile + (l >> 2), low, high);
      }
      buf ^= 1;
    }
    epoch.next(to - from, a);
    from = to;
  }
}

}  // namespace w4
}  // namespace moe

#include "w4_wide.cuh"

namespace moe {
namespace w4 {

// How an item's inputs are shared out.  A warp's time is about its blocks, and
// four more for the item's ends; a launch takes as many rounds as the warps at
// once need for all items.
struct Share {
  int wk;
  int64_t cost;
};
// stages: of a part, rest: some parts have one more; every warp of an item has some.
inline Share share_narrow(int64_t items, int stages, bool rest) {
  const int64_t each_sm = (items + kSms - 1) / kSms;
  Share best = {1, int64_t{1} << 62};
  for (int wk = 1; wk <= kNarrowWarps; wk *= 2) {
    const int each = (stages + wk - 1) / wk, each_rest = (stages + wk) / wk;
    if ((wk - 1) * each >= stages || (rest && (wk - 1) * each_rest > stages)) continue;
    const int64_t groups = kNarrowWarps / wk, rounds = (each_sm + groups - 1) / groups;
    const int64_t cost = rounds * ((rest ? each_rest : each) * 4 + 4);
    if (cost < best.cost) best = {wk, cost};
  }
  return best;
}
// blocks: of inputs, of the longest part; an item's ends cost about four more (64
// tokens, 8 experts of 4096 x 14336: FC2 whole 201 us, in 2 parts 200, in 7, with a
// better balance, 206)
inline Share share_wide(int64_t items, int blocks) {
  return {1, (items + kSms - 1) / kSms * (blocks + 4)};
}
// Parts of a row that are items of their own, where whole rows would leave
// warps idle; `join`: what adding the parts up costs.
constexpr int kMostSplits = 8;
inline int splits_of(int64_t chunks, int N, int blocks, int join, bool wide) {
  int best = 1;
  int64_t least = int64_t{1} << 62;
  const int tile = wide ? 256 : 16;
  const int64_t items = chunks * ((N + tile - 1) / tile);
  const int units = (blocks + 3) / 4;
  for (int s = 1; s <= kMostSplits && s <= units; ++s) {
    const Share h = wide ? share_wide(items * s, (units + s - 1) / s * 4)
                         : share_narrow(items * s, units / s, units % s != 0);
    const int64_t cost = h.cost + (s > 1 ? join : 0);
    if (cost < least) {
      least = cost;
      best = s;
    }
  }
  return best;
}

// The narrow kernel's x: bytes of a column of the longest part; the columns' starts
// fall on the banks' halves in turn.
inline int part_blocks(int blocks, int splits) {
  return ((blocks + 3) / 4 + splits - 1) / splits * 4;
}
inline int narrow_x_pitch(int blocks, int splits) { return part_blocks(blocks, splits) * 256 + 64; }
// rows that a chunk of the narrow kernel can have; 0: none fits
inline int narrow_rows(int mode, int blocks, int splits) {
  const int cp = pieces_of(mode);
  const int64_t fit = kNarrowX / (static_cast<int64_t>(cp) * narrow_x_pitch(blocks, splits));
  return static_cast<int>(fit < 8 / cp ? fit : 8 / cp);
}

// The codes of `rows` rows as [blocks][rows][64 bytes]; boxes of 4 blocks, or of
// 2 with their 16-byte pieces swapped
bool map_codes(CUtensorMap* m, const uint8_t* codes, int64_t rows, int blocks, int box_rows,
               bool swapped);
// Columns of split x as [blocks of 64 inputs][columns][128 bytes], boxes of 2 and
// 8 columns
bool map_x(CUtensorMap* m, const __half* x, int64_t columns, int blocks);

template <int MODE, int G32, bool ZEROS, bool TAIL>
cudaError_t launch_narrow(Args a, cudaStream_t s) {
  const int tile = (MODE == FC1 ? 8 : 16);
  const size_t plan = MODE == LINEAR ? 0 : sizeof(Plan);
  a.tiles = (a.N + tile - 1) / tile;
  a.chunk_rows = narrow_rows(MODE, a.blocks, a.splits);
  const int64_t chunks = MODE == LINEAR ? (a.rows + a.chunk_rows - 1) / a.chunk_rows
                                         : (a.pairs < a.E ? a.pairs : a.E);  // about
  const int64_t items = chunks * a.tiles * a.splits;
  a.split_units = (a.blocks + 3) / 4 / a.splits;
  a.split_rest = (a.blocks + 3) / 4 % a.splits;
  constexpr auto k = w4_narrow_kernel<MODE, G32, ZEROS, TAIL>;
  const size_t smem = kNarrowWarps * 2 * 4096 +
                      2 * kNarrowWarps * (4 / pieces_of(MODE)) * 32 * 4 + kNarrowX + plan;
  const cudaError_t st = allow_most_smem<k>();
  if (st != cudaSuccess) return st;
  a.wk = share_narrow(items, a.split_units, a.split_rest != 0).wk;
  a.each = (a.split_units + a.wk - 1) / a.wk;
  a.each_rest = (a.split_units + a.wk) / a.wk;
  const int64_t all = static_cast<int64_t>(MODE == LINEAR ? 1 : a.E) * a.N;
  CUtensorMap m0, m1;
  if (!map_codes(&m0, a.w0.codes, all, a.blocks, MODE == FC1 ? 8 : 16, false) ||
      !map_codes(&m1, a.w1.codes, all, a.blocks, MODE == FC1 ? 8 : 16, false))
    return cudaErrorInvalidValue;
  a.x_pitch = narrow_x_pitch(a.blocks, a.splits);
  // no more blocks than the longest share of the items asks for: each holds x
  // (512 items: 128 blocks of 4 and not 152 of 3 or 4, 43.9 us instead of 45.8
  // for the experts of one token, 8 x 4096 x 14336)
  const int64_t each_sm = (items + kSms - 1) / kSms;
  const unsigned grid = static_cast<unsigned>((items + each_sm - 1) / each_sm);
  return launch_dependent(k, dim3(grid), dim3(kNarrowWarps * 32), smem, s, m0, m1, a);
}

// rows of a chunk of the wide kernel; few: 32 columns will do
constexpr int wide_rows(int mode, bool few) {
  return kTallColumns / (few ? 2 : 1) / pieces_of(mode);
}

template <int MODE, int G32>
cudaError_t launch_wide(Args a, cudaStream_t s) {
  const int tile = MODE == FC1 ? 128 : 256;
  a.tiles = (a.N + tile - 1) / tile;
  a.chunk_rows = wide_rows(MODE, a.few);
  const int64_t chunks = MODE == LINEAR ? (a.rows + a.chunk_rows - 1) / a.chunk_rows
                                         : (a.pairs < a.E ? a.pairs : a.E);  // about
  const int64_t items = chunks * a.tiles * a.splits;
  a.split_units = (a.blocks + 3) / 4 / a.splits;
  a.split_rest = (a.blocks + 3) / 4 % a.splits;
  constexpr auto k = w4_wide_kernel<MODE, G32>;
  const size_t smem = kTallSmem + (MODE == LINEAR ? 0 : sizeof(Plan));
  const cudaError_t st = allow_most_smem<k>();
  if (st != cudaSuccess) return st;
  const int64_t all = static_cast<int64_t>(MODE == LINEAR ? 1 : a.E) * a.N;
  const int64_t columns = static_cast<int64_t>(MODE == LINEAR ? a.rows : a.pairs) * pieces_of(MODE);
  CUtensorMap m0, m1, mx;
  if (!map_codes(&m0, a.w0.codes, all, a.blocks, 128, true) ||
      !map_codes(&m1, a.w1.codes, all, a.blocks, 128, true) ||
      !map_x(&mx, a.x, columns, a.blocks))
    return cudaErrorInvalidValue;
  const unsigned grid = static_cast<unsigned>(items < kSms ? items : kSms);
  return launch_dependent(k, dim3(grid), dim3(kTallRoles * 32), smem, s, m0, m1, mx, a);
}

template <int MODE, int G32>
cudaError_t launch_group(int K, bool wide, const Args& a, cudaStream_t s) {
  if (wide) return launch_wide<MODE, G32>(a, s);
  // K is a multiple of the group, and of 128 in the layer
  if constexpr (MODE == LINEAR && G32 < 4) {
    if (K % 128 != 0)
      return a.w0.zeros ? launch_narrow<MODE, G32, true, true>(a, s)
                        : launch_narrow<MODE, G32, false, true>(a, s);
  }
  return a.w0.zeros ? launch_narrow<MODE, G32, true, false>(a, s)
                    : launch_narrow<MODE, G32, false, false>(a, s);
}

template <int MODE>
cudaError_t launch_mode(int group, int K, bool wide, const Args& a, cudaStream_t s) {
  switch (group) {
    case 32: return launch_group<MODE, 1>(K, wide, a, s);
    case 64: return launch_group<MODE, 2>(K, wide, a, s);
    default: return launch_group<MODE, 4>(K, wide, a, s);
  }
}

// How a product of about `rows` rows of x (of an expert), `chunks` of them (of
// the experts hit) and N outputs is run.  The narrow kernel for as few rows as
// it can hold: 8 rows take it 10.2 us at 14336 x 4096, 15.7 at 14336 x 7168 and
// 25.0 at 57344 x 4096, and the wide one, which is nearly the same from one row
// to 16, takes 14.7, 21.6 and 33.9 for 9.  For 16 rows the narrow one would read
// the weights twice.  join: see splits_of, negative: no splits.
struct Way {
  bool wide, few;
  int splits;
};
inline Way way_of(int mode, int64_t rows, int64_t chunks, int N, int blocks, int join) {
  Way w = {true, rows * pieces_of(mode) <= kTallColumns / 2, 1};
  if (rows <= 8 / pieces_of(mode)) {
    w.splits = join < 0 ? 1 : splits_of(chunks, N, blocks, join, false);
    // more parts where the rows' x would not fit
    while (join >= 0 && narrow_rows(mode, blocks, w.splits) < rows && w.splits < kMostSplits)
      ++w.splits;
    w.wide = narrow_rows(mode, blocks, w.splits) < rows;
  }
  if (w.wide) w.splits = join < 0 ? 1 : splits_of(chunks, N, blocks, join, true);
  return w;
}

cudaError_t launch_linear(int group, int K, bool wide, const Args& a, cudaStream_t s);
cudaError_t launch_fc1(int group, int K, bool wide, const Args& a, cudaStream_t s);
cudaError_t launch_fc2(int group, int K, bool wide, const Args& a, cudaStream_t s);

}  // namespace w4
}  // namespace moe
