// The whole layer for a few tokens in one launch: router, capacity drops, SwiGLU
// experts (and a shared expert), combine.
//
// At up to 64 tokens the layer is bound by reading the weights of the experts that
// are hit, once: everything else has to stay out of that stream's way.  One
// cooperative grid, a block to an SM, goes through
//   logits: a block takes some features and up to 32 experts, partial sums out;
//   top-k: a block takes a token, adds its partial sums up and chooses (one token: every
//     block, which spares a barrier; 4 tokens so, 8 of 128 of 2048 x 768: 75 us and 72);
//     then every block builds the same plan (rows by expert, drops) in its shared memory;
//   FC1: the stream of all hit experts' W1 and W3, cut into equal runs of units;
//   hidden values: the last block to bring a partial sum of a tile adds them up, in
//     order, forms silu(a) b and counts the tile as done for its expert;
//   FC2: the stream of W2, an expert's part as soon as it is ready, cut the same way or
//     into pieces that blocks take in turn;
//   combine: partial sums of a token's experts added in order, one rounding.
// The barriers of all blocks are those around the top-k and the one before the combine:
// a block's parts of the two streams are nearly the same experts', so that a slow
// block delays its neighbours alone (with a barrier on either side of a step for the
// hidden values, 32 tokens, 8 of 128 experts of 4096 x 1536, took 762 us where this took
// 718).
// A block's part of both streams is one sequence of units, a unit 32 (fp32: 16) inputs of
// a tile's 512 outputs, 64 (32) to each of its 8 (16) warps.  A warp copies its own units
// with cp.async into a ring of its own, up to kSlots - 1 units ahead, from FC1 into FC2
// too: the weights do not depend on the hidden values, so memory stays busy while those
// are waited for.
//
// Measured, all of a call: 1 token, 2 of 8 experts of 4096 x 14336 bf16, 129 us (the bytes
// at the copy rate: 105); 8 tokens 400 (379); 32 tokens, 8 of 128 of 4096 x 1536, 689 (630).
// The 20 to 25 us above the bytes are the logits, two or three barriers, the plan and the
// combine, through most of which memory idles.  Registers are short: bf16 takes 255 and
// spills 24 bytes (48 with pieces), fp32 128 and 556.
//
// The products are mma.sync with the weights as the operand of 16 rows and 8 tokens as
// the columns.  The tensor cores' rate does not matter here (tcgen05 would need 128 rows
// and its operands in another layout than the stream's): a unit feeds 8 instructions for
// every 8 tokens.
//   bf16: weights by ldmatrix.trans out of the ring, whose 16-byte pieces are swapped so
//     that it meets no bank twice; the inputs of 32 are permuted between the instructions
//     so that a lane's share of x is 16 bytes in a row.  A hidden value enters FC2 as two
//     bf16 numbers (together within 2^-17 of it), so nothing between x and y is rounded to
//     16 bits but y.  Before that it is within 4.5e-5 of the RMS (the pieces, and sums that
//     the instruction cuts off); 0.4 to 0.7% of the results are not the nearest bf16 number.
//   fp32: each operand as two tf32 numbers, v = p + q with |q| <= 2^-11 |v| and q itself
//     rounded (2^-22 of v); p p', p q' and q p' are multiplied, q q' (2^-22) is left out.
//     FMAs, two outputs to a lane, took longer from the first row on (7 tokens, 3 of 12 of
//     1032 x 1416: 126 us where this took 71; 64 tokens, 2 of 8 of 1024 x 4096: 782 and
//     168).  An infinity gives NaN, and so does a number within 2^-12 of the largest one,
//     which rounds up to it.
//     From 9 rows on the issue slots bound it: each of 16 warps splits the same x anew, and
//     the sums of 64 rows spill.  64 tokens, 4 of 16 of 2048 x 1408: 221 us (the bytes 83), and
//     443 where one expert has more than 32 of the rows.
//
// All partial sums are added in an order given by sizes alone: repeats are equal
// bit for bit.
#include <type_traits>

#include "topk.cuh"

namespace moe {
namespace {

constexpr int kSlots = 6;                       // units of a warp's ring
constexpr int kRing = kSlots * 32 * 1024;       // of all warps: 192 KB
constexpr int kTokens = MOE_FEW_MAX_TOKENS;
constexpr int kPairs = kTokens * MOE_MAX_TOPK;
constexpr int kRowsAtMost = kPairs + kTokens;
constexpr int kGroups = kPairs / 64;
constexpr int kChunk = 384;                     // features of the router's operands at a time
constexpr int kColumns = 512;                   // a tile's outputs: all warps'
constexpr int kMostThreads = 512;
constexpr int kInPieces = 2;                    // tiles of FC2 to a block from which on pieces pay
constexpr int kLargePieces = 304, kSmallPieces = 304;  // at most
// a grid barrier gives up after about a second
constexpr long long kWaitCycles = 2000000000ll;

static_assert(kChunk * (32 + kTokens) * 4 <= kRing, "router operands");

struct Args {
  int T, h, E, k, f, fs;
  int score, groups, group_topk, capacity, policy;  // capacity < 0: no drops
  const void *x, *W1, *W3, *W2, *V1, *V3, *V2;      // V: the shared expert's
  const float *Wg, *gate_bias, *expert_bias;
  void* y;
  int32_t* idx_out;
  float* prob_out;
  int32_t* tpe_out;
  // workspace
  int* err;
  int* bar;  // barrier count, blocks gone
  float* logits;
  int32_t* idx;
  float* prob;
  float* main[2];   // of a product: partial sums that begin a tile, rows x outputs
  float* extra[2];  // those that go on with one: [run][T][512]
  int* tiles;       // partial sums that a tile of FC1 has
  int* ready;       // tiles of an expert whose hidden values are there
  int* queue;       // pieces of FC2 that were taken
  int counters;     // of the three
  void* hid;     // [rows, f]; bf16: twice (the second pieces)
  int64_t hid_lo;
};

struct Plan {
  int pairs, rows, hits;             // routed rows, experts hit
  int16_t expert[kPairs];            // -1: none
  float prob[kPairs];
  int16_t row_of[kPairs];            // -1: none
  uint16_t token[kRowsAtMost];       // of a row (the shared expert's behind the routed)
  int16_t hit_of_row[kRowsAtMost];
  int16_t hit[MOE_MAX_EXPERTS];      // experts hit
  int16_t first[MOE_MAX_EXPERTS + 1];  // their first rows
  int16_t total[MOE_MAX_EXPERTS], start[MOE_MAX_EXPERTS], hit_of[MOE_MAX_EXPERTS];
  int16_t before[kGroups][MOE_MAX_EXPERTS];  // of 64 pairs each
  uint8_t rank[kPairs];
  float logit[MOE_MAX_EXPERTS], gsel[MOE_MAX_EXPERTS];
  float part[kMostThreads];
  int taken[kLargePieces + kSmallPieces + 1];  // this block's pieces, in turn; -1: not yet
  int on, dropped;
};

// ------------------------------------------------------------------ the grid
__device__ __forceinline__ int load_acquire(const int* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// What thread 0 finds out for its block it leaves in plan.on.  Whoever writes that word has
// a barrier of the block before it, since warps may still be reading what was there, and
// one after it.  (As the result of the barrier itself, without a word: fp32 spills more,
// 7 tokens, 3 of 12 of 1032 x 1416, 69.9 us where this takes 67.9, 64 tokens, 2 of 8 of
// 1024 x 2048, 115 and 108; bf16 alike.)

// The n-th barrier of all blocks.  false, for the whole block, where the wait ran out.
__device__ bool grid_barrier(const Args& a, Plan& plan, int n) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    atomicAdd(a.bar, 1);
    const int want = n * static_cast<int>(gridDim.x);
    const long long began = clock64();
    int on = 1;
    while (load_acquire(a.bar) < want)
      if (clock64() - began > kWaitCycles) {
        report_error(a.err, DEV_ERR_TIMEOUT, n);
        on = 0;
        break;
      }
    plan.on = on;
  }
  __syncthreads();
  return plan.on != 0;
}

// Until an expert's hidden values are there.  false as above.
__device__ bool expert_ready(const Args& a, Plan& plan, int hit, int tiles) {
  __syncthreads();  // tile_done's word is read
  if (threadIdx.x == 0) {
    const long long began = clock64();
    int on = 1;
    while (load_acquire(a.ready + hit) < tiles)
      if (clock64() - began > kWaitCycles) {
        report_error(a.err, DEV_ERR_TIMEOUT, hit);
        on = 0;
        break;
      }
    plan.on = on;
  }
  __syncthreads();
  const bool on = plan.on != 0;
  __syncthreads();
  return on;
}

// The last block to leave sets the counters back, a wait that ran out or not.
__device__ void leave(const Args& a) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(a.bar + 1, 1) == static_cast<int>(gridDim.x) - 1) {
      a.bar[0] = 0;
      a.bar[1] = 0;
      __threadfence();
    }
  }
}

// ------------------------------------------------------------------ copies
__device__ __forceinline__ uint32_t smem_at(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(real ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A warp's unit: kInputs inputs of 128 bytes of outputs each.  More warps hide more of
// what fp32 needs between the ring and the products (8 tokens, 2 experts of 2048 x 8192:
// 100 us with 16 warps, 108 with 8); bf16 with 16 warps of 64 bytes of outputs takes
// longer (one token, 2 of 8 of 4096 x 14336: 145 us and 130).
template <typename T>
struct Form;
template <>
struct Form<__nv_bfloat16> {
  static constexpr int kWarps = 8, kInputs = 32;
  // rows read together by ldmatrix differ in bits 0, 3 and 4 of the input
  __device__ static int place(int row, int piece) {
    return row * 128 + ((piece ^ (((row >> 3) & 3) * 2 + (row & 1))) << 4);
  }
};
template <>
struct Form<float> {
  static constexpr int kWarps = 16, kInputs = 16;
  // rows read together differ in bits 2 and 3 of the input, eight outputs of each
  __device__ static int place(int row, int piece) {
    return row * 128 + ((piece ^ (((row >> 2) & 3) * 2)) << 4);
  }
};

template <typename T>
struct Shape : Form<T> {
  static constexpr int kWarps = Form<T>::kWarps, kThreads = kWarps * 32;
  static constexpr int kInputs = Form<T>::kInputs;
  static constexpr int kStrip = 128 / sizeof(T);   // outputs of a unit
  static constexpr int kUnit = kInputs * 128;      // bytes
  static constexpr int kPieces = 8;                // of 16 bytes
  static constexpr int kCopies = kUnit / 512;      // instructions
  static_assert(kWarps * kStrip == kColumns && kWarps * kSlots * kUnit == kRing, "units");
};

// ------------------------------------------------------------------ the streams
// One product's stream: tiles of 512 outputs (FC1: 256 of W1 and the same of W3), an
// expert's one after another, the shared expert's last; a tile's units follow the
// inputs.  They are cut into equal runs, one to a block.  Units are counted in 32 bits:
// 2^31 of 32 KB are past any memory (the caller checks).
//
// Memory serves some blocks up to a fifth slower than others, and those with many rows have
// more to store.  So of a large bf16 FC2 the blocks' runs are a quarter, and the rest is
// pieces, the small ones last, which blocks take as they come to them: 8, 16, 32 and 64
// tokens, 8 of 128 experts of 4096 x 1536, take 328, 529, 689 and 769 us, in one run to a
// block 337, 547, 716 and 833; 32 tokens, 8 of 64 of 7168 x 2048 and a shared one, 922 and
// 1218.  More partial sums go to the combine: where a block has less than two tiles, or
// tiles are long, that costs more than it gives (1 and 4 tokens of the first layer: 88 and
// 211 us where one run takes 77 and 209; 64 tokens, 2 of 8 of 4096 x 14336: 566 and 557),
// and fp32, which has no registers left for it, is slower by 20 us.  Which piece goes to
// which block differs between calls, the pieces and the order of their sums do not.
struct Stream {
  int S, begin, end;
  int tiles, units;        // of a routed expert; of a tile
  int routed;              // tiles of all of them
  int shared_tiles;        // of the shared expert
  int shared_units;        // of one of the shared expert's tiles
  int routed_units;
  int each, rest;          // units of a block's run; the first `rest` blocks have one more
  int fixed, n0;           // units of all blocks' runs, and how many have any
  int q1, n1, q2, n2;      // the rest: n1 pieces of q1 units, then n2 of q2 (the last fewer)

  __device__ void set(int hits, int tiles_, int units_, int shared_tiles_, int shared_units_,
                      bool in_pieces) {
    tiles = tiles_, units = units_, shared_tiles = shared_tiles_, shared_units = shared_units_;
    routed = hits * tiles;
    routed_units = routed * units;
    S = fixed = routed_units + shared_tiles * shared_units;
    const int G = gridDim.x, b = blockIdx.x;
    q1 = q2 = 1, n1 = n2 = 0;
    if (in_pieces && routed + shared_tiles >= kInPieces * G) {
      const int small = S / 8, large = S / 8 * 5;
      q2 = max(6, (small + kSmallPieces - 1) / kSmallPieces);
      n2 = (small + q2 - 1) / q2;
      q1 = max(8, (large + kLargePieces - 1) / kLargePieces);
      n1 = large / q1;
      fixed = S - small - n1 * q1;
    }
    each = fixed / G, rest = fixed - each * G;
    n0 = min(G, fixed);
    begin = b * each + min(b, rest);
    end = begin + each + (b < rest);
  }
  __device__ void find(int u, int& tile, int& unit) const {
    if (u < routed_units) {
      tile = u / units;
      unit = u - tile * units;
    } else {
      const int t = (u - routed_units) / shared_units;
      tile = routed + t;
      unit = u - routed_units - t * shared_units;
    }
  }
  __device__ int units_of(int tile) const { return tile < routed ? units : shared_units; }
  __device__ void piece(int p, int& from, int& to) const {
    if (p < n1) {
      from = fixed + p * q1;
      to = from + q1;
    } else {
      from = fixed + n1 * q1 + (p - n1) * q2;
      to = min(S, from + q2);
    }
  }
  // the blocks' runs (empty ones not counted), then the pieces
  __device__ int run_of(int u) const {
    const int longer = rest * (each + 1);
    if (u < longer) return u / (each + 1);
    if (u < fixed) return rest + (u - longer) / each;
    u -= fixed;
    return u < n1 * q1 ? n0 + u / q1 : n0 + n1 + (u - n1 * q1) / q2;
  }
  // the runs that have a tile's units
  __device__ void runs(int tile, int& first, int& last) const {
    const int u =
        tile < routed ? tile * units : routed_units + (tile - routed) * shared_units;
    first = run_of(u);
    last = run_of(u + units_of(tile) - 1);
  }
};

// What a tile is: its expert (plan.hits: the shared one) and its place among the
// expert's outputs.
struct Tile {
  int hit, at, rows, first;
};
__device__ __forceinline__ Tile tile_of(const Args& a, const Plan& plan, const Stream& s, int tile) {
  Tile t;
  if (tile < s.routed) {
    t.hit = tile / s.tiles;
    t.at = tile - t.hit * s.tiles;
    t.first = plan.first[t.hit];
    t.rows = plan.first[t.hit + 1] - t.first;
  } else {
    t.hit = plan.hits;
    t.at = tile - s.routed;
    t.first = plan.rows;
    t.rows = a.T;
  }
  return t;
}

// A block's next piece, the same for all its warps: the first that asks for it takes it.
__device__ __noinline__ int take_piece(int* queue, int* turn, int none, int* err) {
  int p = none;
  if ((threadIdx.x & 31) == 0) {
    volatile int* mine = turn;
    p = *mine;
    if (p == -1 && atomicCAS(turn, -1, -2) == -1) {
      p = atomicAdd(queue, 1);
      *mine = p;
    } else if (p < 0) {
      const long long began = clock64();
      while ((p = *mine) < 0)
        if (clock64() - began > kWaitCycles) {
          report_error(err, DEV_ERR_TIMEOUT, none);
          p = none;
          break;
        }
    }
  }
  p = __shfl_sync(~0u, p, 0);
  __syncwarp();
  return p;
}

// A warp's copies: both streams' units in order.  QUEUE: FC2's in pieces too.
template <typename T, bool QUEUE>
struct Copies {
  using F = Shape<T>;
  static constexpr int kStep = 32 / F::kPieces;  // inputs of an instruction
  const Args& a;
  Plan& plan;
  const Stream* streams;
  uint32_t ring;      // this lane's place in a slot
  int product = 0, left = 0, slot = 0;
  int turn = 0;       // pieces so far; -1: no more
  int next = 0;       // unit
  int unit = 0, units = 0, inputs = 0, outputs = 0;
  bool real = false;
  const T* src = nullptr;
  int dst[F::kCopies];

  __device__ Copies(const Args& a_, Plan& p, const Stream* s, const void* smem)
      : a(a_), plan(p), streams(s) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    ring = smem_at(smem) + warp * kSlots * F::kUnit;
#pragma unroll
    for (int i = 0; i < F::kCopies; ++i)
      dst[i] = F::place(lane / F::kPieces + i * kStep, lane % F::kPieces);
    left = s[0].end - s[0].begin;
    next = s[0].begin;
  }

  __device__ void enter(int tile, int unit_) {
    const Stream& s = streams[product];
    const Tile t = tile_of(a, plan, s, tile);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool shared = t.hit == plan.hits;
    const int f = shared ? a.fs : a.f;
    const void* W;
    int column;
    if (product == 0) {
      inputs = a.h, outputs = f;
      column = t.at * 256 + warp % (F::kWarps / 2) * F::kStrip;
      W = shared ? (warp < F::kWarps / 2 ? a.V1 : a.V3) : (warp < F::kWarps / 2 ? a.W1 : a.W3);
    } else {
      inputs = f, outputs = a.h;
      column = t.at * kColumns + warp * F::kStrip;
      W = shared ? a.V2 : a.W2;
    }
    column += lane % F::kPieces * (16 / static_cast<int>(sizeof(T)));
    real = column < outputs;
    const int64_t e = shared ? 0 : plan.hit[t.hit];
    const int row = unit_ * F::kInputs + lane / F::kPieces;
    src = static_cast<const T*>(W) +
          (real ? (e * inputs + row) * outputs + column : int64_t{0});
    unit = unit_;
    units = s.units_of(tile);
  }

  // What comes after a run: FC2's own run, then the pieces that the block takes.
  __device__ __forceinline__ void next_run() {
    unit = units = 0;
    const Stream& s = streams[1];
    if (product == 0) {
      product = 1;
      next = s.begin;
      left = s.end - s.begin;
      if (left > 0) return;
    }
    const int n = QUEUE ? s.n1 + s.n2 : 0;
    const int p = n > 0 ? take_piece(a.queue, &plan.taken[turn], n, a.err) : n;
    ++turn;
    if (p < n) {
      int to;
      s.piece(p, next, to);
      left = to - next;
    } else {
      turn = -1;
    }
  }

  // the next unit, if there is one, and a group in any case
  __device__ __forceinline__ void issue() {
    if (left == 0 && turn >= 0) next_run();
    if (left > 0) {
      if (unit == units) {
        int tile, u;
        streams[product].find(next, tile, u);
        enter(tile, u);
      }
      const int row = unit * F::kInputs + (threadIdx.x & 31) / F::kPieces;
      const uint32_t to = ring + slot * F::kUnit;
#pragma unroll
      for (int i = 0; i < F::kCopies; ++i) {
        const bool there = real && row + i * kStep < inputs;
        copy16(to + dst[i], there ? src + static_cast<int64_t>(i) * kStep * outputs : src, there);
      }
      if (real) src += static_cast<int64_t>(F::kInputs) * outputs;
      ++unit;
      ++next;
      --left;
      if (++slot == kSlots) slot = 0;
    }
    commit();
  }
};

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                               uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// v as two tf32 numbers: the nearest (halves away from zero, by the carry of half a
// step), and that of the rest, whose last bits the instruction does not read.
__device__ __forceinline__ void two_tf32(uint32_t v, uint32_t& p, uint32_t& q) {
  p = (v + 0x1000u) & 0xffffe000u;
  q = __float_as_uint(__uint_as_float(v) - __uint_as_float(p)) + 0x1000u;
}
__device__ __forceinline__ uint32_t load_shared(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

// Not through the read-only path: hidden values are written by this launch.
__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// Where a run's sums of a tile go: the row `n` of the tile's, an output of the warp's.
struct Out {
  float* at;
  int64_t stride;
  int limit;  // outputs from `at` on
};

// A run of units of one tile, up to 8 NT rows, PIECES numbers to an input of bf16.
// x: the rows' inputs from this run's first on; `left`: how many there are.
template <typename T, bool QUEUE, int NT, int PIECES>
__device__ __forceinline__ void run_units(Copies<T, QUEUE>& copies, int& slot, int units,
                                          const T* x, int64_t x_lo, const uint16_t* row_at,
                                          int first, int count, int width, int left,
                                          const Out& out) {
  using F = Shape<T>;
  constexpr bool kHalf = sizeof(T) == 2;
  constexpr int kLane = F::kInputs / 4;  // inputs of a lane: 16 bytes
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  constexpr int M = F::kStrip / 16;
  float acc[M][NT][4];
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;
  // rows past the last one repeat it; their sums are not stored
  uint32_t off[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = first + min(n * 8 + g, count - 1);
    off[n] = (row_at ? static_cast<uint32_t>(row_at[r]) : static_cast<uint32_t>(r - first)) *
                 static_cast<uint32_t>(width) + t * kLane;
  }
  // The unit's inputs are kLane to each t.  bf16: instruction s takes 8 t + 4 s .. + 3, its
  // slots 2 t, 2 t + 1 the first two and 2 t + 8, 2 t + 9 the others.  fp32: 4 t + 2 s, + 1,
  // the slots t and t + 4.
  uint32_t from[2][M];
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int m = 0; m < M; ++m) {
      if (kHalf) {
        const int j = lane >> 3, r = lane & 7;
        from[s][m] = F::place(8 * (r >> 1) + 2 * (j >> 1) + (r & 1) + 4 * s, m * 2 + (j & 1));
      } else {
        from[s][m] = F::place(4 * t + 2 * s, m * 4 + (g >> 2)) + (g & 3) * 4;
      }
    }

  auto read = [&](uint4 (&v)[NT], int p, int at) {  // inputs past the row's end are none
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (kHalf) {
        v[n] = load16(x + p * x_lo + at + off[n]);
      } else {
        v[n] = make_uint4(0u, 0u, 0u, 0u);
        if (at + t * kLane < left) v[n] = load16(x + at + off[n]);
      }
    }
  };
  constexpr bool kAhead = NT * PIECES <= 4;  // as the registers allow
  uint4 ahead[PIECES][NT];
  if (kAhead)
#pragma unroll
    for (int p = 0; p < PIECES; ++p) read(ahead[p], p, 0);
#pragma unroll 1
  for (int u = 0; u < units; ++u) {
    uint4 now[PIECES][NT];  // without kAhead one piece after the other, in the first place
    if (kAhead) {
#pragma unroll
      for (int p = 0; p < PIECES; ++p)
#pragma unroll
        for (int n = 0; n < NT; ++n) now[p][n] = ahead[p][n];
      if (u + 1 < units)
#pragma unroll
        for (int p = 0; p < PIECES; ++p) read(ahead[p], p, (u + 1) * F::kInputs);
    } else {
      read(now[0], 0, u * F::kInputs);
    }
    wait_copies<kSlots - 2>();
    __syncwarp();
    copies.issue();  // into the slot that was read last
    const uint32_t at = copies.ring + slot * F::kUnit;
    if (++slot == kSlots) slot = 0;
    if constexpr (kHalf) {
      uint32_t w[2][M][4];
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int m = 0; m < M; ++m) ldmatrix_x4_trans(at + from[s][m], w[s][m]);
#pragma unroll
      for (int p = 0; p < PIECES; ++p) {
        if (!kAhead && p > 0) read(now[0], p, u * F::kInputs);
        const uint4(&v)[NT] = now[kAhead ? p : 0];
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int m = 0; m < M; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma_bf16(acc[m][n], w[s][m], s ? v[n].z : v[n].x, s ? v[n].w : v[n].y);
      }
    } else {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        uint32_t wp[M][4], wq[M][4];
#pragma unroll
        for (int m = 0; m < M; ++m) {
          // outputs g and g + 8 of 16 (two pieces on), inputs of the slots t and t + 4
          const uint32_t q = at + from[s][m], q8 = at + (from[s][m] ^ 32);
          two_tf32(load_shared(q), wp[m][0], wq[m][0]);
          two_tf32(load_shared(q8), wp[m][1], wq[m][1]);
          two_tf32(load_shared(q + 128), wp[m][2], wq[m][2]);
          two_tf32(load_shared(q8 + 128), wp[m][3], wq[m][3]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          uint32_t xp[2], xq[2];
          two_tf32(s ? now[0][n].z : now[0][n].x, xp[0], xq[0]);
          two_tf32(s ? now[0][n].w : now[0][n].y, xp[1], xq[1]);
#pragma unroll
          for (int m = 0; m < M; ++m) {
            // the instruction cuts its sums off, so that a long chain of them falls short:
            // eight inputs at a time, added up with rounding
            float part[4];
            mma_tf32_first(part, wp[m], xq[0], xq[1]);
            mma_tf32(part, wq[m], xp[0], xp[1]);
            mma_tf32(part, wp[m], xp[0], xp[1]);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][n][i] += part[i];
          }
        }
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int at = n * 8 + t * 2 + c;
      if (at < count) {
        float* o = out.at + at * out.stride;
#pragma unroll
        for (int m = 0; m < M; ++m) {
          if (m * 16 + g < out.limit) o[m * 16 + g] = acc[m][n][c];
          if (m * 16 + g + 8 < out.limit) o[m * 16 + g + 8] = acc[m][n][2 + c];
        }
      }
    }
}

// ------------------------------------------------------------------ the steps
__device__ __forceinline__ float as_float(float v) { return v; }
__device__ __forceinline__ float as_float(__nv_bfloat16 v) { return __bfloat162float(v); }

__host__ __device__ inline int expert_tiles(int E) { return (E + 31) / 32; }
__host__ __device__ inline int slabs(int G, int E, int h) {
  const int n = G / expert_tiles(E);
  return n < 1 ? 1 : n < h / 8 ? n : h / 8;
}

// Partial logits [slab][T][E] of this block's features and experts.
template <typename T>
__device__ void partial_logits(const Args& a, char* smem) {
  const int tiles = expert_tiles(a.E), n_slabs = slabs(gridDim.x, a.E, a.h);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kWarps = Shape<T>::kWarps;
  // more than G tiles of experts only where the grid is smaller than 8 blocks
  for (int job = blockIdx.x; job < tiles * n_slabs; job += gridDim.x) {
    const int e0 = job % tiles * 32, slab = job / tiles;
    const int width = a.E > 16 ? 32 : a.E > 8 ? 16 : 8;  // lanes of experts
    const int ne = min(32, a.E - e0);
    const int begin = static_cast<int>(static_cast<int64_t>(a.h / 8) * slab / n_slabs) * 8;
    const int end = static_cast<int>(static_cast<int64_t>(a.h / 8) * (slab + 1) / n_slabs) * 8;
    const int Tp = a.T <= 16 ? 16 : a.T <= 32 ? 32 : 64;
    float* ws = reinterpret_cast<float*>(smem);                 // [rows][32]
    float* xs = reinterpret_cast<float*>(smem) + kChunk * 32;   // [rows][Tp]
    const int tg = warp % (Tp / 16), splits = kWarps / (Tp / 16) * (32 / width);
    const int split = warp / (Tp / 16) * (32 / width) + lane / width, le = lane % width;
    float acc[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.f;
    for (int r0 = begin; r0 < end; r0 += kChunk) {
      const int rows = min(kChunk, end - r0);
      __syncthreads();
      if (ne == 32 && a.E % 4 == 0) {
        for (int i = threadIdx.x; i < rows * 8; i += blockDim.x)
          copy16(smem_at(ws + i * 4),
                 a.Wg + static_cast<int64_t>(r0 + i / 8) * a.E + e0 + i % 8 * 4, true);
      } else {
        for (int i = threadIdx.x; i < rows * 32; i += blockDim.x)
          if (i % 32 < ne)
            copy4(smem_at(ws + i), a.Wg + static_cast<int64_t>(r0 + i / 32) * a.E + e0 + i % 32);
      }
      commit();
      constexpr int V = 16 / sizeof(T);
      for (int i = threadIdx.x; i < rows / V * a.T; i += blockDim.x) {
        const int t = i % a.T, r = i / a.T * V;
        const uint4 q = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(a.x) +
                                                             static_cast<int64_t>(t) * a.h + r0 + r));
        T v[V];
        memcpy(v, &q, 16);
#pragma unroll
        for (int j = 0; j < V; ++j) xs[(r + j) * Tp + t] = as_float(v[j]);
      }
      wait_copies<0>();
      __syncthreads();
      if (le < ne)
        for (int r = split; r < rows; r += splits) {
          const float w = ws[r * 32 + le];
          const float4* q = reinterpret_cast<const float4*>(xs + r * Tp + tg * 16);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 v = q[i];  // past T: not stored
            acc[i * 4] = fmaf(v.x, w, acc[i * 4]);
            acc[i * 4 + 1] = fmaf(v.y, w, acc[i * 4 + 1]);
            acc[i * 4 + 2] = fmaf(v.z, w, acc[i * 4 + 2]);
            acc[i * 4 + 3] = fmaf(v.w, w, acc[i * 4 + 3]);
          }
        }
    }
    __syncthreads();
    float* red = reinterpret_cast<float*>(smem);  // [split][Tp][width]
#pragma unroll
    for (int i = 0; i < 16; ++i) red[(split * Tp + tg * 16 + i) * width + le] = acc[i];
    __syncthreads();
    for (int i = threadIdx.x; i < a.T * ne; i += blockDim.x) {
      const int t = i / ne, e = i % ne;
      float sum = 0.f;
      for (int s = 0; s < splits; ++s) sum += red[(s * Tp + t) * width + e];
      a.logits[(static_cast<int64_t>(slab) * a.T + t) * a.E + e0 + e] = sum;
    }
    __syncthreads();
  }
}

// A token's experts, by one warp; logits in plan.logit.  own: into this block's plan.
template <int PL>
__device__ void choose(const Args& a, Plan& plan, int t, bool own) {
  const int lane = threadIdx.x & 31;
  float s[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int e = lane + 32 * i;
    s[i] = e < a.E ? plan.logit[e] : -FLT_MAX;
  }
  int idx;
  float p;
  choose_topk<PL>(s, t, a.E, a.k, a.score, a.groups, a.group_topk, a.expert_bias, plan.gsel,
                  a.err, idx, p);
  // A token without k experts to choose (NaN logits, reported) names one twice: the first
  // of them stands, so that no expert has more rows than there are tokens.
  const uint32_t same = __match_any_sync(~0u, lane < a.k ? idx : -1 - lane);
  if (lane >= a.k) return;
  const int i = t * a.k + lane, e = __ffs(same) - 1 == lane ? idx : -1;
  if (own) {
    plan.expert[i] = static_cast<int16_t>(e);
    plan.prob[i] = p;
    if (blockIdx.x != 0) return;
  } else {
    a.idx[i] = e;
    a.prob[i] = p;
  }
  if (a.idx_out) a.idx_out[i] = idx;
  if (a.prob_out) a.prob_out[i] = p;
}

// own: every block for the one token, else each block for its tokens.
__device__ void choose_experts(const Args& a, Plan& plan, bool own) {
  const int n_slabs = slabs(gridDim.x, a.E, a.h);
  int width = 8;
  while (width < a.E) width *= 2;
  const int parts = blockDim.x / width, e = threadIdx.x % width, part = threadIdx.x / width;
  const int warp = threadIdx.x >> 5;
  const float bias = a.gate_bias && threadIdx.x < a.E ? __ldg(a.gate_bias + threadIdx.x) : 0.f;
  for (int t = own ? 0 : blockIdx.x; t < a.T; t += gridDim.x) {
    float sum = 0.f;
    if (e < a.E) {
      const float* l = a.logits + static_cast<int64_t>(t) * a.E + e;
      for (int s = part; s < n_slabs; s += 16 * parts) {  // sixteen loads at a time
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int at = s + i * parts;
          v[i] = at < n_slabs ? __ldcg(l + static_cast<int64_t>(at) * a.T * a.E) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) sum += v[i];
      }
    }
    __syncthreads();
    plan.part[threadIdx.x] = sum;
    __syncthreads();
    if (threadIdx.x < a.E) {
      float l = 0.f;
      for (int i = 0; i < parts; ++i) l += plan.part[i * width + threadIdx.x];
      plan.logit[threadIdx.x] = a.gate_bias ? l + bias : l;
    }
    __syncthreads();
    if (warp == 0) {
      if (a.E <= 32) choose<1>(a, plan, t, own);
      else if (a.E <= 64) choose<2>(a, plan, t, own);
      else if (a.E <= 128) choose<4>(a, plan, t, own);
      else choose<8>(a, plan, t, own);
    }
  }
  __syncthreads();
}

// Rows by expert: pairs counted and ranked in their order, 64 of them to a warp.
__device__ void order_pairs(const Args& a, Plan& plan) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < kGroups * MOE_MAX_EXPERTS; i += blockDim.x)
    plan.before[i / MOE_MAX_EXPERTS][i % MOE_MAX_EXPERTS] = 0;
  __syncthreads();
  for (int r = 0; warp < kGroups && r < 2; ++r) {
    const int i = warp * 64 + r * 32 + lane;
    const int e = i < plan.pairs ? plan.expert[i] : -1;
    const uint32_t same = __match_any_sync(~0u, e);
    if (e >= 0) {
      const int base = plan.before[warp][e];
      plan.rank[i] = static_cast<uint8_t>(base + __popc(same & ((1u << lane) - 1)));
      __syncwarp(same);
      if (lane == __ffs(same) - 1) plan.before[warp][e] = static_cast<int16_t>(base + __popc(same));
    }
    __syncwarp();
  }
  __syncthreads();
  if (threadIdx.x < MOE_MAX_EXPERTS) {
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kGroups; ++w) {
      const int n = plan.before[w][threadIdx.x];
      plan.before[w][threadIdx.x] = static_cast<int16_t>(sum);
      sum += n;
    }
    plan.total[threadIdx.x] = static_cast<int16_t>(sum);
  }
  __syncthreads();
  if (threadIdx.x < 32) {  // eight experts to a lane
    int n[8], rows = 0, hits = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      n[i] = plan.total[lane * 8 + i];
      rows += n[i];
      hits += n[i] > 0;
    }
    int row = rows, hit = hits;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int r = __shfl_up_sync(~0u, row, o), q = __shfl_up_sync(~0u, hit, o);
      if (lane >= o) row += r, hit += q;
    }
    if (lane == 31) {
      plan.rows = row;
      plan.hits = hit;
      plan.first[hit] = static_cast<int16_t>(row);
    }
    row -= rows, hit -= hits;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      plan.start[lane * 8 + i] = static_cast<int16_t>(row);
      if (n[i] > 0) {
        plan.hit[hit] = static_cast<int16_t>(lane * 8 + i);
        plan.hit_of[lane * 8 + i] = static_cast<int16_t>(hit);
        plan.first[hit++] = static_cast<int16_t>(row);
        row += n[i];
      }
    }
  }
  __syncthreads();
}

// The plan of up to 8 pairs, by one warp: a pair to a lane, places by counting (one token,
// 8 of 128 of 2048 x 768: 37.2 us where the other takes 38.9; 32 pairs so: 34.5 and 32.9).
__device__ void plan_of_few(const Args& a, Plan& plan) {
  const int lane = threadIdx.x, pairs = plan.pairs;
  int e = lane < pairs ? plan.expert[lane] : -1;
  const uint32_t bits = lane < pairs ? __float_as_uint(plan.prob[lane]) : 0u;
  int place = 0, members = 0;
  if (a.capacity >= 0) {
    for (int q = 0; q < pairs; ++q) {
      const int oe = __shfl_sync(~0u, e, q);
      const uint32_t ob = __shfl_sync(~0u, bits, q);
      const bool before = a.policy == MOE_DROP_PROBS ? ob > bits || (ob == bits && q < lane) : q < lane;
      place += oe == e && before;
    }
    if (e >= 0 && place >= a.capacity) {
      e = -1;
      if (blockIdx.x == 0 && a.prob_out) a.prob_out[lane] = 0.f;
    }
  }
  // rows before this one, those of its expert, experts before its own
  int row = 0, hit = 0;
  bool leads = e >= 0;
  for (int q = 0; q < pairs; ++q) {
    const int oe = __shfl_sync(~0u, e, q);
    row += oe >= 0 && (oe < e || (oe == e && q < lane));
    members += oe == e;
    leads &= !(oe == e && q < lane);
  }
  for (int q = 0; q < pairs; ++q) {
    const int oe = __shfl_sync(~0u, e, q);
    const bool ol = __shfl_sync(~0u, static_cast<int>(leads), q);
    hit += ol && oe < e;
  }
  const int rows = __popc(__ballot_sync(~0u, e >= 0)), hits = __popc(__ballot_sync(~0u, leads));
  if (lane < pairs) {
    plan.expert[lane] = static_cast<int16_t>(e);
    plan.row_of[lane] = static_cast<int16_t>(e >= 0 ? row : -1);
  }
  if (e >= 0) {
    plan.token[row] = static_cast<uint16_t>(lane / a.k);
    plan.hit_of_row[row] = static_cast<int16_t>(hit);
  }
  if (leads) {
    plan.hit[hit] = static_cast<int16_t>(e);
    plan.first[hit] = static_cast<int16_t>(row);
  }
  if (lane == 0) {
    plan.rows = rows;
    plan.hits = hits;
    plan.first[hits] = static_cast<int16_t>(rows);
  }
  __syncwarp();
  for (int t = lane; t < a.T; t += 32) plan.token[rows + t] = static_cast<uint16_t>(t);
  if (blockIdx.x == 0 && a.tpe_out) {
    for (int i = lane; i < a.E; i += 32) a.tpe_out[i] = 0;
    __syncwarp();
    if (leads) a.tpe_out[e] = members;
  }
}

// Every block builds the same plan.  own: experts and weights are in it already.
__device__ void make_plan(const Args& a, Plan& plan, bool own) {
  const int pairs = a.T * a.k;
  if (threadIdx.x == 0) plan.pairs = pairs, plan.dropped = 0;
  if (!own)
    for (int i = threadIdx.x; i < pairs; i += blockDim.x) {
      plan.expert[i] = static_cast<int16_t>(__ldcg(a.idx + i));
      plan.prob[i] = __ldcg(a.prob + i);
    }
  __syncthreads();
  if (pairs <= MOE_MAX_TOPK) {
    if (threadIdx.x < 32) plan_of_few(a, plan);
    __syncthreads();
    return;
  }
  order_pairs(a, plan);
  if (a.capacity >= 0) {
    uint32_t marked = 0;  // of this thread's pairs, two at most
    for (int i = threadIdx.x, r = 0; i < pairs; i += blockDim.x, ++r) {
      const int e = plan.expert[i];
      if (e < 0 || plan.total[e] <= a.capacity) continue;
      int place = plan.before[i / 64][e] + plan.rank[i];
      if (a.policy == MOE_DROP_PROBS) {
        // a larger probability first, equal ones in token order (bits of numbers >= 0)
        const uint32_t p = __float_as_uint(plan.prob[i]);
        place = 0;
        for (int q = 0; q < pairs; ++q) {
          const uint32_t o = __float_as_uint(plan.prob[q]);
          place += plan.expert[q] == e && (o > p || (o == p && q < i));
        }
      }
      if (place >= a.capacity) marked |= 1u << r;
    }
    __syncthreads();
    for (int i = threadIdx.x, r = 0; i < pairs; i += blockDim.x, ++r)
      if (marked >> r & 1) {
        plan.expert[i] = -1;
        plan.dropped = 1;
        if (blockIdx.x == 0 && a.prob_out) a.prob_out[i] = 0.f;
      }
    __syncthreads();
    if (plan.dropped) order_pairs(a, plan);
  }
  for (int i = threadIdx.x; i < pairs; i += blockDim.x) {
    const int e = plan.expert[i];
    int row = -1;
    if (e >= 0) {
      row = plan.start[e] + plan.before[i / 64][e] + plan.rank[i];
      plan.token[row] = static_cast<uint16_t>(i / a.k);
      plan.hit_of_row[row] = plan.hit_of[e];
    }
    plan.row_of[i] = static_cast<int16_t>(row);
  }
  for (int t = threadIdx.x; t < a.T; t += blockDim.x)
    plan.token[plan.rows + t] = static_cast<uint16_t>(t);
  if (blockIdx.x == 0 && a.tpe_out)
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) a.tpe_out[e] = plan.total[e];
  __syncthreads();
}

// Partial sums of a row's outputs in main: FC1's two products side by side.
__device__ __forceinline__ float* main_row(const Args& a, const Plan& plan, int product, int row,
                                           bool shared) {
  if (product == 1) return a.main[1] + static_cast<int64_t>(row) * a.h;
  if (!shared) return a.main[0] + static_cast<int64_t>(row) * 2 * a.f;
  return a.main[0] + static_cast<int64_t>(plan.rows) * 2 * a.f +
         static_cast<int64_t>(row - plan.rows) * 2 * a.fs;
}
__device__ __forceinline__ int64_t hid_row(const Args& a, const Plan& plan, int row, bool shared) {
  if (!shared) return static_cast<int64_t>(row) * a.f;
  return static_cast<int64_t>(plan.rows) * a.f + static_cast<int64_t>(row - plan.rows) * a.fs;
}

// A row's sums of four neighbouring outputs of FC2, the runs in order.
__device__ __forceinline__ float4 sum_runs(const Args& a, const float* main, int first, int last,
                                           int row, int column) {
  float4 v = __ldcg(reinterpret_cast<const float4*>(main));
  for (int b = first + 1; b <= last; b += 8) {  // eight loads at a time
    float4 w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (b + i <= last)
        w[i] = __ldcg(reinterpret_cast<const float4*>(
            a.extra[1] + (static_cast<int64_t>(b + i) * a.T + row) * kColumns + column));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v.x += w[i].x, v.y += w[i].y, v.z += w[i].z, v.w += w[i].w;
  }
  return v;
}

__device__ __forceinline__ float swiglu(float g, float u) { return g / (1.f + expf(-g)) * u; }

// A tile's hidden values, from the partial sums of the blocks `first` to `last`.
template <typename T>
__device__ void hidden_tile(const Args& a, const Plan& plan, const Tile& t, int first, int last) {
  const bool shared = t.hit == plan.hits;
  const int f = shared ? a.fs : a.f;
#pragma unroll 2
  for (int i = threadIdx.x; i < t.rows * 64; i += blockDim.x) {
    const int n = i / 64, in = i % 64 * 4, column = t.at * 256 + in;
    if (column >= f) continue;
    const int row = t.first + n;
    const float* m = main_row(a, plan, 0, row, shared) + column;
    float4 g = __ldcg(reinterpret_cast<const float4*>(m));
    float4 w = __ldcg(reinterpret_cast<const float4*>(m + f));
    const float* e = a.extra[0] + (static_cast<int64_t>(first + 1) * a.T + n) * kColumns + in;
    const int64_t step = static_cast<int64_t>(a.T) * kColumns;
#pragma unroll 1
    for (int b = first + 1; b <= last; b += 4, e += 4 * step) {
      float4 v[4][2];
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          v[q][c] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (b + q <= last)
            v[q][c] = __ldcg(reinterpret_cast<const float4*>(e + q * step + c * 256));
        }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        g.x += v[q][0].x, g.y += v[q][0].y, g.z += v[q][0].z, g.w += v[q][0].w;
        w.x += v[q][1].x, w.y += v[q][1].y, w.z += v[q][1].z, w.w += v[q][1].w;
      }
    }
    const float o[4] = {swiglu(g.x, w.x), swiglu(g.y, w.y), swiglu(g.z, w.z), swiglu(g.w, w.w)};
    T* to = static_cast<T*>(a.hid) + hid_row(a, plan, row, shared) + column;
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(to) = make_float4(o[0], o[1], o[2], o[3]);
    } else {
      // the nearest bf16 number and that of what is left (none past the largest one)
      __nv_bfloat16 hi[4], lo[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        hi[q] = __float2bfloat16_rn(o[q]);
        const float r = o[q] - __bfloat162float(hi[q]);
        lo[q] = __float2bfloat16_rn(isfinite(r) ? r : 0.f);
      }
      memcpy(to, hi, 8);
      memcpy(to + a.hid_lo, lo, 8);
    }
  }
}

// A run of one of FC1's tiles is through: the last block to come forms the hidden values.
template <typename T>
__device__ void tile_done(const Args& a, Plan& plan, const Stream& s, int tile, const Tile& t) {
  int first, last;
  s.runs(tile, first, last);
  __syncthreads();
  if (threadIdx.x == 0) {
    int is_last = 1;
    if (last > first) {
      __threadfence();
      is_last = atomicAdd(a.tiles + tile, 1) == last - first;
      __threadfence();
    }
    plan.on = is_last;
  }
  __syncthreads();
  if (plan.on) {
    hidden_tile<T>(a, plan, t, first, last);
    __syncthreads();
    if (threadIdx.x == 0) {
      __threadfence();
      atomicAdd(a.ready + t.hit, 1);
    }
  }
}

// This block's units of a product.  false where a wait ran out.
template <typename T, bool QUEUE>
__device__ bool stream_product(const Args& a, Plan& plan, const Stream* streams, int product,
                               Copies<T, QUEUE>& copies, int& slot) {
  using F = Shape<T>;
  const Stream& s = streams[product];
  const int warp = threadIdx.x >> 5;
  int ready = -1, turn = 0, run = blockIdx.x;
  for (int u = s.begin, end = s.end;;) {
    if (u == end) {
      // this warp's copies are ahead, so the next piece is known
      if (!QUEUE || product == 0 || s.n1 + s.n2 == 0) break;
      const int p = *const_cast<volatile int*>(&plan.taken[turn++]);
      if (p < 0 || p >= s.n1 + s.n2) break;
      s.piece(p, u, end);
      run = s.n0 + p;
    }
    int tile, unit;
    s.find(u, tile, unit);
    const Tile t = tile_of(a, plan, s, tile);
    const bool shared = t.hit == plan.hits;
    const int f = shared ? a.fs : a.f, units = min(s.units_of(tile) - unit, end - u);
    if (product == 1 && ready != t.hit) {
      if (!expert_ready(a, plan, t.hit, shared ? streams[0].shared_tiles : streams[0].tiles))
        return false;
      ready = t.hit;
    }
    const int outputs = product ? a.h : f, inputs = product ? f : a.h;
    const int column = product ? t.at * kColumns + warp * F::kStrip
                               : t.at * 256 + warp % (F::kWarps / 2) * F::kStrip;
    Out out;
    out.limit = outputs - column;
    if (unit == 0) {
      out.at = main_row(a, plan, product, t.first, shared) + column +
               (product == 0 && warp >= F::kWarps / 2 ? f : 0);
      out.stride = product ? a.h : 2 * f;
    } else {
      out.at = a.extra[product] + static_cast<int64_t>(run) * a.T * kColumns + warp * F::kStrip;
      out.stride = kColumns;
    }
    const int k0 = unit * F::kInputs;
    // FC1 reads the rows' tokens, FC2 the hidden values in the rows' order
    const uint16_t* row_at = product ? nullptr : plan.token;
    const T* x = product ? static_cast<const T*>(a.hid) + hid_row(a, plan, t.first, shared)
                         : static_cast<const T*>(a.x);
    x += k0;
    constexpr int P2 = sizeof(T) == 2 ? 2 : 1;
    auto run = [&](auto nt, auto pieces) {
      run_units<T, QUEUE, decltype(nt)::value, decltype(pieces)::value>(
          copies, slot, units, x, a.hid_lo, row_at, t.first, t.rows, inputs, inputs - k0, out);
    };
    auto by_rows = [&](auto pieces) {
      if (t.rows <= 8) run(std::integral_constant<int, 1>(), pieces);
      else if (t.rows <= 16) run(std::integral_constant<int, 2>(), pieces);
      else if (t.rows <= 32) run(std::integral_constant<int, 4>(), pieces);
      else run(std::integral_constant<int, 8>(), pieces);
    };
    if (product == 0 || P2 == 1) by_rows(std::integral_constant<int, 1>());
    else by_rows(std::integral_constant<int, P2>());
    if (product == 0) tile_done<T>(a, plan, s, tile, t);
    u += units;
  }
  return true;
}

__device__ __forceinline__ void store4(float* p, float4 v) {
  *reinterpret_cast<float4*>(p) = v;
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  const __nv_bfloat162 q[2] = {__floats2bfloat162_rn(v.x, v.y), __floats2bfloat162_rn(v.z, v.w)};
  memcpy(p, q, 8);
}

template <typename T>
__device__ void combine(const Args& a, const Plan& plan, const Stream& s) {
  const int per = a.h / 4;
  for (int64_t i = blockIdx.x * blockDim.x + threadIdx.x; i < static_cast<int64_t>(a.T) * per;
       i += gridDim.x * blockDim.x) {
    const int t = static_cast<int>(i / per);
    const int column = static_cast<int>(i - static_cast<int64_t>(t) * per) * 4;
    const int at = column / kColumns;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int j = 0; j < a.k; ++j) {
      const int row = plan.row_of[t * a.k + j];
      if (row < 0) continue;
      const int hit = plan.hit_of_row[row];
      const float p = plan.prob[t * a.k + j];
      int first, last;
      s.runs(hit * s.tiles + at, first, last);
      const float4 v = sum_runs(a, main_row(a, plan, 1, row, false) + column, first, last,
                                row - plan.first[hit], column % kColumns);
      y.x = fmaf(p, v.x, y.x), y.y = fmaf(p, v.y, y.y);
      y.z = fmaf(p, v.z, y.z), y.w = fmaf(p, v.w, y.w);
    }
    if (a.fs) {
      int first, last;
      s.runs(s.routed + at, first, last);
      const float4 v = sum_runs(a, main_row(a, plan, 1, plan.rows + t, true) + column, first,
                                last, t, column % kColumns);
      y.x += v.x, y.y += v.y, y.z += v.z, y.w += v.w;
    }
    store4(static_cast<T*>(a.y) + static_cast<int64_t>(t) * a.h + column, y);
  }
}

template <typename T, bool QUEUE>
__global__ void __launch_bounds__(Shape<T>::kThreads, 1) few_kernel(const __grid_constant__ Args a) {
  extern __shared__ __align__(1024) char smem[];
  Plan& plan = *reinterpret_cast<Plan*>(smem + kRing);
  __shared__ Stream streams[2];
  // nobody counts in these before the barrier after the logits
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < a.counters; i += gridDim.x * blockDim.x)
    a.tiles[i] = 0;
  partial_logits<T>(a, smem);
  bool on = grid_barrier(a, plan, 1);
  const bool own = a.T == 1;
  if (on) {
    choose_experts(a, plan, own);
    if (!own) on = grid_barrier(a, plan, 2);
  }
  if (on) {
    make_plan(a, plan, own);
    if constexpr (QUEUE)
      for (int i = threadIdx.x; i < kLargePieces + kSmallPieces + 1; i += blockDim.x)
        plan.taken[i] = -1;
    if (threadIdx.x < 2) {
      constexpr int U = Shape<T>::kInputs;
      auto up = [](int n, int d) { return (n + d - 1) / d; };
      if (threadIdx.x == 0)
        streams[0].set(plan.hits, up(a.f, 256), up(a.h, U), up(a.fs, 256), up(a.h, U), false);
      else
        streams[1].set(plan.hits, up(a.h, kColumns), up(a.f, U), a.fs ? up(a.h, kColumns) : 0,
                       up(a.fs, U), QUEUE);
    }
    __syncthreads();
    Copies<T, QUEUE> copies(a, plan, streams, smem);
#pragma unroll 1
    for (int i = 0; i < kSlots - 1; ++i) copies.issue();
    int slot = 0;
    on = stream_product<T, QUEUE>(a, plan, streams, 0, copies, slot) &&
         stream_product<T, QUEUE>(a, plan, streams, 1, copies, slot);
    wait_copies<0>();
    on = on && grid_barrier(a, plan, own ? 2 : 3);
    if (on) combine<T>(a, plan, streams[1]);
  }
  leave(a);
}

size_t up256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

struct Layout {
  size_t logits, idx, prob, main[2], extra[2], counters, hid, total;
  int64_t hid_lo;
  int tiles, all;  // counters
  bool in_pieces;
};
Layout layout(int T, int h, int E, int k, int f, int fs, int dtype) {
  Layout L;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t r = o;
    o += up256(bytes);
    return r;
  };
  const size_t pairs = static_cast<size_t>(T) * k, rows = pairs + (fs ? T : 0);
  const size_t values = pairs * f + static_cast<size_t>(fs) * T;
  L.logits = take(static_cast<size_t>(slabs(kFewBlocks, E, h)) * T * E * 4);
  L.idx = take(pairs * 4);
  L.prob = take(pairs * 4);
  L.main[0] = take(2 * values * 4);
  L.main[1] = take(rows * h * 4);
  const int most = pairs < static_cast<size_t>(E) ? static_cast<int>(pairs) : E;  // experts hit
  const int64_t fc2_tiles = static_cast<int64_t>(most + (fs > 0)) * ((h + kColumns - 1) / kColumns);
  L.in_pieces = dtype == MOE_BF16 && fc2_tiles >= kInPieces * kFewBlocks;
  for (int i = 0; i < 2; ++i) {
    const int runs = kFewBlocks + (i && L.in_pieces ? kLargePieces + kSmallPieces : 0);
    L.extra[i] = take(static_cast<size_t>(runs) * T * kColumns * 4);
  }
  L.tiles = most * ((f + 255) / 256) + (fs + 255) / 256;
  L.all = L.tiles + most + 1 + 1;  // the shared expert's, the queue's
  L.counters = take(static_cast<size_t>(L.all) * 4);
  L.hid_lo = static_cast<int64_t>(up256(values * 2) / 2);
  L.hid = take(dtype == MOE_F32 ? values * 4 : static_cast<size_t>(L.hid_lo) * 2 * 2);
  L.total = o;
  return L;
}

template <typename T, bool QUEUE>
cudaError_t launch(Args& a, cudaStream_t s) {
  cudaError_t st = allow_most_smem<few_kernel<T, QUEUE>>();
  if (st != cudaSuccess) return st;
  cudaLaunchConfig_t cfg = {};
  const int sms = device_sm_count();
  cfg.gridDim = dim3(sms < kFewBlocks ? sms : kFewBlocks);
  cfg.blockDim = dim3(Shape<T>::kThreads);
  cfg.dynamicSmemBytes = kRing + sizeof(Plan);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, few_kernel<T, QUEUE>, static_cast<const Args>(a));
}

}  // namespace

size_t few_scratch(const moe_config& c, int fs) {
  return layout(c.num_tokens, c.hidden, c.num_experts, c.topk, c.ffn_hidden, fs, c.dtype).total;
}

cudaError_t launch_few(const moe_config& c, int fs, int64_t capacity, const void* x,
                       const float* Wg, const float* gate_bias, const float* expert_bias,
                       const void* W1, const void* W3, const void* W2, const void* W1s,
                       const void* W3s, const void* W2s, void* y, int32_t* topk_idx,
                       float* topk_prob, int32_t* tokens_per_expert, void* scratch, int* err,
                       cudaStream_t s) {
  const Layout L = layout(c.num_tokens, c.hidden, c.num_experts, c.topk, c.ffn_hidden, fs, c.dtype);
  char* at = static_cast<char*>(scratch);
  Args a;
  a.T = c.num_tokens, a.h = c.hidden, a.E = c.num_experts, a.k = c.topk, a.f = c.ffn_hidden;
  a.fs = fs;
  a.score = c.score, a.groups = c.num_groups, a.group_topk = c.group_topk;
  a.capacity = capacity < 0 || capacity >= c.num_tokens ? -1 : static_cast<int>(capacity);
  a.policy = c.drop_policy;
  a.x = x, a.W1 = W1, a.W3 = W3, a.W2 = W2, a.V1 = W1s, a.V3 = W3s, a.V2 = W2s;
  a.Wg = Wg, a.gate_bias = gate_bias, a.expert_bias = expert_bias;
  a.y = y, a.idx_out = topk_idx, a.prob_out = topk_prob, a.tpe_out = tokens_per_expert;
  a.err = err;
  a.bar = err + kFewCounters;
  a.logits = reinterpret_cast<float*>(at + L.logits);
  a.idx = reinterpret_cast<int32_t*>(at + L.idx);
  a.prob = reinterpret_cast<float*>(at + L.prob);
  for (int i = 0; i < 2; ++i) {
    a.main[i] = reinterpret_cast<float*>(at + L.main[i]);
    a.extra[i] = reinterpret_cast<float*>(at + L.extra[i]);
  }
  a.tiles = reinterpret_cast<int*>(at + L.counters);
  a.ready = a.tiles + L.tiles;
  a.queue = a.tiles + L.all - 1;
  a.counters = L.all;
  a.hid = at + L.hid;
  a.hid_lo = L.hid_lo;
  if (c.dtype == MOE_F32) return launch<float, false>(a, s);
  return L.in_pieces ? launch<__nv_bfloat16, true>(a, s) : launch<__nv_bfloat16, false>(a, s);
}

}  // namespace moe
