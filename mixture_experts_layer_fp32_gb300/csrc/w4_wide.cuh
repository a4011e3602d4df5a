// Products with 4-bit weights for more rows: chunks of up to 64 columns (64 rows
// of x; FC2: 32, two columns each) on tcgen05.
//
// A block, one to an SM, takes 256 outputs of a chunk at a time (FC1: 128 gate
// rows and the 128 up rows of the same features) as two tiles of 128.  For each
// 128 inputs
//   - TMA brings the tiles' codes (two blocks of inputs in a copy) and x;
//   - four warps a tile turn a row's 64 bytes of codes, a row to a thread, into
//     fp16 differences q - zero in the tensor memory, the A operand, as the narrow
//     kernel does in registers.  Two slots, with warps of their own each: one set of
//     warps took 237 us where two take 215 (below);
//   - one thread multiplies, a fresh sum for each group of inputs;
//   - eight warps, an output of both tiles to a thread and half the columns each,
//     read the groups' sums back and add them up under their scales in fp32.
// All of them run at once and hand each other slots through mbarriers.  A warp whose
// wait runs out reports it, and then every warp leaves its loop; the block's copies
// and products end (again within a limit) before its tensor memory is freed.
//
// Measured, the experts of 64 tokens (2 of 8 of 4096 x 14336, zero points): 194 us
// with the splits and the combine; FC1 117 and FC2 78 us cold.  mma.sync from
// registers took 453 us: every warp read the whole x for its 32 outputs, and the
// conversion, the products and the scaling waited for one another within a warp.
// What is used most now is the issue slots: 740 instructions of an SM quarter for
// 16 KB of codes, 62% of its slots, half of them masks and subtractions; the
// products alone, whose A operand of 4 KB takes some 33 cycles to read whatever the
// number of columns, would take 530 of the 1190 cycles.
//
// Tried and left: the next item's scales and zeros loaded ahead (211 us where the
// kernel took 206), two multiply-adds in an instruction (209), those lines brought
// into L2 ahead (203 where it took 198).
#pragma once

#include <type_traits>

namespace moe {
namespace w4 {

constexpr int kTallRoles = 28;             // warps: 8 add up, 16 convert, codes, x, products, none
constexpr int kTallColumns = 64;           // most columns of a chunk
constexpr int kTallStages = 4;             // of codes: 2 blocks of inputs of 2 tiles
constexpr int kTallStage = 2 * 2 * 128 * 64;
constexpr int kTallXs = 4;                 // of x: a block of inputs
constexpr int kTallX = kTallColumns * 256;
constexpr int kTallSmem = kTallStages * kTallStage + kTallXs * kTallX + 1024;

struct TallBars {
  uint64_t code_full[kTallStages], code_free[kTallStages];
  uint64_t x_full[kTallXs], x_free[kTallXs];
  uint64_t a_full[2], a_free[2];  // of both tiles
  uint64_t d_full[4], d_free[4];
  uint64_t products;  // all of them
};

// Waits of a converged warp.
struct Waits {
  int* err;
  volatile int* given_up;  // the block's

  // false, for the whole warp, where this wait or another warp's ran out
  __device__ __forceinline__ bool operator()(uint32_t bar, int parity) const {
    if (__all_sync(~0u, ptx::mbar_try_wait(bar, parity))) return true;
    const long long began = clock64();
    do {
      if (__any_sync(~0u, *given_up != 0 || clock64() - began > kWaitCycles)) {
        *given_up = 1;
        report_error(err, DEV_ERR_TIMEOUT, static_cast<int>(blockIdx.x));
        return false;
      }
    } while (!__all_sync(~0u, ptx::mbar_try_wait(bar, parity)));
    return true;
  }
  // what is in flight, given up or not
  __device__ __forceinline__ void end(uint32_t bar, int parity) const {
    if (!__all_sync(~0u, arrives(bar, parity))) {
      *given_up = 1;
      report_error(err, DEV_ERR_TIMEOUT, static_cast<int>(blockIdx.x));
    }
  }
};

// A slot of a ring and the parity of its barriers' phase.
struct Ring {
  int slots, at = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if (++at == slots) {
      at = 0;
      phase ^= 1;
    }
  }
  // the parity of a slot's last use (a barrier that was never used counts as past 1)
  __device__ __forceinline__ int last(int slot) const { return slot < at ? phase : phase ^ 1; }
};

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]),
                 "=f"(r[6]), "=f"(r[7])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
        "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]),
        "=f"(r[14]), "=f"(r[15])
      : "r"(taddr)
      : "memory");
}
// D[tmem] (+)= A[tmem] B[smem], fp16 operands, by one thread
__device__ __forceinline__ void umma_f16_ta(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Four neighbouring groups' scales (bf16) and zeros of a row, `left` the groups
// from there to the row's end; past it 0.  `whole`: rows of a multiple of 4 groups.
__device__ __forceinline__ uint2 four_scales(const unsigned short* p, int left, bool whole) {
  if (whole) return left > 0 ? __ldg(reinterpret_cast<const uint2*>(p)) : make_uint2(0u, 0u);
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = i < left ? __ldg(p + i) : 0u;
  return make_uint2(v[0] | v[1] << 16, v[2] | v[3] << 16);
}
__device__ __forceinline__ uint32_t four_zeros(const uint8_t* p, int left, bool whole) {
  if (whole) return left > 0 ? __ldg(reinterpret_cast<const uint32_t*>(p)) : 0u;
  uint32_t v = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) v |= (i < left ? static_cast<uint32_t>(__ldg(p + i)) : 0u) << 8 * i;
  return v;
}

// This warpgroup's registers to a thread.
template <int N, bool MORE>
__device__ __forceinline__ void registers() {
  if (MORE) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// One thread of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

template <int MODE, int G32>
__global__ void __launch_bounds__(kTallRoles * 32, 1)
    w4_wide_kernel(const __grid_constant__ CUtensorMap map0,
                   const __grid_constant__ CUtensorMap map1,
                   const __grid_constant__ CUtensorMap map_x, Args a) {
  constexpr int GPB = 4 / G32;
  constexpr int CP = pieces_of(MODE);
  constexpr int kTile = MODE == FC1 ? 128 : 256;  // outputs of an item
  constexpr int SB = 4;                           // blocks of a unit of a part
  extern __shared__ uint8_t smem_raw[];
  __shared__ TallBars bars;
  __shared__ float units[8][32];
  __shared__ uint32_t tmem_at;
  __shared__ int given_up;
  const uint32_t base = (ptx::smem_u32(smem_raw) + 1023) & ~1023u;
  const uint32_t xs_at = base + kTallStages * kTallStage;
  Plan& plan = *reinterpret_cast<Plan*>(smem_raw + kTallSmem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto bar = [](const uint64_t& b) { return ptx::smem_u32(&b); };
  pdl_trigger();

  if (threadIdx.x == 0) {
    for (int i = 0; i < kTallStages; ++i) {
      ptx::mbar_init(bar(bars.code_full[i]), 1);
      ptx::mbar_init(bar(bars.code_free[i]), 16);
    }
    for (int i = 0; i < kTallXs; ++i) {
      ptx::mbar_init(bar(bars.x_full[i]), 1);
      ptx::mbar_init(bar(bars.x_free[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bar(bars.a_full[i]), 8);
      ptx::mbar_init(bar(bars.a_free[i]), 1);
    }
    for (int i = 0; i < 4; ++i) {
      ptx::mbar_init(bar(bars.d_full[i]), 1);
      ptx::mbar_init(bar(bars.d_free[i]), 8);
    }
    ptx::mbar_init(bar(bars.products), 1);
    given_up = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 26) {
    ptx::tmem_alloc(ptx::smem_u32(&tmem_at), 512);
    ptx::tmem_relinquish();
  }
  int chunks;
  if (MODE == LINEAR) {
    chunks = (a.rows + a.chunk_rows - 1) / a.chunk_rows;
  } else {
    make_plan(plan, a, a.chunk_rows);
    chunks = plan.chunks;
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = tmem_at;
  // A: 64 columns of a block's 128 inputs, [tile][slot]; D: 64 columns or, if no
  // chunk has more than 32, 32, [tile][slot]
  const int d_columns = a.chunk_rows * CP, d_slots = 128 / d_columns;
  auto a_at = [&](int d, int slot) { return tmem + d * 128 + slot * 64; };
  auto d_at = [&](int d, int slot) { return tmem + 256 + d * 128 + slot * d_columns; };

  // Registers: 896 threads are launched with 72 each; 256 with 112 and 640
  // with 56 come to the same.
  const Waits wait{a.err, &given_up};
  Item it(blockIdx.x, a);
  // of the item: its first block of inputs, how many, its rows of x
  int kb = 0, nb = 0, row_first = 0, row_count = 0;
  uint32_t row = 0;  // of its weights
  auto enter = [&]() {
    if (it.chunk >= chunks) return false;
    const int first = it.part * a.split_units + min(it.part, a.split_rest);
    const int units = a.split_units + (it.part < a.split_rest);
    kb = first * SB;
    nb = min(units * SB, a.blocks - kb);
    uint32_t e = 0;
    if (MODE == LINEAR) {
      row_first = it.chunk * a.chunk_rows;
      row_count = min(a.chunk_rows, a.rows - row_first);
    } else {
      e = plan.chunk_expert[it.chunk];
      row_first = plan.chunk_row[it.chunk];
      row_count = min(a.chunk_rows, plan.end[e] - row_first);
    }
    row = e * a.N + static_cast<uint32_t>(it.tile) * kTile;
    return true;
  };

  if (warp < 8) {
    registers<112, true>();
    // ---- sums: an output of each tile, half of the columns ----
    const int e = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // << 16, by 32
    const bool whole = a.groups % 4 == 0;
    pdl_wait();  // the rows' units; and the output is free
    Ring ring{d_slots};
    bool on = true;
    for (; on && enter(); it.next(gridDim.x, a)) {
      const int o[2] = {it.tile * kTile + r, it.tile * kTile + (MODE == FC1 ? 0 : 128) + r};
      const unsigned short* ps[2];
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        const W4& w = MODE == FC1 && d ? a.w1 : a.w0;
        ps[d] = reinterpret_cast<const unsigned short*>(w.scales) +
                static_cast<uint64_t>(row - it.tile * kTile + min(o[d], a.N - 1)) * a.groups +
                kb * GPB;
      }
      const int n = nb * GPB, left = a.groups - kb * GPB;
      // with half of the columns known, what is read of a group is fixed
      auto item = [&](auto known) {
        constexpr int half = decltype(known)::value;
        constexpr int R = half / CP;  // rows of x
        uint2 now[2], next[2];
#pragma unroll
        for (int d = 0; d < 2; ++d) next[d] = four_scales(ps[d], left, whole);
        // the rows' units, read at the end
        if (lane < R && e * R + lane < row_count)
          copy_async4(ptx::smem_u32(&units[warp][lane]), a.unit + row_first + e * R + lane);
        copies_commit();
        float acc[2][R];
#pragma unroll
        for (int i = 0; i < R; ++i) acc[0][i] = acc[1][i] = 0.f;
#pragma unroll 1
        for (int g = 0; g < n; ++g) {
          if ((g & 3) == 0) {
#pragma unroll
            for (int d = 0; d < 2; ++d) {
              now[d] = next[d];
              next[d] = four_scales(ps[d] + g + 4, left - g - 4, whole);
            }
          }
          float s[2];
#pragma unroll
          for (int d = 0; d < 2; ++d) {
            s[d] = __uint_as_float(now[d].x << 16);
            now[d].x = __funnelshift_r(now[d].x, now[d].y, 16);
            now[d].y >>= 16;
          }
          if (!wait(bar(bars.d_full[ring.at]), ring.phase)) {
            copies_wait<0>();
            return false;
          }
          ptx::tc_fence_after();
          const uint32_t at = d_at(0, ring.at) + lanes + e * half;
          // a few columns of both tiles at a time, as the registers allow
          constexpr int some = half <= 16 ? half : 8;
#pragma unroll
          for (int c = 0; c < half; c += some) {
            float v[2][some];
#pragma unroll
            for (int d = 0; d < 2; ++d) {
              if (some == 8) tmem_ld8(at + d * 128 + c, v[d]);
              else tmem_ld16(at + d * 128 + c, v[d]);
            }
            ptx::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < some; ++i)
              asm volatile("" : "+f"(v[0][i]), "+f"(v[1][i]));
            if (c + some == half) {  // the last of them
              ptx::tc_fence_before();
              __syncwarp();
              if (lane == 0) ptx::mbar_arrive(bar(bars.d_free[ring.at]));
            }
#pragma unroll
            for (int i = 0; i < some; i += CP)
#pragma unroll
              for (int d = 0; d < 2; ++d) {
                // FC2: the second piece is in 2^-11 of the first's unit
                const float sum =
                    CP == 2 ? v[d][i] + 0.00048828125f * v[d][i + CP - 1] : v[d][i];
                acc[d][(c + i) / CP] += s[d] * sum;
              }
          }
          ring.next();
        }
        // Rows past the last one are worked out too and not stored: no branch stands
        // between one and the next.
        copies_wait<0>();
        __syncwarp();
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const float unit = units[warp][i];
          acc[0][i] *= unit;
          acc[1][i] *= unit;
          if (MODE == FC1) acc[0][i] = acc[0][i] / (1.f + expf(-acc[0][i])) * acc[1][i];
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const int rx = e * R + i;
          if (rx >= row_count) break;
          if (MODE == FC1) {
            if (o[0] < a.N)
              static_cast<float*>(a.out)[static_cast<int64_t>(row_first + rx) * a.N + o[0]] =
                  acc[0][i];
            continue;
          }
          const int64_t at =
              MODE == FC2 ? static_cast<int64_t>(it.part) * a.pairs + plan.pair[row_first + rx]
                          : static_cast<int64_t>(it.part) * a.rows + row_first + rx;
          if (MODE == FC2 || a.out_f32) {
            float* out = static_cast<float*>(a.out) + at * a.N;
            if (o[0] < a.N) out[o[0]] = acc[0][i];
            if (o[1] < a.N) out[o[1]] = acc[1][i];
          } else {
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + at * a.N;
            if (o[0] < a.N) out[o[0]] = __float2bfloat16_rn(acc[0][i]);
            if (o[1] < a.N) out[o[1]] = __float2bfloat16_rn(acc[1][i]);
          }
        }
        return true;
      };
      switch ((row_count * CP + 15) / 16) {
        case 1: on = item(std::integral_constant<int, 8>()); break;
        case 2: on = item(std::integral_constant<int, 16>()); break;
        case 3: on = item(std::integral_constant<int, 24>()); break;
        default: on = item(std::integral_constant<int, 32>());
      }
    }
  } else if (warp < 24) {
    registers<56, false>();
    // ---- codes: a row to a thread; a slot of A and a tile to four warps ----
    const int d = (warp >> 2) & 1, slot = (warp - 8) >> 3, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
    const bool whole = a.groups % 4 == 0;
    const W4& w = MODE == FC1 && d ? a.w1 : a.w0;
    // the copy's 16-byte pieces are swapped by bits 7 and 8 of their place
    const uint32_t src = base + d * (kTallStage / 2) + r * 64;
    const uint32_t swap = ((r >> 1) & 3) << 4;
    const uint32_t a_slot = a_at(d, slot) + lanes;
    const uint32_t held = held_1024();
    Ring code{kTallStages};
    int turn = 0, phase = 0;  // the slot of the block to come; this slot's phase
    bool on = true;
    for (; on && enter(); it.next(gridDim.x, a)) {
      const int o = it.tile * kTile + (MODE == FC1 ? 0 : d * 128) + r;
      const int left = a.groups - kb * GPB;
      const uint8_t* pz = nullptr;
      // zeros of four groups, one block of this slot's ahead
      uint32_t z_next = 0x08080808u;
      const int mine = (slot - turn) & 1;  // this slot's blocks: mine, mine + 2, ..
      if (w.zeros != nullptr) {
        pz = w.zeros +
             static_cast<uint64_t>(row - it.tile * kTile + min(o, a.N - 1)) * a.groups + kb * GPB;
        const int g = mine * GPB & ~3;
        z_next = four_zeros(pz + g, left - g, whole);
      }
#pragma unroll 1
      for (int b = mine; b < nb + mine; b += 2) {
        on = wait(bar(bars.code_full[code.at]), code.phase);
        if (!on) break;
        if (b < nb) {
          uint4 q[4];
#pragma unroll
          for (int c = 0; c < 4; ++c)
            q[c] = lds16(src + code.at * kTallStage + mine * 8192 + ((c << 4) ^ swap));
          uint32_t z = z_next >> (8 * (b * GPB & 3));
          if (pz != nullptr) {
            const int g = (b + 2) * GPB & ~3;
            z_next = four_zeros(pz + g, left - g, whole);
          }
          on = wait(bar(bars.a_free[slot]), phase ^ 1);
          if (!on) break;
          ptx::tc_fence_after();
#pragma unroll
          for (int j = 0; j < 4; ++j) {  // inputs 32 j ..
            const ZeroPair zero = zero_pair((z >> (8 * (j / G32))) & 15u);
            uint32_t v[16];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t p[4];
              pairs_of(j == 0 ? q[c].x : j == 1 ? q[c].y : j == 2 ? q[c].z : q[c].w, held, zero, p);
#pragma unroll
              for (int i = 0; i < 4; ++i) v[c * 4 + i] = p[i];
            }
            tmem_st16(a_slot + j * 16, v);
          }
          tmem_wait_st();
          ptx::tc_fence_before();
          phase ^= 1;
        }
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive(bar(bars.code_free[code.at]));
          if (b < nb) ptx::mbar_arrive(bar(bars.a_full[slot]));
        }
        code.next();
      }
      turn ^= nb & 1;
    }
  } else {
    registers<56, false>();
    if (warp == 24) {
      // ---- the codes' copies ----
      Ring code{kTallStages};
      bool on = true;
      for (; on && enter(); it.next(gridDim.x, a)) {
        const bool second = MODE == FC1 || it.tile * kTile + 128 < a.N;
        for (int b = 0; b < nb; b += 2) {
          on = wait(bar(bars.code_free[code.at]), code.phase ^ 1);
          if (!on) break;
          if (lane == 0) {
            const uint32_t dst = base + code.at * kTallStage, full = bar(bars.code_full[code.at]);
            ptx::mbar_arrive_expect_tx(full, second ? kTallStage : kTallStage / 2);
            // blocks past the row's end come as zeros
            ptx::tma_load_3d(dst, &map0, 0, static_cast<int>(row), kb + b, full);
            if (second)
              ptx::tma_load_3d(dst + kTallStage / 2, MODE == FC1 ? &map1 : &map0, 0,
                               static_cast<int>(row) + (MODE == FC1 ? 0 : 128), kb + b, full);
          }
          __syncwarp();
          code.next();
        }
      }
      for (int i = 0; i < kTallStages; ++i) wait.end(bar(bars.code_full[i]), code.last(i));
    } else if (warp == 25) {
      // ---- the copies of x: 8 columns of a block's inputs each ----
      pdl_wait();
      Ring ring{kTallXs};
      bool on = true;
      for (; on && enter(); it.next(gridDim.x, a)) {
        const int copies = (row_count * CP + 7) / 8;
        for (int b = 0; b < nb; ++b) {
          const uint32_t full = bar(bars.x_full[ring.at]);
          on = wait(bar(bars.x_free[ring.at]), ring.phase ^ 1);
          if (!on) break;
          if (lane == 0) ptx::mbar_arrive_expect_tx(full, copies * 2048);
          __syncwarp();
          if (lane < copies)
            ptx::tma_load_3d(xs_at + ring.at * kTallX + lane * 2048, &map_x, 0,
                             row_first * CP + lane * 8, (kb + b) * 2, full);
          ring.next();
        }
      }
      for (int i = 0; i < kTallXs; ++i) wait.end(bar(bars.x_full[i]), ring.last(i));
    } else if (warp == 26) {
      // ---- products: the warp keeps together, so that addresses stay in uniform
      // registers, and one thread of it issues ----
      const bool issues = elect_one();
      Ring ring{kTallXs};
      Ring as{2}, ds{d_slots};  // of A and D, both tiles' together
      bool on = true;
      for (; on && enter(); it.next(gridDim.x, a)) {
        const uint32_t columns = (row_count * CP + 15) / 16 * 16;
        const uint32_t idesc = (1u << 4) | (columns >> 3) << 17 | (128u >> 4) << 24;
#pragma unroll 1
        for (int b = 0; on && b < nb; ++b) {
          on = wait(bar(bars.x_full[ring.at]), ring.phase) &&
               wait(bar(bars.a_full[as.at]), as.phase);
          if (!on) break;
          // a step of 16 inputs is 32 bytes on, 64 inputs 1024
          const uint64_t x = ptx::sw128_desc(xs_at + ring.at * kTallX, 0, 2048);
#pragma unroll
          for (int q = 0; q < GPB; ++q) {
            on = wait(bar(bars.d_free[ds.at]), ds.phase ^ 1);
            if (!on) break;
            ptx::tc_fence_after();
            if (issues) {
#pragma unroll
              for (int d = 0; d < 2; ++d)
#pragma unroll
                for (int k = q * G32 * 2; k < (q + 1) * G32 * 2; ++k)
                  umma_f16_ta(d_at(d, ds.at), a_at(d, as.at) + k * 8,
                              x + ((k >> 2) * 64 + (k & 3) * 2), idesc, k > q * G32 * 2);
              ptx::umma_commit(bar(bars.d_full[ds.at]));
            }
            __syncwarp();
            ds.next();
          }
          if (issues) {
            ptx::umma_commit(bar(bars.a_free[as.at]));
            ptx::umma_commit(bar(bars.x_free[ring.at]));
          }
          __syncwarp();
          as.next();
          ring.next();
        }
      }
      if (issues) ptx::umma_commit(bar(bars.products));
      __syncwarp();
      wait.end(bar(bars.products), 0);
    }
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 26) ptx::tmem_dealloc(tmem, 512);
}

}  // namespace w4
}  // namespace moe
