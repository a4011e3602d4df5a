// 8-bit integer products for more rows: tcgen05 on whole numbers in fp16.
//
// This chip's integer tensor-core instruction runs at 150 TOP/s (measured), fp16 at
// 1.9 PFLOP/s: so the codes become fp16 numbers, which hold them exactly.  x is laid
// out as fp16 by the launch before (it is the smaller operand); W stays in 8 bits until
// it is on the SM, where warps turn it into the A operand in the tensor memory (a byte
// under a mask with 0x64 before it is the fp16 number 1024 + 128 + code; a subtraction
// takes the 1152 off).  A product is 2^14 at most, so fp32 sums of 1024 of them are whole
// numbers up to 2^24, exact; then they are read out and added up as integers.
//
// A block, one to an SM, takes 256 outputs (two tiles of 128, which share x) of NC rows
// of x at a time, with roles for its warps that hand each other slots through
// mbarriers:
//   8 add up: an output of both tiles to a thread and half of the columns each;
//   8 convert: an output of a tile to a thread, 128 inputs at a time;
//   one copies W (TMA), one x (TMA), a thread of one more each multiplies a tile.
// The two tiles' sums are read out 4 blocks of 128 inputs apart, and three places for
// sums serve the two: a tile goes on in the spare one while its last is read.  8192 x
// 14336 x 4096 (codes, bf16 results), step by step: 837 us with two places and a warp for
// all products, 805 with three places, 712 with a warp for each tile's products (one
// could not issue them as fast as they run), 653 with an epilogue without branches between
// the rows (a tile's first sums wait for the eight warps that store the last item's).
//
// What bounds it: shared memory (x is read for each tile: 160 KB for 256 x 128 x 128
// products, 1250 cycles where these take 1024) beside the reading of sums; with sums read
// once an item, or codes not converted, the 712 were 623 and 670.  The kernel of 128 columns
// spills besides (128 sums and 16 loads in a thread's 152 registers: 592 bytes of stores,
// 236 where parts of sums are stored; none with 64 and 32 columns).  Few rows: memory (64 x
// 151936 x 4096: 110 us, 5.9 TB/s).  Tried and left: pairs of blocks that share a product
// (256 outputs a tile, half of x in each): 1280 us, whatever the number of slots.
#include <type_traits>

#include "i8.cuh"
#include "roles.cuh"

namespace moe {
namespace i8 {
namespace {

using namespace roles;

constexpr int kWarpsWide = 20;
constexpr int kWStage = 2 * 128 * 128;       // of W: 128 inputs of both tiles
constexpr int kExact = 8;                    // blocks of 128 inputs whose sums are exact
template <int NC>
struct Wide {
  static constexpr int kWStages = NC == 128 ? 4 : 5;
  static constexpr int kXStages = NC == 128 ? 3 : 4;
  static constexpr int kXStage = NC * 256;
  static constexpr int kASlots = NC == 128 ? 2 : 4;  // of A, each tile's: 64 inputs
  static constexpr int kSmem = kWStages * kWStage + kXStages * kXStage + 1024;
};

struct Items {
  int tiles, chunks, splits, blocks;  // blocks of 128 inputs
  int total;
};

struct Bars {
  uint64_t w_full[5], w_free[5];
  uint64_t x_full[4], x_free[4];
  uint64_t a_full[2][4], a_free[2][4];  // [tile][slot]
  uint64_t d_full[3], d_free[3];        // places of sums
  uint64_t products;
};

// One item: 256 outputs, NC rows, a part of the inputs.  Sixteen tiles of W go with all
// chunks of x before the next sixteen: what runs at a time then reads few of either.
constexpr int kRaster = 16;
struct Item {
  int tile, chunk, part, first, count;  // count: blocks of inputs
  __device__ __forceinline__ Item(int i, const Items& s) {
    part = i % s.splits;
    i /= s.splits;
    const int group = i / (kRaster * s.chunks), in = i - group * kRaster * s.chunks;
    const int width = min(kRaster, s.tiles - group * kRaster);
    chunk = in / width;
    tile = group * kRaster + in - chunk * width;
    first = static_cast<int>(static_cast<int64_t>(s.blocks) * part / s.splits);
    count = static_cast<int>(static_cast<int64_t>(s.blocks) * (part + 1) / s.splits) - first;
  }
};
// whether tile d's sums are read out after block b of an item
__device__ __forceinline__ bool read_after(int d, int b, int count) {
  return b + 1 == count || (b + 1) % kExact == d * (kExact / 2);
}

// Which of the three places for sums is whose, and the parity of each one's use; the
// same for the warp that multiplies and those that read.
struct Places {
  int of[2] = {0, 1}, spare = 2;
  uint32_t phase = 0;  // a bit each
  __device__ __forceinline__ int parity(int d) const { return phase >> of[d] & 1; }
  // tile d goes on in the spare place
  __device__ __forceinline__ void next(int d) {
    phase ^= 1u << of[d];
    const int was = of[d];
    of[d] = spare;
    spare = was;
  }
};

// Four codes to two pairs of fp16 numbers.
__device__ __forceinline__ void pairs_of(uint32_t word, uint32_t& p, uint32_t& q) {
  const uint32_t v = word ^ 0x80808080u;  // code + 128
  const uint32_t lo = __byte_perm(v, 0x64646464u, 0x4140), hi = __byte_perm(v, 0x64646464u, 0x4342);
  const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
  __half2 a, b;
  memcpy(&a, &lo, 4);
  memcpy(&b, &hi, 4);
  a = __hsub2(a, off), b = __hsub2(b, off);
  memcpy(&p, &a, 4);
  memcpy(&q, &b, 4);
}
__device__ __forceinline__ uint4 lds16(uint32_t at) {
  uint4 q;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
               : "r"(at)
               : "memory");
  return q;
}

__device__ __forceinline__ void store(float* p, float v) { *p = v; }
__device__ __forceinline__ void store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Out: what is stored, the type of y or whole numbers (parts of a sum)
template <int NC, typename Out>
__global__ void __launch_bounds__(kWarpsWide * 32, 1)
    wide_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                const __grid_constant__ Args a, const __grid_constant__ Items items) {
  using W = Wide<NC>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Bars bars;
  __shared__ uint32_t tmem_at;
  __shared__ int given_up;
  const uint32_t base = (ptx::smem_u32(smem_raw) + 1023) & ~1023u;
  const uint32_t xs_at = base + W::kWStages * kWStage;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto bar = [](const uint64_t& b) { return ptx::smem_u32(&b); };
  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int i = 0; i < W::kWStages; ++i) {
      ptx::mbar_init(bar(bars.w_full[i]), 1);
      ptx::mbar_init(bar(bars.w_free[i]), 8);
    }
    for (int i = 0; i < W::kXStages; ++i) {
      ptx::mbar_init(bar(bars.x_full[i]), 1);
      ptx::mbar_init(bar(bars.x_free[i]), 2);
    }
    for (int d = 0; d < 2; ++d)
      for (int i = 0; i < W::kASlots; ++i) {
        ptx::mbar_init(bar(bars.a_full[d][i]), 4);
        ptx::mbar_init(bar(bars.a_free[d][i]), 1);
      }
    for (int i = 0; i < 3; ++i) {
      ptx::mbar_init(bar(bars.d_full[i]), 1);
      ptx::mbar_init(bar(bars.d_free[i]), 8);
    }
    ptx::mbar_init(bar(bars.products), 2);
    given_up = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 18) {
    ptx::tmem_alloc(ptx::smem_u32(&tmem_at), 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = tmem_at;
  // A: 32 columns of 64 inputs, [tile][slot]; sums: three places
  auto a_at = [&](int d, int slot) { return tmem + (d * W::kASlots + slot) * 32; };
  auto d_at = [&](int place) { return tmem + 2 * W::kASlots * 32 + place * NC; };
  const Waits wait{a.err, &given_up};
  const int step = gridDim.x;

  // 640 threads are launched with 96 registers each; 256 with 152 and 384 with 56 are
  // less than those.
  if (warp < 8) {
    registers<152, true>();
    // ---- sums ----
    constexpr int half = NC / 2;
    const int e = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // << 16, by 32
    pdl_wait();  // the rows' scales; and the output is free
    Places places;
    bool on = true;
    for (int i = blockIdx.x; on && i < items.total; i += step) {
      const Item it(i, items);
      int acc[2][half];
#pragma unroll
      for (int c = 0; c < half; ++c) acc[0][c] = acc[1][c] = 0;
#pragma unroll 1
      for (int b = 0; on && b < it.count; ++b)
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          if (!on || !read_after(d, b, it.count)) continue;
          on = wait(bar(bars.d_full[places.of[d]]), places.parity(d));
          if (!on) break;
          ptx::tc_fence_after();
          const uint32_t at = d_at(places.of[d]) + lanes + e * half;
#pragma unroll
          for (int c = 0; c < half; c += 16) {
            float v[16];
            tmem_ld16(at + c, v);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int q = 0; q < 16; ++q) asm volatile("" : "+f"(v[q]));
            if (c + 16 == half) {
              ptx::tc_fence_before();
              __syncwarp();
              if (lane == 0) ptx::mbar_arrive(bar(bars.d_free[places.of[d]]));
            }
#pragma unroll
            for (int q = 0; q < 16; ++q) acc[d][c + q] += __float2int_rn(v[q]);
          }
          places.next(d);
        }
      if (!on) break;
      // No branch stands between one row and the next, so that loads and stores run on; the
      // next item's first sums are ready for reading 4 blocks of inputs from now.
      const int row0 = it.chunk * NC + e * half;
      const int rows = min(half, a.rows - row0);
      float row_scale[(half + 31) / 32];  // of the rows lane, lane + 32
#pragma unroll
      for (int i = 0; i < (half + 31) / 32; ++i) {
        const int c = i * 32 + lane;
        row_scale[i] = c < rows ? a.x_scale[row0 + c] : 0.f;
      }
      const int64_t first = static_cast<int64_t>(row0) * a.N;
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        const int o = it.tile * 256 + d * 128 + r, at = min(o, a.N - 1);
        const float scale = a.w_scale[at], bias = a.bias ? a.bias[at] : 0.f;
        const int there = o < a.N ? rows : 0;
        Out* p = (std::is_same<Out, int32_t>::value
                      ? reinterpret_cast<Out*>(a.part) + static_cast<int64_t>(it.part) * a.rows * a.N
                      : static_cast<Out*>(a.y)) + first + o;
#pragma unroll
        for (int c = 0; c < half; ++c, p += a.N) {
          if constexpr (std::is_same<Out, int32_t>::value) {
            if (c < there) *p = acc[d][c];
          } else {
            const float v =
                scaled(acc[d][c], __shfl_sync(~0u, row_scale[c / 32], c % 32), scale, bias);
            if (c < there) store(p, v);
          }
        }
      }
    }
  } else if (warp < 16) {
    registers<56, false>();
    // ---- codes ----
    const int d = (warp >> 2) & 1, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
    const uint32_t src = base + d * (kWStage / 2) + r * 128, swap = (r & 7) << 4;
    Ring ws{W::kWStages}, as{W::kASlots};
    bool on = true;
    for (int i = blockIdx.x; on && i < items.total; i += step) {
      const Item it(i, items);
#pragma unroll 1
      for (int b = 0; b < it.count; ++b) {
        on = wait(bar(bars.w_full[ws.at]), ws.phase);
        const uint32_t from = src + ws.at * kWStage;
#pragma unroll
        for (int h = 0; on && h < 2; ++h) {
          uint4 q[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) q[c] = lds16(from + ((h * 64 + c * 16) ^ swap));
          on = wait(bar(bars.a_free[d][as.at]), as.phase ^ 1);
          if (!on) break;
          ptx::tc_fence_after();
          const uint32_t to = a_at(d, as.at) + lanes;
#pragma unroll
          for (int j = 0; j < 2; ++j) {  // 32 inputs
            uint32_t v[16];
            pairs_of(q[j * 2].x, v[0], v[1]), pairs_of(q[j * 2].y, v[2], v[3]);
            pairs_of(q[j * 2].z, v[4], v[5]), pairs_of(q[j * 2].w, v[6], v[7]);
            pairs_of(q[j * 2 + 1].x, v[8], v[9]), pairs_of(q[j * 2 + 1].y, v[10], v[11]);
            pairs_of(q[j * 2 + 1].z, v[12], v[13]), pairs_of(q[j * 2 + 1].w, v[14], v[15]);
            tmem_st16(to + j * 16, v);
          }
          tmem_wait_st();
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (h == 1) ptx::mbar_arrive(bar(bars.w_free[ws.at]));
            ptx::mbar_arrive(bar(bars.a_full[d][as.at]));
          }
          as.next();
        }
        if (!on) break;
        ws.next();
      }
    }
  } else {
    registers<56, false>();
    if (warp == 16) {
      // ---- copies of W ----
      Ring ws{W::kWStages};
      bool on = true;
      for (int i = blockIdx.x; on && i < items.total; i += step) {
        const Item it(i, items);
        const bool second = it.tile * 256 + 128 < a.N;
        for (int b = 0; b < it.count; ++b) {
          on = wait(bar(bars.w_free[ws.at]), ws.phase ^ 1);
          if (!on) break;
          if (lane == 0) {
            const uint32_t dst = base + ws.at * kWStage, full = bar(bars.w_full[ws.at]);
            ptx::mbar_arrive_expect_tx(full, second ? kWStage : kWStage / 2);
            ptx::tma_load_2d(dst, &map_w, (it.first + b) * 128, it.tile * 256, full);
            if (second)
              ptx::tma_load_2d(dst + kWStage / 2, &map_w, (it.first + b) * 128, it.tile * 256 + 128,
                               full);
          }
          __syncwarp();
          ws.next();
        }
      }
      for (int i = 0; i < W::kWStages; ++i) wait.end(bar(bars.w_full[i]), ws.last(i));
    } else if (warp == 17) {
      // ---- copies of x ----
      pdl_wait();
      Ring xs{W::kXStages};
      bool on = true;
      for (int i = blockIdx.x; on && i < items.total; i += step) {
        const Item it(i, items);
        for (int b = 0; b < it.count; ++b) {
          on = wait(bar(bars.x_free[xs.at]), xs.phase ^ 1);
          if (!on) break;
          if (lane == 0) {
            const uint32_t dst = xs_at + xs.at * W::kXStage, full = bar(bars.x_full[xs.at]);
            ptx::mbar_arrive_expect_tx(full, W::kXStage);
            // rows and inputs past the last one come as zeros
            ptx::tma_load_2d(dst, &map_x, (it.first + b) * 128, it.chunk * NC, full);
            ptx::tma_load_2d(dst + NC * 128, &map_x, (it.first + b) * 128 + 64, it.chunk * NC, full);
          }
          __syncwarp();
          xs.next();
        }
      }
      for (int i = 0; i < W::kXStages; ++i) wait.end(bar(bars.x_full[i]), xs.last(i));
    } else {
      // ---- products of a tile: the warp keeps together, one thread of it issues.
      const bool issues = elect_one();
      auto products = [&](auto tile) {  // places are kept in registers with the tile known
        constexpr int d = decltype(tile)::value;
        constexpr uint32_t idesc = (1u << 4) | (NC >> 3) << 17 | (128u >> 4) << 24;
        Ring xs{W::kXStages}, as{W::kASlots};
        Places places;
        bool on = true;
        for (int i = blockIdx.x; on && i < items.total; i += step) {
          const Item it(i, items);
          bool fresh = true;
#pragma unroll 1
          for (int b = 0; on && b < it.count; ++b) {
            if (fresh) on = wait(bar(bars.d_free[places.of[d]]), places.parity(d) ^ 1);
            on = on && wait(bar(bars.x_full[xs.at]), xs.phase);
            const uint64_t x = ptx::sw128_desc(xs_at + xs.at * W::kXStage, 0, 1024);
            const uint32_t to = d_at(places.of[d]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              on = on && wait(bar(bars.a_full[d][as.at]), as.phase);
              if (!on) break;
              ptx::tc_fence_after();
              if (issues) {
#pragma unroll
                for (int k = 0; k < 4; ++k)  // 16 inputs
                  umma_f16_ta(to, a_at(d, as.at) + k * 8, x + (h * (NC * 8) + k * 2), idesc,
                              h > 0 || k > 0 || !fresh);
                ptx::umma_commit(bar(bars.a_free[d][as.at]));
              }
              __syncwarp();
              as.next();
            }
            if (!on) break;
            if (issues) {
              ptx::umma_commit(bar(bars.x_free[xs.at]));
              if (read_after(d, b, it.count)) ptx::umma_commit(bar(bars.d_full[places.of[d]]));
            }
            __syncwarp();
            xs.next();
            fresh = read_after(d, b, it.count);
            // the other tile's turns too: both tiles' places follow one order
            if (read_after(0, b, it.count)) places.next(0);
            if (read_after(1, b, it.count)) places.next(1);
          }
        }
      };
      if (warp == 18) products(std::integral_constant<int, 0>());
      else products(std::integral_constant<int, 1>());
      if (issues) ptx::umma_commit(bar(bars.products));
      __syncwarp();
      wait.end(bar(bars.products), 0);
    }
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 18) ptx::tmem_dealloc(tmem, 512);
}

// The parts of the inputs added up, scaled and stored.
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ Args a) {
  const int64_t n = static_cast<int64_t>(a.rows) * a.N;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  pdl_wait();
  if (i >= n) return;
  const int m = static_cast<int>(i / a.N), o = static_cast<int>(i - static_cast<int64_t>(m) * a.N);
  int sum = 0;
#pragma unroll 4
  for (int p = 0; p < a.splits; ++p) sum += a.part[p * n + i];
  const float v = scaled(sum, a.x_scale[m], a.w_scale[o], a.bias ? a.bias[o] : 0.f);
  if (a.out_f32) static_cast<float*>(a.y)[i] = v;
  else static_cast<__nv_bfloat16*>(a.y)[i] = __float2bfloat16_rn(v);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
// A matrix of `width` values a row, boxes of 128 bytes by `rows`.
bool map_2d(CUtensorMap* m, CUtensorMapDataType type, int size, const void* at, int64_t width,
            int64_t height, int rows) {
  static const EncodeTiledFn encode = []() -> EncodeTiledFn {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(height)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(width) * size};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / size), static_cast<cuuint32_t>(rows)};
  const cuuint32_t unit[2] = {1, 1};
  return encode != nullptr &&
         encode(m, type, 2, const_cast<void*>(at), dims, strides, box, unit,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int columns_of(int64_t rows) { return rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }

constexpr int kSMs = 152;

template <int NC, typename Out>
cudaError_t launch(const Args& a, const __half* x, cudaStream_t s) {
  cudaError_t st = allow_most_smem<wide_kernel<NC, Out>>();
  if (st != cudaSuccess) return st;
  CUtensorMap mw, mx;
  if (!map_2d(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.W, a.K, a.N, 128) ||
      !map_2d(&mx, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, x, a.K, a.rows, NC))
    return cudaErrorInvalidValue;
  Items items;
  items.tiles = (a.N + 255) / 256;
  items.chunks = (a.rows + NC - 1) / NC;
  items.splits = a.splits;
  items.blocks = (a.K + 127) / 128;
  items.total = items.tiles * items.chunks * items.splits;
  const int grid = items.total < kSMs ? items.total : kSMs;
  st = launch_dependent(wide_kernel<NC, Out>, dim3(grid), dim3(kWarpsWide * 32), Wide<NC>::kSmem, s, mw,
                        mx, a, items);
  if (st != cudaSuccess || a.splits == 1) return st;
  const int64_t n = static_cast<int64_t>(a.rows) * a.N;
  return launch_dependent(join_kernel, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0, s,
                          a);
}

}  // namespace

// Into how many parts the inputs are cut, where the outputs alone do not fill the SMs:
// counted in blocks of inputs, with three for an item's beginning and end and three for
// the launch that adds the parts up.
int wide_splits(int64_t rows, int N, int K) {
  const int64_t items = static_cast<int64_t>((N + 255) / 256) *
                        ((rows + columns_of(rows) - 1) / columns_of(rows));
  const int blocks = (K + 127) / 128;
  int best = 1;
  int64_t least = 0;
  for (int s = 1; s == 1 || (s <= 16 && s <= blocks && items < kSMs); ++s) {
    const int64_t cost = (items * s + kSMs - 1) / kSMs * ((blocks + s - 1) / s + 3) + (s > 1 ? 3 : 0);
    if (s == 1 || cost < least) best = s, least = cost;
  }
  return best;
}

template <typename Out>
cudaError_t launch_columns(const Args& a, const __half* x, cudaStream_t s) {
  switch (columns_of(a.rows)) {
    case 32: return launch<32, Out>(a, x, s);
    case 64: return launch<64, Out>(a, x, s);
    default: return launch<128, Out>(a, x, s);
  }
}

cudaError_t launch_wide(const Args& a, const __half* x, cudaStream_t s) {
  if (a.splits > 1) return launch_columns<int32_t>(a, x, s);
  return a.out_f32 ? launch_columns<float>(a, x, s) : launch_columns<__nv_bfloat16>(a, x, s);
}

}  // namespace i8
}  // namespace moe
