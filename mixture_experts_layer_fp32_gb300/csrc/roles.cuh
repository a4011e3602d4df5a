// What kernels of warps with roles share: bounded waits on mbarriers, rings of slots,
// register shares, and fp16 products whose first operand is in the tensor memory.
#pragma once

#include "common.cuh"
#include "sm100_ptx.cuh"

namespace moe {
namespace roles {

// Whether a barrier's phase ends within a second.
constexpr long long kWaitCycles = 2000000000ll;
__device__ __forceinline__ bool arrives(uint32_t bar, int parity) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const long long began = clock64();
  while (!ptx::mbar_try_wait(bar, parity))
    if (clock64() - began > kWaitCycles) return false;
  return true;
}

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

}  // namespace roles
}  // namespace moe
