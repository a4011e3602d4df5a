// The layout of 4-bit weights (moe.h): a row is w4_blocks(K) blocks of 64 bytes.
#pragma once

#include "common.cuh"

namespace moe {

__host__ __device__ constexpr int w4_blocks(int K) { return (K + 127) / 128; }

}  // namespace moe
