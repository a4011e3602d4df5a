// Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy
// as 1, 2, 3", SC 2011) and the dropout mask that is drawn from it.  The mask
// is a function of the key, the offset and an element's place alone, so the
// backward pass draws it again instead of reading it.
#pragma once

#include <stdint.h>

namespace moe {

struct Philox {
  uint32_t k0, k1, c2, c3;  // key = seed, counter words 2 and 3 = offset
};

__device__ __forceinline__ Philox philox_of(const uint64_t* rng) {
  const uint64_t seed = rng[0], offset = rng[1];
  return {static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32),
          static_cast<uint32_t>(offset), static_cast<uint32_t>(offset >> 32)};
}

// the four words of block `ctr`
__device__ __forceinline__ uint4 philox_words(const Philox& g, uint64_t ctr) {
  uint32_t x0 = static_cast<uint32_t>(ctr), x1 = static_cast<uint32_t>(ctr >> 32), x2 = g.c2,
           x3 = g.c3, k0 = g.k0, k1 = g.k1;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = static_cast<uint64_t>(x0) * 0xD2511F53u;
    const uint64_t b = static_cast<uint64_t>(x2) * 0xCD9E8D57u;
    x0 = static_cast<uint32_t>(b >> 32) ^ x1 ^ k0;
    x2 = static_cast<uint32_t>(a >> 32) ^ x3 ^ k1;
    x1 = static_cast<uint32_t>(b);
    x3 = static_cast<uint32_t>(a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(x0, x1, x2, x3);
}

// Dropout of probability p, 0 < p <= 1: an element is kept iff its word is
// above `limit` = floor(p 2^32) - 1, and scaled by 1/(1-p).  p below 2^-32
// keeps everything: `on` is 0.
struct Dropout {
  uint32_t limit;
  float scale;
  int on;
};

inline Dropout dropout_of(double p) {
  const double t = p * 4294967296.0;
  const uint64_t threshold = static_cast<uint64_t>(t);  // floor, at most 2^32
  Dropout d;
  d.on = threshold > 0;
  d.limit = d.on ? static_cast<uint32_t>(threshold - 1) : 0u;
  d.scale = p < 1.0 ? static_cast<float>(1.0 / (1.0 - p)) : 0.f;
  return d;
}

}  // namespace moe
