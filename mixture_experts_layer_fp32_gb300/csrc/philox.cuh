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

// The four words of each of N blocks.  The blocks go through a round together:
// they share the key's steps and hide the multiplications' latency.
template <int N>
__device__ __forceinline__ void philox_words(const Philox& g, const uint64_t (&ctr)[N],
                                             uint4 (&out)[N]) {
  uint32_t k0 = g.k0, k1 = g.k1;
#pragma unroll
  for (int n = 0; n < N; ++n)
    out[n] = make_uint4(static_cast<uint32_t>(ctr[n]), static_cast<uint32_t>(ctr[n] >> 32), g.c2,
                        g.c3);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      uint4& x = out[n];
      const uint64_t a = static_cast<uint64_t>(x.x) * 0xD2511F53u;
      const uint64_t b = static_cast<uint64_t>(x.z) * 0xCD9E8D57u;
      x.x = static_cast<uint32_t>(b >> 32) ^ x.y ^ k0;
      x.z = static_cast<uint32_t>(a >> 32) ^ x.w ^ k1;
      x.y = static_cast<uint32_t>(b);
      x.w = static_cast<uint32_t>(a);
    }
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
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
