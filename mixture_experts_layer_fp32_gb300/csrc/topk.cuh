// The router's choice for one token, by one warp: scores, (group scores and the
// kept groups), top-k by k rounds of a warp arg-max, combine weights.  Shared by
// the router's own kernels and the layer for few tokens.
#pragma once

#include <float.h>

#include "common.cuh"

namespace moe {

__device__ __forceinline__ bool better(float v, int i, float bv, int bi) {
  return v > bv || (v == bv && i < bi);
}

// s: the token's logits with the gate bias, expert lane + 32 i in s[i], -FLT_MAX
// past E.  gsel: E floats of shared memory of this warp's own (used with groups).
// Lane j < k is left with slot j: my_idx and its weight p.
// PL: experts per lane (E <= 32 * PL): the per-lane loops cover no more entries
// than E needs.
template <int PL>
__device__ __forceinline__ void choose_topk(float (&s)[PL], int t, int E, int k, int score,
                                            int num_groups, int group_topk,
                                            const float* __restrict__ expert_bias, float* gsel,
                                            int* err, int& my_idx, float& p) {
  const int lane = threadIdx.x & 31;
  const int per_group = num_groups > 1 ? E / num_groups : E;
  float sel[PL];
  if (score == MOE_SCORE_SOFTMAX_PRE) {
    float m = -FLT_MAX;
#pragma unroll
    for (int i = 0; i < PL; ++i) m = fmaxf(m, s[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int e = lane + 32 * i;
      s[i] = (e < E) ? expf(s[i] - m) : 0.f;
      z += s[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int e = lane + 32 * i;
      s[i] = (e < E) ? s[i] / z : 0.f;
      sel[i] = (e < E) ? s[i] : -FLT_MAX;
    }
  } else if (score == MOE_SCORE_SIGMOID || score == MOE_SCORE_SQRTSOFTPLUS) {
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int e = lane + 32 * i;
      if (e < E) {
        if (score == MOE_SCORE_SIGMOID) {
          s[i] = 1.f / (1.f + expf(-s[i]));
        } else {
          // softplus(l) = log(1 + e^l) = max(l, 0) + log1p(e^-|l|): no overflow
          s[i] = sqrtf(fmaxf(s[i], 0.f) + log1pf(expf(-fabsf(s[i]))));
        }
        sel[i] = expert_bias ? s[i] + expert_bias[e] : s[i];
      } else {
        s[i] = 0.f;
        sel[i] = -FLT_MAX;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < PL; ++i) sel[i] = s[i];
  }

  // group-limited top-k: lane g < num_groups scores group g (the sum of its
  // k/group_topk best selection scores, largest first), then group_topk
  // rounds of a warp arg-max keep the best groups; the other groups'
  // experts are marked taken so that the expert rounds skip them
  uint32_t taken = 0;
  if (num_groups > 1) {
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int e = lane + 32 * i;
      if (e < E) gsel[e] = sel[i];
    }
    __syncwarp();
    float gs = -INFINITY;
    if (lane < num_groups) {
      const float* g = gsel + lane * per_group;
      const int m = k / group_topk;
      uint32_t used[MOE_MAX_EXPERTS / 32] = {0, 0, 0, 0, 0, 0, 0, 0};
      gs = 0.f;
      for (int r = 0; r < m; ++r) {
        float bv = -INFINITY;
        int bi = 0x7fffffff;
        for (int c = 0; c < per_group; ++c)
          if (!(used[c >> 5] >> (c & 31) & 1u) && better(g[c], c, bv, bi)) {
            bv = g[c];
            bi = c;
          }
        if (bi >= per_group) break;  // only on NaN scores (reported by the expert rounds)
        used[bi >> 5] |= 1u << (bi & 31);
        gs += bv;
      }
    }
    __syncwarp();  // gsel is rewritten for the next token
    uint32_t kept = 0;
    for (int r = 0; r < group_topk; ++r) {
      float bv = (lane < num_groups && !(kept >> lane & 1u)) ? gs : -INFINITY;
      int bi = (lane < num_groups && !(kept >> lane & 1u)) ? lane : 0x7fffffff;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float ov = __shfl_xor_sync(0xffffffffu, bv, o);
        const int oi = __shfl_xor_sync(0xffffffffu, bi, o);
        if (better(ov, oi, bv, bi)) {
          bv = ov;
          bi = oi;
        }
      }
      if (bi < num_groups) kept |= 1u << bi;
    }
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int e = lane + 32 * i;
      if (e < E && !(kept >> (e / per_group) & 1u)) taken |= 1u << i;
    }
  }

  // k rounds of a warp-wide arg-max over the not-yet-taken experts
  my_idx = -1;  // lane j < k keeps slot j
  float my_s = 0.f;
  for (int j = 0; j < k; ++j) {
    // this lane's best candidate as an ordered key (a larger score, a larger
    // key; -0 as +0; 0 = none, NaN scores never count), the lower expert on
    // ties (i rises with e); then the warp's largest key and, among the
    // lanes holding it, the lowest expert: two warp reductions
    uint32_t bk = 0;
    int bi = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int e = lane + 32 * i;
      if (e < E && !(taken >> i & 1u) && !isnan(sel[i])) {
        uint32_t u = __float_as_uint(sel[i]);
        if (u == 0x80000000u) u = 0u;
        const uint32_t key = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
        if (key > bk) {
          bk = key;
          bi = e;
        }
      }
    }
    const uint32_t mk = __reduce_max_sync(0xffffffffu, bk);
    bi = static_cast<int>(
        __reduce_min_sync(0xffffffffu, (mk != 0u && bk == mk) ? static_cast<uint32_t>(bi)
                                                              : 0x7fffffffu));
    if (mk == 0u || bi >= E) {  // only on NaN logits
      if (lane == 0) report_error(err, DEV_ERR_INDEX, t);
      bi = 0;
    }
    const int owner = bi & 31;
    float sv = 0.f;
#pragma unroll
    for (int i = 0; i < PL; ++i)
      if (lane == owner && (bi >> 5) == i) {
        taken |= 1u << i;
        sv = s[i];
      }
    sv = __shfl_sync(0xffffffffu, sv, owner);
    if (lane == j) {
      my_idx = bi;
      my_s = sv;
    }
  }

  // combine weights
  p = 0.f;
  if (score == MOE_SCORE_SOFTMAX_POST) {
    const float m = __shfl_sync(0xffffffffu, my_s, 0);
    const float ex = (lane < k) ? expf(my_s - m) : 0.f;
    float z = ex;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    p = ex / z;
  } else if (score == MOE_SCORE_SOFTMAX_PRE) {
    p = my_s;
  } else {
    float z = (lane < k) ? my_s : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    p = my_s / (z + 1e-20f);
  }
}

}  // namespace moe
