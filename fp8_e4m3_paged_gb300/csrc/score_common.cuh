// Device helpers shared by the kernels of the gathered weights.
#pragma once

#include <cstdint>

#include "chunk_common.cuh"
#include "dependent.cuh"
#include "score.h"

namespace fp8kv {

// What a query vector's weights are made of: p_t = 2^(x_t - m) * inv for its base-2 logits x_t.
// A vector that saw nothing (or only logits of -inf) has inv = 0.
struct Norm {
  float m, inv;
};

// Joins the partitions' (maximum, sum) pairs of a vector (whole maxima: weights are powers of
// two), lane after lane of `lanes` neighbouring ones, each of which gets the result.
__device__ __forceinline__ Norm join_norm(const float2* ml, int64_t plane, int64_t vec, int S, int lane = 0,
                                          int lanes = 1) {
  float M = kNoMax, L = 0.f;
  for (int s = lane; s < S; s += lanes) {
    const float2 y = ml[s * plane + vec];
    if (y.y == 0.f) continue;
    const float top = fmaxf(M, y.x);
    L = (L == 0.f ? 0.f : L * part_weight(M, top)) + y.y * part_weight(y.x, top);
    M = top;
  }
  for (int o = lanes / 2; o > 0; o /= 2) {
    const float m = __shfl_xor_sync(0xffffffffu, M, o), l = __shfl_xor_sync(0xffffffffu, L, o);
    const float top = fmaxf(M, m);
    // (the same order of the two in both lanes: the sum is the same)
    const float a = L == 0.f ? 0.f : L * part_weight(M, top), b = l == 0.f ? 0.f : l * part_weight(m, top);
    L = a + b;
    M = top;
  }
  return {M == kNoMax ? 0.f : M, L == 0.f ? 0.f : 1.f / L};
}

// The new weight of position t: what it had gathered, unless it is one of the new tokens, and `got`.
__device__ __forceinline__ void write_score(const ScoreParams& p, int b, int g, int t, int base, float got) {
  if (p.in && t < base) got = fmaf(p.decay, p.in[b * p.in_sr + g * p.in_sh + t], got);
  p.out[b * p.out_sr + g * p.out_sh + t] = got;
}

}  // namespace fp8kv
