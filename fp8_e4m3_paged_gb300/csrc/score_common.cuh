// Device helpers shared by the kernels of the gathered weights.
#pragma once

#include <cstdint>

#include "chunk_common.cuh"
#include "score.h"

namespace fp8kv {

// What a query vector's weights are made of: p_t = 2^(x_t - m) * inv for its base-2 logits x_t.
// A vector that saw nothing (or only logits of -inf) has inv = 0.
struct Norm {
  float m, inv;
};

// Joins the partitions' (maximum, sum) pairs of a vector (whole maxima: weights are powers of two).
__device__ __forceinline__ Norm join_norm(const float2* ml, int64_t plane, int64_t vec, int S) {
  float M = kNoMax, L = 0.f;
  for (int s = 0; s < S; ++s) M = fmaxf(M, ml[s * plane + vec].x);
  for (int s = 0; s < S; ++s) {
    const float2 y = ml[s * plane + vec];
    if (y.y != 0.f) L = fmaf(part_weight(y.x, M), y.y, L);
  }
  return {M == kNoMax ? 0.f : M, L == 0.f ? 0.f : 1.f / L};
}

// The new weight of position t: what it had gathered, unless it is one of the new tokens, and `got`.
__device__ __forceinline__ void write_score(const ScoreParams& p, int b, int g, int t, int base, float got) {
  if (p.in && t < base) got = fmaf(p.decay, p.in[b * p.in_sr + g * p.in_sh + t], got);
  p.out[b * p.out_sr + g * p.out_sh + t] = got;
}

}  // namespace fp8kv
