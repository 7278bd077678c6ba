// Declarations shared by the units of the gathered weights (score_*.cu, score_api.cpp).
#pragma once

#include "chunk.h"

namespace fp8kv {

constexpr int kScoreStreamRows = 256;   // most query vectors per KV head of the streaming kernel
constexpr int kScoreGroupRows = 16;     // ... of one of its CTAs
constexpr int kScoreAccTokens = 2048;   // positions of a CTA that adds up several row blocks

// Vectors that the streaming kernel keeps the logits of, per position: 4, 8 or a multiple of 16.
inline int score_vectors(int64_t rows) { return rows <= 4 ? 4 : rows <= 8 ? 8 : (int)((rows + 15) / 16 * 16); }

struct ScoreParams {
  ChunkParams c;           // no V, no output; c.S partitions of the rows' sums, c.ml [S][total_q][Hq]
  int32_t stat_part;       // positions of such a partition (tile kernel with per_head above 0: not used)
  int32_t col_part;        // positions of a CTA of the column pass (tile kernel)
  int32_t groups;          // row groups of the column pass; above 1 they meet in `partial`
  int32_t per_head;        // tile kernel, above 0: CTAs per KV head, which find their shares from the lengths
  int32_t vectors;         // as score_vectors
  float* logits;           // [B][Hkv][max_kv_len][vectors] base-2 logits (streaming kernel)
  float* partial;          // [groups][B][Hkv][max_kv_len] (tile kernel, groups > 1)
  const float* in;         // NULL: nothing gathered before
  int64_t in_sr, in_sh;
  float decay;
  float* out;
  int64_t out_sr, out_sh;
};

cudaError_t launch_score_stream(const fp8kv_cache_score_plan_t* plan, const ScoreParams& p, cudaStream_t s);
cudaError_t launch_score_tile(const fp8kv_cache_score_plan_t* plan, const ScoreParams& p, cudaStream_t s);

}  // namespace fp8kv
