// Declarations shared by the chunk-attention units (chunk_*.cu, chunk_api.cpp).
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "fp8kv_attn.h"

namespace fp8kv {

constexpr int kChunkStreamRows = 16;      // query vectors per CTA of the stream kernel
constexpr int kChunkClusterMax = 8;       // partitions that the stream kernel joins in one launch (portable cluster size)
constexpr int kChunkStreamBlock = 16;     // positions per warp step of the stream kernel
constexpr int kChunkTileTokens = 128;     // positions per tile of the tile kernel
// Most positions of one FP32 sum: the tensor core's accumulation truncates, so
// a sum drifts by about 2^-25 of itself per K16 step; 2048 steps keep that below
// 2^-14, a quarter of the half-step of an fp16 output.  The tile kernel sums a
// partition in one chain, a step for 16 positions; the stream kernel in a chain per
// warp, two steps for 16 positions (both halves of P).
constexpr int kChunkMaxSum = 32768;
constexpr int kChunkStreamWarps = 4;
inline int64_t chunk_max_part(int32_t kernel) {
  return kernel == FP8KV_CHUNK_STREAM ? kChunkStreamWarps * kChunkMaxSum / 2 : kChunkMaxSum;
}
constexpr int kShareMax = 128;             // requests that a CTA finds its share among (share_of)
constexpr int kTreeNodesMax = 1024;         // nodes of one request's tree
inline int chunk_tile_rows(int head_dim) { return head_dim == 256 ? 128 : 256; }  // query vectors per CTA

// Everything the chunk kernels need, resolved on the host.
struct ChunkParams {
  int32_t B, total_q, max_q, Hq, Hkv, G, S;
  int32_t parts, max_part;  // a context's partitions: `parts`, more (up to S) of max_part positions if it is longer
  int32_t page_size, max_kv_len, num_kv_blocks;
  uint64_t page_div;       // as Params::page_div
  uint64_t g_div, s_div, parts_div, hkv_div;  // the same for G, S, parts and Hkv
  int32_t window, sinks;   // window 0: every earlier position
  int32_t row_tiles;
  const uint16_t* q;
  int64_t q_st, q_sh;      // elements
  uint16_t* out;
  int64_t o_st, o_sh;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  int64_t ksb, kst, ksh, vsb, vst, vsh;  // bytes
  const int32_t* block_table;
  int64_t bt_stride;
  const int32_t* cu_q;
  const int32_t* kv_len;
  float softmax_scale, k_scale, v_scale;
  const float* k_scale_dev;
  const float* v_scale_dev;
  unsigned int* status;
  float* partial;          // [S][total_q][Hq][D] (S > 1)
  float2* ml;              // [S][total_q][Hq]
  // trees of drafted tokens
  const uint32_t* mask;    // [total_q][mask_stride] bit j % 32 of word j / 32: the row sees new token j
  int64_t mask_stride;     // words
  const int32_t* depth;    // [total_q] (windows only)
  int32_t per_head;        // above 0: CTAs per KV head, which find their shares from the lengths (share_of)
  int32_t* share;          // where they leave the partitions' length for the join
};

// Whether the partitions form a cluster that joins them itself: only where all of them have
// work, since a CTA that waits for its cluster holds its place on the SM (64 decodes of 4000
// positions planned for 131072, two partitions of which one is empty: 158 us in
// clusters, 98 through the workspace).
inline bool chunk_clustered(const fp8kv_chunk_plan_t* plan) {
  return plan->kernel == FP8KV_CHUNK_STREAM && plan->num_splits > 1 && plan->num_splits <= kChunkClusterMax &&
         plan->min_splits == plan->num_splits;
}

cudaError_t launch_chunk_stream(const fp8kv_chunk_plan_t* plan, const ChunkParams& p, cudaStream_t s);
cudaError_t launch_chunk_tile(const fp8kv_chunk_plan_t* plan, const ChunkParams& p, cudaStream_t s);
cudaError_t launch_tree_stream(const fp8kv_chunk_plan_t* plan, const ChunkParams& p, cudaStream_t s);
cudaError_t launch_tree_tile(const fp8kv_chunk_plan_t* plan, const ChunkParams& p, cudaStream_t s);
cudaError_t launch_chunk_join(const fp8kv_chunk_plan_t* plan, const ChunkParams& p, cudaStream_t s);
cudaError_t launch_tree_join(const fp8kv_chunk_plan_t* plan, const ChunkParams& p, cudaStream_t s);
cudaError_t launch_cache_read(const fp8kv_cache_read_args& a, cudaStream_t s);
cudaError_t launch_calibrate(const fp8kv_calibrate_args& a, cudaStream_t s);

}  // namespace fp8kv
