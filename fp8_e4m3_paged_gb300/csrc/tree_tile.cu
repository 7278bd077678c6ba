// Tree attention: instances of the tile kernel whose new tokens see each other by their masks.
#include "chunk_tile_kernel.cuh"

namespace fp8kv {

cudaError_t launch_tree_tile(const fp8kv_chunk_plan_t* plan, const ChunkParams& p, cudaStream_t st) {
  return launch<true>(plan, p, st);
}

}  // namespace fp8kv
