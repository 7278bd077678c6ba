// Chunk attention: instances of the tile kernel.
#include "chunk_tile_kernel.cuh"

namespace fp8kv {

cudaError_t launch_chunk_tile(const fp8kv_chunk_plan_t* plan, const ChunkParams& p, cudaStream_t st) {
  return launch<false>(plan, p, st);
}

}  // namespace fp8kv
