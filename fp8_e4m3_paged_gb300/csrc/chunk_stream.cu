// Chunk attention: instances of the stream kernel.
#include "chunk_stream_kernel.cuh"

namespace fp8kv {

cudaError_t launch_chunk_stream(const fp8kv_chunk_plan_t* plan, const ChunkParams& p, cudaStream_t st) {
  return launch<false>(plan, p, st);
}

}  // namespace fp8kv
