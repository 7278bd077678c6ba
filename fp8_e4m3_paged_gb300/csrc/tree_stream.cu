// Tree attention: instances of the stream kernel whose new tokens see each other by their masks (a bit per row
// and node, looked up for nodes only).  Latency bounds it: a tree of 26 with 6 heads of
// D 256 on 611 positions takes 12 us, its ten CTAs' rows and their join in the cluster.
#include "chunk_stream_kernel.cuh"

namespace fp8kv {

cudaError_t launch_tree_stream(const fp8kv_chunk_plan_t* plan, const ChunkParams& p, cudaStream_t st) {
  return launch<true>(plan, p, st);
}

}  // namespace fp8kv
