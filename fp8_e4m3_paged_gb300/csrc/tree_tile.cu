// Tree attention: instances of the tile kernel whose new tokens see each other by their masks.  Tiles of the
// context are as in the chunk attention; a tile that holds nodes takes 32 bits of the row's mask at a time, shifted
// to the tile, so masks cost a load per row and 32 nodes, and the context, which bounds the call, nothing.
// 16 trees of 9 to 64 nodes, 32 heads over 8, D 128, on 100 to 8000 positions: 69 us with the join (shares by
// the lengths: share_of), most of it CTAs' starts and tiles' hand-offs; one of 64 on 131008: 76 us, 0.9 PFLOP/s.
#include "chunk_tile_kernel.cuh"

namespace fp8kv {

cudaError_t launch_tree_tile(const fp8kv_chunk_plan_t* plan, const ChunkParams& p, cudaStream_t st) {
  return launch<true>(plan, p, st);
}

}  // namespace fp8kv
