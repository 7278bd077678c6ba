// Barriers of the tile kernel whose order is not plain (no CUDA headers: the
// host test walks every interleaving with these functions).
#pragma once

namespace fp8kv {

struct BarrierAt {
  int slot, parity;
};

// Barrier on which the four warps of row tile q say that half h of P(j) is
// written, and the parity of that phase.
//
// Two row tiles (nq = 2): QK(j+1) is issued behind both halves' waits of tile j, so no
// warp can see S(j+1), let alone arrive for it, before every warp has arrived for
// tile j: one barrier per row tile and half, a phase per tile.
//
// One row tile (nq = 1, D = 256): QK(j+1) is issued between the halves, with only the
// first one waited for, so a fast warp may finish tile j+1 while a slow one has not
// written the second half of P(j).  On one barrier its arrival would complete phase
// j in the slow warp's place.  The second half therefore has a barrier per tile parity:
// tile j+2 arrives on the same one, but needs S(j+2), and QK(j+2) is issued behind the
// wait for the second half of P(j).
constexpr BarrierAt p_ready_at(int nq, int q, int h, int j) {
  return nq == 1 && h == 1 ? BarrierAt{j & 1, (j >> 1) & 1} : BarrierAt{q, j & 1};
}

}  // namespace fp8kv
