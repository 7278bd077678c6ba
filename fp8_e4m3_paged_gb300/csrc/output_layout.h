// Layout check of a call's outputs (no CUDA headers: the host test compiles it by itself).
#pragma once

#include <algorithm>
#include <cstdint>

namespace fp8kv {

// No two rows or heads of an output, D elements each, share a place (strides >= 0).
inline bool apart(int64_t rows, int64_t stride_row, int64_t heads, int64_t stride_head, int64_t D) {
  using wide = __int128;  // products of any count and stride
  if (rows < 2 || heads < 2) return (rows < 2 || stride_row >= D) && (heads < 2 || stride_head >= D);
  const bool by_row = stride_row >= stride_head;
  const int64_t outer = by_row ? stride_row : stride_head, inner = by_row ? stride_head : stride_row;
  const int64_t n_outer = by_row ? rows : heads, n_inner = by_row ? heads : rows;
  if (inner < D) return false;
  const wide span = (wide)(n_inner - 1) * inner + D;
  if (outer >= span) return true;  // one inside of the other, as usual
  // Interleaved: each multiple of the outer stride against the inner multiples next to
  // it, as far as those reach (no further than the smaller count, as inner <= outer).
  const int64_t reach = (int64_t)std::min<wide>(n_outer - 1, span / outer);
  for (int64_t i = 1; i <= reach; ++i) {
    const wide at = (wide)i * outer, k = at / inner;
    const wide below = at - std::min<wide>(k, n_inner - 1) * inner, above = (k + 1) * inner - at;
    if (below < D || (k + 1 < n_inner && above < D)) return false;
  }
  return true;
}

}  // namespace fp8kv
