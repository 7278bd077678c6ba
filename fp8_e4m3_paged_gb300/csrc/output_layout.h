// Layout checks of a call's arrays (no CUDA headers: the host test compiles them by itself).
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

// Rows of L elements of an array in requests and heads (strides >= 0).
struct RowsAt {
  int64_t requests, stride_request, heads, stride_head;
};

// Whether `from` and a whole number (lo to hi) of each of n strides, the longest first, add up to less than L on
// either side of 0.  Of a stride only the numbers are tried that the shorter ones can make up for.
struct Steps {
  int64_t stride, lo, hi;
};
inline bool reach_zero(const Steps* step, int n, __int128 from, int64_t L) {
  using wide = __int128;
  if (n == 0) return from < L && from > -L;
  wide lo = from, hi = from;  // with the shorter ones
  for (int i = 1; i < n; ++i) {
    lo += (wide)step[i].stride * step[i].lo;
    hi += (wide)step[i].stride * step[i].hi;
  }
  auto floor_div = [](wide a, wide b) { return a / b - (a % b < 0); };
  const wide stride = step->stride;
  const wide first = std::max<wide>(step->lo, floor_div(-L - hi, stride) + 1);
  const wide last = std::min<wide>(step->hi, -floor_div(lo - L, stride) - 1);
  for (wide k = first; k <= last; ++k)
    if (reach_zero(step + 1, n - 1, from + stride * k, L)) return true;
  return false;
}

// Whether a row of x and a row of y share a place; y begins `ahead` elements behind x.
inline bool meet(const RowsAt& x, const RowsAt& y, int64_t L, int64_t ahead) {
  if (x.requests < 1 || x.heads < 1 || y.requests < 1 || y.heads < 1) return false;
  // Row starts differ by `ahead` and a whole number of each stride, equal ones joined.
  Steps step[4];
  int n = 0;
  auto add = [&](int64_t stride, int64_t lo, int64_t hi) {
    if (stride == 0 || lo == hi) return;
    int i = 0;
    while (i < n && step[i].stride > stride) ++i;
    if (i < n && step[i].stride == stride) {
      step[i].lo += lo;
      step[i].hi += hi;
      return;
    }
    for (int k = n++; k > i; --k) step[k] = step[k - 1];
    step[i] = {stride, lo, hi};
  };
  add(x.stride_request, 1 - x.requests, 0);
  add(x.stride_head, 1 - x.heads, 0);
  add(y.stride_request, 0, y.requests - 1);
  add(y.stride_head, 0, y.heads - 1);
  return reach_zero(step, n, ahead, L);
}

}  // namespace fp8kv
