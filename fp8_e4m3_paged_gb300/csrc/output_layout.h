// Layout checks of a call's arrays (no CUDA headers: the host test compiles them by itself).
#pragma once

#include <algorithm>
#include <cstdint>
#include <utility>

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

// Whether a row of x and a row of y share a place; y begins `ahead` elements behind x.
inline bool meet(const RowsAt& x, const RowsAt& y, int64_t L, int64_t ahead) {
  using wide = __int128;
  if (x.requests < 1 || x.heads < 1 || y.requests < 1 || y.heads < 1) return false;
  // Row starts differ by `ahead` and a whole number of each of these steps, equal ones joined.
  struct {
    int64_t stride, lo, hi;
  } step[4];
  int n = 0;
  auto add = [&](int64_t stride, int64_t lo, int64_t hi) {
    if (stride == 0 || lo == hi) return;
    for (int i = 0; i < n; ++i)
      if (step[i].stride == stride) {
        step[i].lo += lo;
        step[i].hi += hi;
        return;
      }
    step[n++] = {stride, lo, hi};
  };
  add(x.stride_request, 1 - x.requests, 0);
  add(x.stride_head, 1 - x.heads, 0);
  add(y.stride_request, 0, y.requests - 1);
  add(y.stride_head, 0, y.heads - 1);
  wide lo = ahead, hi = ahead;
  for (int i = 0; i < n; ++i) {
    lo += (wide)step[i].stride * step[i].lo;
    hi += (wide)step[i].stride * step[i].hi;
  }
  if (lo >= L || hi <= -L) return false;  // one behind the other, as usual
  if (n == 0) return true;
  // Views into each other: all of the shorter steps, and of the longest one the two that come nearest.
  for (int i = 0; i + 1 < n; ++i)
    if (step[i].hi - step[i].lo > step[n - 1].hi - step[n - 1].lo) std::swap(step[i], step[n - 1]);
  const wide stride = step[n - 1].stride;
  int64_t at[3];
  wide from = ahead;
  for (int i = 0; i + 1 < n; ++i) {
    at[i] = step[i].lo;
    from += (wide)step[i].stride * at[i];
  }
  while (true) {
    const wide below = -from / stride - (-from % stride < 0);
    for (wide k = below; k <= below + 1; ++k) {
      const wide d = from + stride * std::min<wide>(std::max<wide>(k, step[n - 1].lo), step[n - 1].hi);
      if (d < L && d > -L) return true;
    }
    int i = 0;
    while (i + 1 < n && at[i] == step[i].hi) {
      from -= (wide)step[i].stride * (step[i].hi - step[i].lo);
      at[i] = step[i].lo;
      ++i;
    }
    if (i + 1 >= n) return false;
    ++at[i];
    from += step[i].stride;
  }
}

}  // namespace fp8kv
