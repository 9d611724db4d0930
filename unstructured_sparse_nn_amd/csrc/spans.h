// spans.h -- the memory that a call's arguments take, and whether it is shared
// (host).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <algorithm>

namespace snk {

// Memory of a call: n rows of `row` bytes, ld bytes apart (wide: sizes and
// strides are the caller's).
struct span_t {
  __int128 p, row, ld, n;
  span_t(const void* at, __int128 bytes, __int128 stride = 0, __int128 rows = 1)
      : p((uintptr_t)at), row(bytes), ld(stride), n(at && bytes > 0 ? rows : 0) {
    if (n > 1 && ld == row) row *= n, n = 1;
  }
  __int128 end() const { return p + (n - 1) * ld + row; }
  // Whether a row meets the bytes from lo up to hi.
  bool meets(__int128 lo, __int128 hi) const {
    // the first row that ends past lo
    const __int128 i = lo < p + row ? 0 : n == 1 ? 1 : (lo - row - p) / ld + 1;
    return i < n && p + i * ld < hi;
  }
};

// Whether a byte belongs to both.  Rows may lie between the other's rows.
inline bool overlap(const span_t& a, const span_t& b) {
  if (a.n == 0 || b.n == 0 || a.end() <= b.p || b.end() <= a.p) return false;
  if (a.n > b.n) return overlap(b, a);
  if (a.n > 1 && a.ld == b.ld) {  // row i of b begins `at` bytes after row i + q of a
    const __int128 d = b.p - a.p, q = d >= 0 ? d / a.ld : -((a.ld - 1 - d) / a.ld), at = d - q * a.ld;
    auto both = [&](__int128 k) { return std::max<__int128>(0, -k) < std::min(b.n, a.n - k); };
    return (at < a.row && both(q)) || (at + b.row > a.ld && both(q + 1));
  }
  for (__int128 i = 0; i < a.n; ++i)
    if (b.meets(a.p + i * a.ld, a.p + i * a.ld + a.row)) return true;
  return false;
}

// Whether an output lies over an input or over another output.
template <size_t O, size_t I>
inline bool any_overlap(const span_t (&out)[O], const span_t (&in)[I]) {
  for (size_t o = 0; o < O; ++o) {
    for (const span_t& i : in)
      if (overlap(out[o], i)) return true;
    for (size_t q = 0; q < o; ++q)
      if (overlap(out[o], out[q])) return true;
  }
  return false;
}

}  // namespace snk
