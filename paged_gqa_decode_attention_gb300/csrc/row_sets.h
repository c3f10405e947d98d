// Strided row sets and their overlap, for the aliasing checks of the entry
// points that take token-strided views.
#pragma once

#include <algorithm>
#include <cstdint>

namespace pda {

// A set of equally spaced byte ranges: rows [base + i*stride, + len), i < n.
struct Rows {
  int64_t base, stride, len, n;
};

// Whether two row sets share a byte. Exact for a single range against
// anything and for two sets with the same stride (the views of one fused
// projection buffer); otherwise conservative (whole extents).
inline bool overlaps(Rows a, Rows b) {
  if (a.len <= 0 || b.len <= 0 || a.n <= 0 || b.n <= 0) return false;
  if (a.n == 1 && b.n > 1) std::swap(a, b);
  auto fdiv = [](int64_t x, int64_t y) { return x / y - ((x % y != 0) && ((x < 0) != (y < 0))); };
  if (b.n == 1) {
    if (a.n == 1 || a.stride <= 0) {
      const int64_t a1 = a.base + (a.n - 1) * a.stride + a.len;
      return a.base < b.base + b.len && b.base < a1;
    }
    // rows i with a.base + i*stride in (b.base - a.len, b.base + b.len)
    const int64_t lo = fdiv(b.base - a.len - a.base, a.stride) + 1;
    const int64_t hi = -fdiv(-(b.base + b.len - a.base), a.stride) - 1;
    return std::max<int64_t>(lo, 0) <= std::min<int64_t>(hi, a.n - 1);
  }
  if (a.stride == b.stride && a.stride > 0) {
    // rows i of a and k of b meet iff d - a.len < (i - k) * stride < d + b.len
    const int64_t d = b.base - a.base, S = a.stride;
    const int64_t lo = fdiv(d - a.len, S) + 1;
    const int64_t hi = -fdiv(-(d + b.len), S) - 1;
    return std::max<int64_t>(lo, -(b.n - 1)) <= std::min<int64_t>(hi, a.n - 1);
  }
  const int64_t a1 = a.base + (a.n - 1) * a.stride + a.len;
  const int64_t b1 = b.base + (b.n - 1) * b.stride + b.len;
  return a.base < b1 && b.base < a1;
}

}  // namespace pda
