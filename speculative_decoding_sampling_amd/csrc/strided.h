// Whether rows at strides lie over each other: what a call asks before it launches,
// so in steps that grow with the shorter of two axes alone.
#pragma once

#include <cstddef>
#include <cstdint>

#include "abi_checks.h"

namespace specv {

// One axis of an array's rows: n of them, s >= 0 bytes apart.
struct Axis {
  int64_t n, s;
};
inline Axis axis(int n, size_t s) { return {n, n > 1 ? (int64_t)s : 0}; }
// The axes of an array, the shorter one first.
struct Axes {
  Axis few, many;
};
inline Axes axes(const Rows& r) {
  const Axis b = axis(r.B, r.sb), k = axis(r.nk, r.sk);
  return b.n < k.n ? Axes{b, k} : Axes{k, b};
}

inline int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b < 0 ? 1 : 0); }   // b > 0
inline int64_t ceil_div(int64_t a, int64_t b) { return -floor_div(-a, b); }

// Whether c + d s lies in [lo, hi] for some d in [from, to].
inline bool any_in(int64_t c, int64_t s, int64_t from, int64_t to, int64_t lo, int64_t hi) {
  if (s == 0) return from <= to && lo <= c && c <= hi;
  const int64_t first = ceil_div(lo - c, s), d = first > from ? first : from;
  return d <= to && c + d * s <= hi;
}

// The least x in [0, n] with lo <= a x mod m <= hi, where 0 < lo <= hi < m; -1 for
// none.  If no multiple of a lies in [lo, hi] itself, a x = m y + v with v there:
// (m y) mod a then lies in [-hi mod a, -lo mod a], the same question of smaller
// numbers, whose least y gives the least x (Euclid's steps).  No product here exceeds a n.
inline int64_t least_multiple(int64_t a, int64_t m, int64_t lo, int64_t hi, int64_t n) {
  if (a == 0) return -1;
  int64_t x = ceil_div(lo, a);
  if (x > n) return -1;
  if (a * x <= hi) return x;
  const int64_t y = least_multiple(m % a, a, a - hi % a, a - lo % a, a * n / m);
  if (y < 0) return -1;
  x = ceil_div(lo + m * y, a);
  return x <= n ? x : -1;
}

// Whether c + i a.s - j b.s lies in [lo, hi] for some i < a.n, j < b.n.
inline bool axes_meet(int64_t c, const Axis& a, const Axis& b, int64_t lo, int64_t hi) {
  if (a.s == b.s) return any_in(c, a.s, -(b.n - 1), a.n - 1, lo, hi);
  if (a.s > b.s) return axes_meet(-c, b, a, -hi, -lo);
  // the i at which the other axis is near: there j is in range if any is, and the
  // question is whether c - lo + i a.s is at most hi - lo above a multiple of b.s
  int64_t i0 = 0, i1 = a.n - 1;
  const int64_t end = (b.n - 1) * b.s + hi - c;              // c + i a.s at most that
  if (a.s == 0) {
    if (c < lo || end < 0) return false;
    i1 = 0;
  } else {
    const int64_t first = ceil_div(lo - c, a.s), last = floor_div(end, a.s);
    if (first > i0) i0 = first;
    if (last < i1) i1 = last;
    if (i0 > i1) return false;
  }
  const int64_t r = (c - lo + i0 * a.s) % b.s;
  if (r <= hi - lo) return true;
  return least_multiple(a.s, b.s, b.s - r, b.s - r + hi - lo, i1 - i0) >= 0;
}

// Whether a row of one array lies over a row of the other.
inline bool rows_overlap(const Rows& a, const Rows& b) {
  if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
  const Axes x = axes(a), y = axes(b);
  auto extent = [](const Rows& r, const Axes& e) {
    return Span{r.p, (size_t)((e.few.n - 1) * e.few.s + (e.many.n - 1) * e.many.s) + r.n};
  };
  if (!overlap(extent(a, x), extent(b, y))) return false;
  // the distance of two starts at which rows meet
  const int64_t lo = 1 - (int64_t)a.n, hi = (int64_t)b.n - 1;
  const int64_t c = (int64_t)(reinterpret_cast<uintptr_t>(a.p) - reinterpret_cast<uintptr_t>(b.p));
  if (x.few.s == y.few.s) {
    for (int64_t d = -(y.few.n - 1); d < x.few.n; ++d)
      if (axes_meet(c + d * x.few.s, x.many, y.many, lo, hi)) return true;
    return false;
  }
  for (int64_t i = 0; i < x.few.n; ++i)
    for (int64_t j = 0; j < y.few.n; ++j)
      if (axes_meet(c + i * x.few.s - j * y.few.s, x.many, y.many, lo, hi)) return true;
  return false;
}

// Whether the rows of an array lie over each other: two of them, d apart along the
// shorter axis and e along the other.
inline bool self_overlap(const Rows& r) {
  if (!r.p || r.n == 0) return false;
  const Axes x = axes(r);
  const int64_t near = (int64_t)r.n - 1;
  if (x.many.n > 1 && x.many.s <= near) return true;                     // d = 0
  for (int64_t d = 1; d < x.few.n; ++d)
    if (any_in(d * x.few.s, x.many.s, 1 - x.many.n, x.many.n - 1, -near, near)) return true;
  return false;
}

}  // namespace specv
