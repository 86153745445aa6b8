// Whether strided sets of rows share memory (host code, no CUDA).
//
// Row (i0, i1, i2) of a set starts st . i elements past p.  Two sets meet when some
// two of their rows overlap: when an integer combination of strides, each index
// within its bounds, comes within a row of the distance between them.  Indices of
// equal strides act as one; the largest stride is tried first and only the
// indices that the smaller ones can still make up for, one or two each when the
// strides are nested, as views' are.  A search that gets long ends with "may meet".
#pragma once

#include <algorithm>
#include <cstdint>

namespace csa {

struct Rows {
  const void* p;
  int dims;      // <= 3
  int64_t n[3];
  int64_t st[3];  // elements, non-negative
  int64_t row;   // elements of a row, dense
  int es;        // bytes of an element

  bool empty() const {
    for (int i = 0; i < dims; ++i)
      if (n[i] <= 0) return true;
    return row <= 0;
  }
  // bytes from the first to past the last element
  __int128 span() const {
    __int128 most = row;
    for (int i = 0; i < dims; ++i) most += static_cast<__int128>(n[i] - 1) * st[i];
    return most * es;
  }
};

namespace rows_detail {

struct Term {
  __int128 step, lo, hi;  // step > 0, times an integer in [lo, hi]
};

inline __int128 floor_div(__int128 a, __int128 b) {  // b > 0
  const __int128 q = a / b;
  return q * b > a ? q - 1 : q;
}

struct Search {
  Term t[6];
  int nt = 0;
  __int128 least[7], most[7];  // what the terms from k on add up to
  __int128 lo, hi;             // the sum must lie strictly between
  int left = 4096;             // steps

  void add(__int128 step, __int128 a, __int128 b) {
    if (step == 0 || a == b) return;
    t[nt++] = Term{step, a, b};
  }
  void merge_equal() {
    std::sort(t, t + nt, [](const Term& a, const Term& b) { return a.step > b.step; });
    int m = 0;
    for (int i = 0; i < nt; ++i) {
      if (m > 0 && t[m - 1].step == t[i].step) {
        t[m - 1].lo += t[i].lo;
        t[m - 1].hi += t[i].hi;
      } else {
        t[m++] = t[i];
      }
    }
    nt = m;
  }
  bool run(__int128 start, bool nonzero) {
    least[nt] = most[nt] = 0;
    for (int k = nt - 1; k >= 0; --k) {
      least[k] = least[k + 1] + t[k].step * t[k].lo;
      most[k] = most[k + 1] + t[k].step * t[k].hi;
    }
    return from(0, start, nonzero);
  }
  bool from(int k, __int128 v, bool nonzero) {
    if (k == nt) return nonzero && lo < v && v < hi;
    const __int128 s = t[k].step;
    const __int128 a = std::max(t[k].lo, -floor_div(-(lo + 1 - v - most[k + 1]), s));
    const __int128 b = std::min(t[k].hi, floor_div(hi - 1 - v - least[k + 1], s));
    for (__int128 i = a; i <= b; ++i) {
      if (--left < 0) return true;
      if (from(k + 1, v + s * i, nonzero || i != 0)) return true;
    }
    return false;
  }
};

}  // namespace rows_detail

// Some row of a and some row of b share a byte.
inline bool rows_meet(const Rows& a, const Rows& b) {
  if (a.empty() || b.empty()) return false;
  const __int128 pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  if (pa + a.span() <= pb || pb + b.span() <= pa) return false;
  rows_detail::Search s;
  for (int i = 0; i < b.dims; ++i) s.add(static_cast<__int128>(b.st[i]) * b.es, 0, b.n[i] - 1);
  for (int i = 0; i < a.dims; ++i) s.add(static_cast<__int128>(a.st[i]) * a.es, -(a.n[i] - 1), 0);
  s.merge_equal();
  s.lo = -static_cast<__int128>(b.row) * b.es;
  s.hi = static_cast<__int128>(a.row) * a.es;
  return s.run(pb - pa, true);
}

// Two rows of a share an element.
inline bool rows_meet_themselves(const Rows& a) {
  if (a.empty()) return false;
  int order[3] = {0, 1, 2};
  std::sort(order, order + a.dims, [&](int x, int y) { return a.st[x] < a.st[y]; });
  __int128 extent = a.row;
  bool nested = true;  // each stride reaches past all that lies within it
  for (int k = 0; k < a.dims; ++k) {
    const int i = order[k];
    if (a.n[i] <= 1) continue;
    if (a.st[i] == 0) return true;
    nested = nested && a.st[i] >= extent;
    extent += static_cast<__int128>(a.n[i] - 1) * a.st[i];
  }
  if (nested) return false;
  rows_detail::Search s;
  for (int i = 0; i < a.dims; ++i) s.add(a.st[i], -(a.n[i] - 1), a.n[i] - 1);
  std::sort(s.t, s.t + s.nt,
            [](const rows_detail::Term& x, const rows_detail::Term& y) { return x.step > y.step; });
  s.lo = -a.row;
  s.hi = a.row;
  return s.run(0, false);
}

}  // namespace csa
