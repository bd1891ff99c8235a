// Whether sets of strided rows share memory (host side).
#pragma once

#include <stdint.h>

namespace lf {

// Rows of `bytes` bytes: row (i, j, k) starts at byte at + i stride[0] + j stride[1] + k stride[2], i < n[0], ...
struct RowSet {
  uintptr_t at;
  int64_t n[3], stride[3];   // n >= 1, strides >= 0
  int64_t bytes;
};

enum class Overlap { kNo, kYes, kUnknown };

namespace overlap_detail {

typedef __int128 Wide;       // sizes times strides

struct Term {
  Wide stride, lo, hi;       // adds i * stride for one i of [lo, hi]
};

// Is there a choice of the terms from t[0] on (not all of them zero, where `other` is not set yet) whose sum lies within
// bytes - 1 of `target`?  The terms come with their strides falling: once the later ones' reach is taken off, few i are
// left of each, and one or two where rows lie inside rows as those of a view of a tensor do.
inline Overlap find(const Term* t, int n, Wide target, Wide bytes, bool other, int* steps) {
  if (n == 0) return other && target < bytes && -target < bytes ? Overlap::kYes : Overlap::kNo;
  Wide lo = 0, hi = 0;       // reach of the later terms
  for (int j = 1; j < n; ++j) {
    lo += t[j].lo * t[j].stride;
    hi += t[j].hi * t[j].stride;
  }
  // i stride + [lo, hi] meets (target - bytes, target + bytes)
  auto floor_div = [](Wide a, Wide b) { return a / b - (a % b != 0 && a < 0 ? 1 : 0); };
  Wide first = -floor_div(-(target - bytes + 1 - hi), t[0].stride);
  Wide last = floor_div(target + bytes - 1 - lo, t[0].stride);
  if (first < t[0].lo) first = t[0].lo;
  if (last > t[0].hi) last = t[0].hi;
  Overlap all = Overlap::kNo;
  for (Wide i = first; i <= last; ++i) {
    if (--*steps < 0) return Overlap::kUnknown;
    const Overlap one = find(t + 1, n - 1, target - i * t[0].stride, bytes, other || i != 0, steps);
    if (one == Overlap::kYes) return one;
    if (one == Overlap::kUnknown) all = one;
  }
  return all;
}

inline void put(Term* t, int* n, Term x) {   // kept in falling order of strides
  int i = (*n)++;
  for (; i > 0 && t[i - 1].stride < x.stride; --i) t[i] = t[i - 1];
  t[i] = x;
}

constexpr int kSteps = 2000;   // looked at before the answer is "unknown"; views of a tensor take a few dozen

}  // namespace overlap_detail

// Do two rows of a set share a byte?
inline Overlap rows_overlap_themselves(const RowSet& a) {
  using namespace overlap_detail;
  Term t[3];
  int n = 0, steps = kSteps;
  for (int d = 0; d < 3; ++d) {
    if (a.n[d] == 1) continue;
    if (a.stride[d] == 0) return Overlap::kYes;
    put(t, &n, Term{a.stride[d], -(Wide)(a.n[d] - 1), a.n[d] - 1});
  }
  Wide reach = a.bytes;        // most often every stride reaches over all that lies inside it
  int inside = n;
  while (inside > 0 && t[inside - 1].stride >= reach) {
    --inside;
    reach += t[inside].hi * t[inside].stride;
  }
  if (inside == 0) return Overlap::kNo;
  return find(t, n, 0, a.bytes, false, &steps);
}

// Are they the same rows in the same places?
inline bool same_rows(const RowSet& a, const RowSet& b) {
  bool same = a.at == b.at && a.bytes == b.bytes;
  for (int d = 0; d < 3; ++d) same = same && a.n[d] == b.n[d] && (a.n[d] == 1 || a.stride[d] == b.stride[d]);
  return same;
}

// Does a row of one set share a byte with a row of the other (of rows as long)?
inline Overlap rows_overlap(const RowSet& a, const RowSet& b) {
  using namespace overlap_detail;
  Term t[6];
  int n = 0, steps = kSteps;
  bool pairs = true;           // dimensions with one stride make one term of both indexes
  for (int d = 0; d < 3; ++d) pairs = pairs && (a.n[d] == 1 || b.n[d] == 1 || a.stride[d] == b.stride[d]);
  Wide lo = 0, hi = 0;
  auto add = [&](Wide stride, Wide first, Wide last) {
    lo += first * stride;
    hi += last * stride;
    if (stride > 0 && first < last) put(t, &n, Term{stride, first, last});
  };
  for (int d = 0; d < 3; ++d) {
    if (pairs) {
      add(a.n[d] > 1 ? a.stride[d] : b.stride[d], -(Wide)(b.n[d] - 1), a.n[d] - 1);
    } else {
      add(a.stride[d], 0, a.n[d] - 1);
      add(b.stride[d], -(Wide)(b.n[d] - 1), 0);
    }
  }
  const Wide target = (Wide)b.at - (Wide)a.at;
  if (target - a.bytes >= hi || target + a.bytes <= lo) return Overlap::kNo;   // one lies behind the other
  return find(t, n, target, a.bytes, true, &steps);
}

}  // namespace lf
