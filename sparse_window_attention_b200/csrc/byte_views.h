// Whether two strided views of memory have a byte in common (host only).
#pragma once

#include <stdint.h>

#include <algorithm>

namespace basa {

// A view: rows of `row` bytes at base plus every sum of its axes' steps (in bytes, >= 0).
struct ByteView {
  uintptr_t base;
  int64_t row, step[3], ext[3];
  uintptr_t end() const {
    return base + uintptr_t(row + step[0] * (ext[0] - 1) + step[1] * (ext[1] - 1) + step[2] * (ext[2] - 1));
  }
};

// Two rows meet where the distance of their starts, delta + the sum of step times entry over
// all axes (the first view's counted up, the second's down), is less than a row. Steps of the
// same size are one term. The terms are gone through from the largest; what the smaller ones
// can reach leaves few entries of each, in slices of one buffer one or two. kMeetTries bounds
// the search, and what it leaves open counts as met.
constexpr int kMeetTries = 4096;
struct Meet {
  int64_t step[6], lo[6], hi[6], rest_lo[7], rest_hi[7], row_a, row_b;
  int n = 0, tries = 0;

  void add(int64_t s, int64_t a, int64_t b) {
    if (s == 0 || a == b) return;
    int at = 0;
    while (at < n && step[at] > s) ++at;
    if (at == n || step[at] != s) {
      for (int i = n++; i > at; --i) step[i] = step[i - 1], lo[i] = lo[i - 1], hi[i] = hi[i - 1];
      step[at] = s;
      lo[at] = hi[at] = 0;
    }
    lo[at] += a;
    hi[at] += b;
  }
  static int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b < 0); }

  // delta: start of the first view's row less the second's; they meet in (-row_a, row_b)
  bool from(int i, int64_t delta) {
    if (++tries > kMeetTries) return true;
    if (i == n) return -row_a < delta && delta < row_b;
    const int64_t first = std::max(lo[i], -floor_div(delta + rest_hi[i + 1] + row_a - 1, step[i]));
    const int64_t last = std::min(hi[i], floor_div(row_b - 1 - rest_lo[i + 1] - delta, step[i]));
    for (int64_t x = first; x <= last; ++x)
      if (from(i + 1, delta + x * step[i])) return true;
    return false;
  }
};

inline bool views_meet(const ByteView &a, const ByteView &b) {
  if (a.base >= b.end() || b.base >= a.end()) return false;
  Meet m;
  m.row_a = a.row;
  m.row_b = b.row;
  for (int k = 0; k < 3; ++k) {
    m.add(a.step[k], 0, a.ext[k] - 1);
    m.add(b.step[k], 1 - b.ext[k], 0);
  }
  m.rest_lo[m.n] = m.rest_hi[m.n] = 0;
  for (int i = m.n; i-- > 0;) {
    m.rest_lo[i] = m.rest_lo[i + 1] + m.step[i] * m.lo[i];
    m.rest_hi[i] = m.rest_hi[i + 1] + m.step[i] * m.hi[i];
  }
  return m.from(0, int64_t(a.base - b.base));
}

}  // namespace basa
