// Whether two strided views share memory: an output whose rows or heads share elements, or that
// shares them with an input that other blocks still read, would come out by chance.
#pragma once

#include <algorithm>
#include <cstdint>

namespace qs {
namespace views {

// Runs of `bytes` bytes at p + sum of i_d * dim[d].stride, 0 <= i_d < dim[d].size; strides in
// bytes, not negative.
struct View {
  const void* p;
  int64_t bytes;
  struct {
    int64_t size, stride;
  } dim[3];
};

inline View flat(const void* p, int64_t bytes) { return {p, bytes, {{1, 0}, {1, 0}, {1, 0}}}; }

// The search for whole numbers c_j in [lo_j, hi_j] whose sum of c_j * stride_j lies in a range:
// largest stride first, where the others' reach leaves few values to try.  Views of one buffer with
// rows, heads and elements inside one another take a few steps.
struct Search {
  struct Term {
    int64_t stride, lo, hi;
  } term[6];
  int n = 0;
  int64_t least[7], most[7];  // reach of the terms from j on
  int steps = 1 << 14;        // then the answer is yes: such views are refused

  void add(int64_t stride, int64_t lo, int64_t hi) {
    if (lo == hi) return;  // sizes of 1: always 0
    for (int j = 0; j < n; ++j)
      if (term[j].stride == stride) {
        term[j].lo += lo, term[j].hi += hi;
        return;
      }
    term[n++] = {stride, lo, hi};
  }
  void close() {
    std::sort(term, term + n, [](const Term& a, const Term& b) { return a.stride > b.stride; });
    least[n] = most[n] = 0;
    for (int j = n - 1; j >= 0; --j) {
      least[j] = least[j + 1] + term[j].lo * term[j].stride;
      most[j] = most[j + 1] + term[j].hi * term[j].stride;
    }
  }
  static int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b != 0 && a < 0); }
  // other: whether the c_j so far are not all 0 (or need not be)
  bool find(int j, int64_t from, int64_t to, bool other) {
    if (j == n) return other && from <= 0 && 0 <= to;
    if (--steps < 0) return true;
    const Term& t = term[j];
    if (t.stride == 0) return find(j + 1, from, to, true);  // any c_j, one that is not 0 among them
    const int64_t lo = std::max(t.lo, -floor_div(most[j + 1] - from, t.stride));
    const int64_t hi = std::min(t.hi, floor_div(to - least[j + 1], t.stride));
    for (int64_t c = lo; c <= hi; ++c) {
      if (find(j + 1, from - c * t.stride, to - c * t.stride, other || c != 0)) return true;
      if (steps < 0) return true;
    }
    return false;
  }
};

inline int64_t span(const View& v) {
  int64_t s = v.bytes;
  for (const auto& d : v.dim) s += (d.size - 1) * d.stride;
  return s;
}

inline bool overlap(const View& a, const View& b) {
  const int64_t pa = reinterpret_cast<int64_t>(a.p), pb = reinterpret_cast<int64_t>(b.p);
  if (pa + span(a) <= pb || pb + span(b) <= pa) return false;
  Search s;
  for (int d = 0; d < 3; ++d) {
    s.add(a.dim[d].stride, -(a.dim[d].size - 1), 0);
    s.add(b.dim[d].stride, 0, b.dim[d].size - 1);
  }
  s.close();
  // a run of b begins less than a run of a behind one of a's, or less than one of its own before it
  return s.find(0, 1 - b.bytes - (pb - pa), a.bytes - 1 - (pb - pa), true);
}

inline bool overlaps_itself(const View& v) {
  Search s;
  int terms = 0;
  for (const auto& d : v.dim) {
    terms += d.size > 1;
    s.add(d.stride, -(d.size - 1), d.size - 1);
  }
  if (s.n < terms) return true;  // two dimensions of one stride
  s.close();
  return s.find(0, 1 - v.bytes, v.bytes - 1, false);
}

inline bool same(const View& a, const View& b) {
  if (a.p != b.p || a.bytes != b.bytes) return false;
  for (int d = 0; d < 3; ++d)
    if (a.dim[d].size != b.dim[d].size || (a.dim[d].size > 1 && a.dim[d].stride != b.dim[d].stride))
      return false;
  return true;
}

}  // namespace views
}  // namespace qs
