// Whether two tensors [rows][heads][dim] of one element type, each with strides of its own, share memory (abi.hip, bind.cpp).
#pragma once

#include <algorithm>
#include <cstdint>

namespace tc {

struct HeadsAt {
  const void* p;
  int64_t row, head;  // elements between rows and between heads, at least 0
};

enum class Overlap { none, some, unknown };

namespace overlap_detail {

typedef __int128 Wide;
struct Span {
  Wide step, most;  // multiples 0 to `most` of step
};

inline Wide floor_div(Wide a, Wide b) { return a >= 0 ? a / b : -((b - 1 - a) / b); }

// Whether a sum of a multiple of each step lies in [lo, hi]. From the largest step on: what the smaller ones reach leaves few
// multiples where rows and heads are nested, as they mostly are; `tries` bounds the others.
inline Overlap reaches(const Span* s, int n, Wide lo, Wide hi, int& tries) {
  if (hi < 0) return Overlap::none;
  if (n == 0) return lo <= 0 ? Overlap::some : Overlap::none;
  Wide rest = 0;
  for (int i = 1; i < n; ++i) rest += s[i].step * s[i].most;
  const Wide first = std::max<Wide>(0, floor_div(lo - rest + s->step - 1, s->step)), last = std::min(s->most, hi / s->step);
  for (Wide i = first; i <= last; ++i) {
    if (--tries < 0) return Overlap::unknown;
    const Overlap r = reaches(s + 1, n - 1, lo - i * s->step, hi - i * s->step, tries);
    if (r != Overlap::none) return r;
  }
  return Overlap::none;
}

}  // namespace overlap_detail

// Elements r x.row + h x.head + c of x and r' y.row + h' y.head + c' of y. An exact answer but for strides whose multiples
// interleave more than 2^18 times without meeting.
inline Overlap overlap(const HeadsAt& x, const HeadsAt& y, int64_t rows, int64_t heads, int64_t dim, int64_t size) {
  using namespace overlap_detail;
  const Wide x_reach = (Wide)(rows - 1) * x.row + (Wide)(heads - 1) * x.head, y_reach = (Wide)(rows - 1) * y.row + (Wide)(heads - 1) * y.head;
  const Wide apart = (Wide)(uintptr_t)y.p - (Wide)(uintptr_t)x.p;  // bytes
  if (apart >= (x_reach + dim) * size || -apart >= (y_reach + dim) * size) return Overlap::none;
  // x's place less y's, in elements, within less than `dim` of `apart`; y's multiples are counted from their ends, so that all add up
  Span s[4];
  int n = 0;
  const Span all[4] = {{x.row, rows - 1}, {x.head, heads - 1}, {y.row, rows - 1}, {y.head, heads - 1}};
  for (const Span& v : all) {
    if (v.step == 0 || v.most == 0) continue;
    int i = 0;
    while (i < n && s[i].step != v.step) ++i;
    if (i < n) s[i].most += v.most;
    else s[n++] = v;
  }
  std::sort(s, s + n, [](const Span& a, const Span& b) { return a.step > b.step; });
  int tries = 1 << 18;
  return reaches(s, n, floor_div(apart - (Wide)dim * size, size) + 1 + y_reach, floor_div(apart + (Wide)dim * size - 1, size) + y_reach, tries);
}

}  // namespace tc
