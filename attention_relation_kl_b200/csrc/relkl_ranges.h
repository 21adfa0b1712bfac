// The arrays of AdamW tables by address: none that is written may overlap
// another.  Plain C++: the library and the binding's marshalling module share it.
#pragma once
#include <algorithm>
#include <cstdint>

#include "../../include/relkl.h"

namespace relkl {

struct Range {
  uintptr_t begin, end;
  bool written;
};

constexpr int kAdamwRanges = 7;   // arrays of one tensor, at most

// Appends a tensor's arrays to r; returns how many.
inline int adamw_ranges(const relkl_adamw_tensor& t, bool bits8, Range* r) {
  int n = 0;
  auto add = [&](const void* x, int64_t bytes, bool written) {
    if (!x || bytes == 0) return;
    const uintptr_t b = reinterpret_cast<uintptr_t>(x);
    r[n++] = Range{b, b + static_cast<uintptr_t>(bytes), written};
  };
  const int64_t blocks = (t.n + 255) / 256, state = bits8 ? 1 : 4;
  add(t.grad, t.n * (t.grad_dtype == RELKL_BF16 ? 2 : 4), false);
  add(t.param, t.n * (t.param_dtype == RELKL_BF16 ? 2 : 4), true);
  add(t.copy, t.n * 2, true);
  add(t.m, t.n * state, true);
  add(t.v, t.n * state, true);
  add(t.m_scale, blocks * 4, true);
  add(t.v_scale, blocks * 4, true);
  return n;
}

// Whether a written array overlaps another; sorts them.
inline bool overlaps(Range* r, int64_t n) {
  std::sort(r, r + n, [](const Range& x, const Range& y) { return x.begin < y.begin; });
  uintptr_t read = 0, written = 0;   // the ends so far
  for (int64_t i = 0; i < n; ++i) {
    if (r[i].begin < written || (r[i].written && r[i].begin < read)) return true;
    uintptr_t& end = r[i].written ? written : read;
    end = r[i].end > end ? r[i].end : end;
  }
  return false;
}

}  // namespace relkl
