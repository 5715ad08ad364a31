// tbe_overlap.cuh -- whether arguments share memory (host): exact where rows
// of one tensor lie between those of another, as slices of one buffer do.
#pragma once

#include <algorithm>
#include <cstdint>

namespace tbe {

// Rows of `width` bytes at p + o outer_step + i inner_step, all rows of an o
// before those of the next.
struct Region {
  intptr_t p;
  int64_t width;
  int64_t outer, outer_step;
  int64_t inner, inner_step;

  int64_t inner_span() const { return (inner - 1) * inner_step + width; }
  intptr_t end() const { return p + (outer - 1) * outer_step + inner_span(); }
  bool empty() const { return p == 0 || width <= 0 || outer <= 0 || inner <= 0; }
};
inline Region bytes_of(const void* p, int64_t bytes) { return {(intptr_t)p, bytes, 1, 0, 1, 0}; }
inline Region rows_of(const void* p, int64_t rows, int64_t stride, int64_t width) {
  return {(intptr_t)p, width, rows, stride, 1, 0};
}

// Whether [x, x + width) holds a byte of one of r's rows: the first row that
// ends behind x is the only one to look at.
inline bool meets(const Region& r, intptr_t x, int64_t width) {
  const int64_t at = x - r.p;
  int64_t o = 0, i = 0;
  if (r.outer > 1 && at >= r.inner_span()) o = (at - r.inner_span()) / r.outer_step + 1;
  if (o >= r.outer || (r.outer == 1 && at >= r.inner_span())) return false;
  const int64_t in = at - o * r.outer_step;
  if (r.inner > 1 && in >= r.width) i = (in - r.width) / r.inner_step + 1;
  return o * r.outer_step + i * r.inner_step < at + width;
}

// Whether a and b share a byte.  With the same outer step, or where one has a
// single outer row, this is exact; else regions whose ranges meet count as
// sharing.
inline bool share(Region a, Region b) {
  if (a.empty() || b.empty() || a.end() <= b.p || b.end() <= a.p) return false;
  if (b.outer == 1) std::swap(a, b);
  if (a.outer > 1) {
    if (a.outer_step != b.outer_step) return true;
    // a's rows of all o against b is a's first against all of b's places relative to them
    b.p -= (a.outer - 1) * a.outer_step;
    b.outer += a.outer - 1;
  }
  for (int64_t i = 0; i < a.inner; ++i)
    if (meets(b, a.p + i * a.inner_step, a.width)) return true;
  return false;
}

}  // namespace tbe
