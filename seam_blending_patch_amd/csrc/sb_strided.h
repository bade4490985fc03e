// sb_strided.h -- host-side checks of strided tensors: extents and strides in
// elements, the innermost run contiguous.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace sb {

constexpr int64_t kMaxExtent = (int64_t)1 << 31; // extents of a strided tensor
constexpr int64_t kMaxStride = (int64_t)1 << 40; // strides, in elements
constexpr int64_t kMaxSpan = (int64_t)1 << 52;   // elements from a tensor's first to its last

// Up to three outer axes, longest stride first, over runs of `run` elements;
// axes of extent 1 are dropped.
struct Strided {
  int n = 0;
  int64_t ext[3], str[3];
  int64_t run = 0;

  void add(int64_t extent, int64_t stride) {
    if (extent == 1) return;
    int k = n++;
    while (k > 0 && str[k - 1] < stride) {
      ext[k] = ext[k - 1];
      str[k] = str[k - 1];
      --k;
    }
    ext[k] = extent;
    str[k] = stride;
  }
  // elements from the first to the last of the axes from `level` on; kMaxSpan
  // where they are that many or more (an extent times a stride passes 64 bits)
  int64_t span(int level = 0) const {
    int64_t s = run;
    for (int k = level; k < n; ++k) {
      if (ext[k] > 1 && str[k] > (kMaxSpan - s) / (ext[k] - 1)) return kMaxSpan;
      s += (ext[k] - 1) * str[k];
    }
    return s;
  }
  // no element is reached by two indices
  bool distinct() const {
    for (int k = 0; k < n; ++k)
      if (str[k] < span(k + 1)) return false;
    return true;
  }
  bool same(const Strided &o) const {
    if (n != o.n || run != o.run) return false;
    for (int k = 0; k < n; ++k)
      if (ext[k] != o.ext[k] || str[k] != o.str[k]) return false;
    return true;
  }
};

// Whether a and b can share an element when b starts `off` elements after a.
// Exact for tensors whose axes from `level` on have the same strides (views of
// one packed buffer: the query and key heads of one projection); others are
// taken to overlap as soon as their spans do.
inline bool can_overlap(const Strided &a, const Strided &b, int64_t off, int level = 0) {
  if (off >= a.span(level) || -off >= b.span(level)) return false;
  if (level >= a.n || level >= b.n || a.str[level] != b.str[level]) return true;
  const int64_t s = a.str[level], la = a.span(level + 1), lb = b.span(level + 1);
  if (s < la || s < lb) return true;
  // b's index minus a's: only where the inner spans meet, at most three of them
  const int64_t lo = std::max<int64_t>(-(a.ext[level] - 1), -(off + lb) / s - 1);
  const int64_t hi = std::min<int64_t>(b.ext[level] - 1, (la - off) / s + 1);
  for (int64_t m = lo; m <= hi; ++m)
    if (can_overlap(a, b, off + m * s, level + 1)) return true;
  return false;
}

} // namespace sb
