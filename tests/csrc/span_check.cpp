// Compares Strided::span of sb_strided.h with the exact count in 128 bits, over
// extents and strides up to their limits: exact below kMaxSpan, at least
// kMaxSpan otherwise (built with the signed-overflow sanitizer).
#include "sb_strided.h"

#include <cstdio>
#include <random>

int main() {
  std::mt19937_64 gen(1);
  auto log_uniform = [&](int bits) { return (int64_t)(gen() >> 1) >> (63 - gen() % (bits + 1)); };
  long cases = 0, wide = 0;
  for (int n = 0; n < 200000; ++n) {
    sb::Strided s;
    s.run = 1 + log_uniform(28);
    __int128 exact = s.run;
    const int axes = 1 + (int)(gen() % 3);
    for (int k = 0; k < axes; ++k) {
      const int64_t extent = 1 + log_uniform(31), stride = log_uniform(40);
      if (extent > sb::kMaxExtent || stride >= sb::kMaxStride) return std::printf("bad case\n"), 1;
      s.add(extent, stride);
      exact += (__int128)(extent - 1) * stride;
    }
    const int64_t got = s.span();
    if (exact >= sb::kMaxSpan ? got < sb::kMaxSpan : got != (int64_t)exact)
      return std::printf("case %d: span %lld\n", n, (long long)got), 1;
    wide += exact >= sb::kMaxSpan;
    ++cases;
  }
  // two tensors that start inside one another, of a span past 64 bits
  sb::Strided s;
  s.run = 64;
  s.add(((int64_t)1 << 24) + 1, sb::kMaxStride - 1);
  if (s.span() < sb::kMaxSpan) return std::printf("2^64 elements: span %lld\n", (long long)s.span()), 1;
  if (!sb::can_overlap(s, s, 0)) return std::printf("a tensor taken not to overlap itself\n"), 1;
  std::printf("%ld cases, %ld wide\n", cases, wide);
  return 0;
}
