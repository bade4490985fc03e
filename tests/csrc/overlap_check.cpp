// Compares can_overlap and distinct of sb_strided.h with a count of every
// element, on small random strided tensors.  Prints the number of cases and
// exits with 1 on the first unsound answer; "told apart" counts the pairs of
// interleaved but disjoint tensors that are recognised as such.
#include "sb_strided.h"

#include <cstdio>
#include <cstdlib>
#include <random>
#include <set>

struct T {
  int64_t ext[3], str[3], run;
};

static sb::Strided describe(const T &t) {
  sb::Strided s;
  s.run = t.run;
  for (int k = 0; k < 3; ++k) s.add(t.ext[k], t.str[k]);
  return s;
}

static bool elements(const T &t, int64_t at, std::set<int64_t> &out) {
  bool once = true;
  for (int64_t a = 0; a < t.ext[0]; ++a)
    for (int64_t b = 0; b < t.ext[1]; ++b)
      for (int64_t c = 0; c < t.ext[2]; ++c)
        for (int64_t r = 0; r < t.run; ++r)
          once = out.insert(at + a * t.str[0] + b * t.str[1] + c * t.str[2] + r).second && once;
  return once;
}

int main() {
  std::mt19937 gen(1);
  auto pick = [&](int lo, int hi) { return (int64_t)std::uniform_int_distribution<int>(lo, hi)(gen); };
  long cases = 0, disjoint = 0, told = 0;
  for (int n = 0; n < 60000; ++n) {
    T a, b;
    a.run = pick(1, 4);
    b.run = pick(0, 1) ? a.run : pick(1, 4);
    const bool packed = pick(0, 3) > 0; // views of one buffer: the same strides
    for (int k = 0; k < 3; ++k) {
      a.ext[k] = pick(1, 4);
      b.ext[k] = pick(0, 1) ? a.ext[k] : pick(1, 4);
      a.str[k] = pick(0, 40);
      b.str[k] = packed ? a.str[k] : pick(0, 40);
    }
    const int64_t off = pick(-60, 60);
    std::set<int64_t> ea, eb;
    const bool once = elements(a, 0, ea);
    elements(b, off, eb);
    bool shared = false;
    for (int64_t e : eb) shared = shared || ea.count(e);
    const sb::Strided da = describe(a), db = describe(b);
    const bool said = sb::can_overlap(da, db, off);
    if (shared && !said) return std::printf("missed an overlap in case %d\n", n), 1;
    if (!once && da.distinct()) return std::printf("missed a repeated element in case %d\n", n), 1;
    if (!said) ++told;
    if (!shared) ++disjoint;
    ++cases;
  }
  // the query and key heads of one projection [B, T, q + 2 k, D], both orders
  const int64_t B = 2, L = 6, q = 4, k = 2, D = 8, row = (q + 2 * k) * D;
  const T tq{{B, L, q}, {L * row, row, D}, D}, tk{{B, L, k}, {L * row, row, D}, D};
  if (sb::can_overlap(describe(tq), describe(tk), q * D) || sb::can_overlap(describe(tk), describe(tq), -q * D))
    return std::printf("query and key heads of one projection taken to overlap\n"), 1;
  if (!sb::can_overlap(describe(tq), describe(tk), (q - 1) * D)) return std::printf("a shared head missed\n"), 1;
  const T one{{1, L, 1}, {0, row, 0}, D}; // a single key head beside them
  if (!describe(one).distinct() || !describe(tq).distinct()) return std::printf("distinct tensors refused\n"), 1;
  std::printf("%ld cases, %ld disjoint, %ld told apart\n", cases, disjoint, told);
  return 0;
}
