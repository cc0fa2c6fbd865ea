// Which queries and which cached tokens a sequence of an attention call has.
// Plain C++, for the kernels (constexpr functions are device functions too)
// and for the host's tests.
#pragma once

#include <stdint.h>

namespace qamw {

// A sequence's queries and cached tokens, whatever the arrays hold: queries
// stay inside [0, T), tokens inside the page table.
struct Sequence {
  int64_t first;                                   // its first query
  int n, length;
};
// queries [s0, s1) of T (at most 2^30), len tokens cached of the `most` (at
// most 2^30) that the table can name
constexpr Sequence clamped_sequence(int64_t s0, int64_t s1, int64_t T, int64_t len, int64_t most) {
  // in 64 bits as far as the clamps: the entries are any 32-bit numbers, their differences are not
  const int64_t first = s0 < 0 ? 0 : s0 > T ? T : s0, end = s1 < first ? first : s1 > T ? T : s1;
  return {first, (int)(end - first), (int)(len < 0 ? 0 : len > most ? most : len)};
}

}  // namespace qamw
