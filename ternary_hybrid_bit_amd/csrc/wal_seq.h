// The cutting of an attention call into sequences: plain arithmetic, the same
// on the host (where it is tested) and in the kernels.
#pragma once

#include <stdint.h>

namespace wal {

// A sequence's part of a call.
struct Seq {
  int32_t first, rows, len, old;   // first query row, rows, tokens, tokens before the first row's own
};

constexpr int32_t between(int32_t x, int32_t low, int32_t high) { return x < low ? low : x > high ? high : x; }

// The sequence of query rows start .. end - 1 with len tokens in the cache (packed: its own rows), cut to the rows and
// tokens that there are whatever start, end and len hold.  n and max_new are at most 2^24, max_len 2^30.
constexpr Seq cut_seq(int32_t start, int32_t end, int32_t len, int32_t n, int32_t max_new, int32_t max_len, bool paged) {
  Seq q{};
  q.first = between(start, 0, n);
  const int32_t new_s = between(end, q.first, n) - q.first;   // both ends first: their difference may not fit
  q.rows = between(new_s, 0, max_new);
  q.len = between(paged ? len : new_s, 0, max_len);
  q.old = paged ? q.len - new_s : 0;
  return q;
}

}  // namespace wal
