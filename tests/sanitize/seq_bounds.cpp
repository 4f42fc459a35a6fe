// Driver of tests/test_attention_bounds.py: cut_seq over extreme and ordinary
// values, under UndefinedBehaviorSanitizer.  Prints the first case that leaves
// the rows or tokens of a call, or differs from the definition.
#include <cstdio>
#include <initializer_list>

#include "../../ternary_hybrid_bit_amd/csrc/wal_seq.h"

int main() {
  const int32_t lo = INT32_MIN, hi = INT32_MAX;
  long cases = 0;
  for (int32_t n : {0, 1, 8, 1 << 24})
    for (int32_t max_new : {0, 1, 4, 1 << 24})
      for (int32_t max_len : {0, 1, 100, 1 << 30})
        for (int32_t start : {lo, lo + 1, -(1 << 24), -9, -1, 0, 1, 3, 5, 8, 9, 1 << 24, (1 << 24) + 1, hi - 1, hi})
          for (int32_t end : {lo, lo + 1, lo + 7, -(1 << 24), -9, -2, -1, 0, 1, 4, 5, 8, 9, 1 << 24, hi - 1, hi})
            for (int32_t len : {lo, -1, 0, 1, 60, 100, 1 << 24, 1 << 30, hi})
              for (bool paged : {false, true}) {
                const wal::Seq q = wal::cut_seq(start, end, len, n, max_new, max_len, paged);
                ++cases;
                bool ok = q.first >= 0 && q.rows >= 0 && q.rows <= max_new && (int64_t)q.first + q.rows <= n;
                ok = ok && q.len >= 0 && q.len <= max_len;
                if (!paged) ok = ok && q.old == 0 && (int64_t)q.first + q.len <= n;
                // no row sees a token past the last
                if (paged && q.rows) ok = ok && (int64_t)q.old + q.rows <= q.len;
                if (ok && 0 <= start && start <= end && end <= n && end - start <= max_new && 0 <= len && len <= max_len) {
                  const int32_t tokens = paged ? len : end - start;
                  if (paged || tokens <= max_len)
                    ok = q.first == start && q.rows == end - start && q.len == tokens && q.old == (paged ? len - (end - start) : 0);
                }
                if (!ok) {
                  std::printf("start %d end %d len %d n %d max_new %d max_len %d paged %d -> first %d rows %d len %d old %d\n",
                              start, end, len, n, max_new, max_len, paged, q.first, q.rows, q.len, q.old);
                  return 1;
                }
              }
  std::printf("%ld cases\n", cases);
  return 0;
}
