// Host-only harness for tests/test_place.py: row_place over every combination of
// words at the ends of 32 bits and around a page, beside the definition in 128 bits.
// Prints the number of combinations and of places found, or the first that differs.
#include <cstdio>

#include "place.h"

int main() {
  const int32_t words[] = {INT_MIN, INT_MIN + 1, -(1 << 30), -17, -1, 0, 1, 2, 3, 17, 40, 1 << 27, 1 << 30, INT_MAX - 1, INT_MAX};
  const int32_t lens[] = {INT_MIN, -16, -1, 0, 1, 8, 16, 17, INT_MAX};
  const int32_t rows[] = {0, 1, 2, 16, 39, 1 << 27, INT_MAX - 1, INT_MAX};
  using wide = __int128;
  long long n = 0, found = 0;
  for (int32_t row : rows)
    for (int32_t a0 : words)
      for (int32_t a1 : words)
        for (int32_t p0 : words)
          for (int32_t p1 : words)
            for (int32_t end : words)
              for (int32_t last : lens) {
                const wide kv = ((wide)p1 - p0 - 1) * 16 + last, fresh = (wide)a1 - a0;
                const bool want = 0 <= a0 && a0 <= row && row < a1 && 0 <= p0 && p0 < p1 && p1 <= end && 1 <= last &&
                                  last <= 16 && fresh <= kv && kv <= INT_MAX;
                int32_t pos = -1, at = -1;
                const bool got = daa::row_place(row, a0, a1, p0, p1, end, last, pos, at);
                const wide w = kv - fresh + row - a0;
                if (got != want || (got && (pos != w || at != p0 + w / 16 || at < p0 || at >= p1))) {
                  std::printf("row %d of [%d, %d), pages [%d, %d) of %d, last %d: %d, position %d, page %d\n", row, a0,
                              a1, p0, p1, end, last, got, pos, at);
                  return 1;
                }
                ++n;
                found += got;
              }
  std::printf("%lld %lld\n", n, found);
  return 0;
}
