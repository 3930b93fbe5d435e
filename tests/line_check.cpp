// The arithmetic by which thread blocks divide a line of work, on the host:
// parts cover the line once, every place has the owner that holds it, no owner
// lies outside the grid, and sums of contradictory lengths stop instead of wrapping.
#include <cstdio>
#include <initializer_list>

#include "line.h"

using namespace bsa;

#define CHECK(c)                                        \
  do {                                                  \
    if (!(c)) {                                         \
      std::fprintf(stderr, "line %d: %s\n", __LINE__, #c); \
      return 1;                                         \
    }                                                   \
  } while (0)

int main() {
  // 656 sequences of 65536 tokens (64 heads over 8, tiles of 128 rows) before
  // 127999 tokens, as cu_seqlens 0, T, 0, T, ... makes them
  const uint32_t work = line_places(uint64_t(65536 * 8 / 128) * 8 * ((127999 + 127) / 128));
  uint32_t sum = 0, wrapped = 0;
  bool over = false;
  for (int b = 0; b < 656; ++b) {
    const uint32_t before = sum;
    sum = line_add(sum, work);
    wrapped += work;
    CHECK(sum >= before);
    over = over || sum == kLineOver;
  }
  CHECK(uint64_t(work) * 656 > kLineOver && wrapped < sum && over && sum == kLineOver);
  CHECK(line_add(kLineOver, 0) == kLineOver && line_add(kLineOver, kLineOver) == kLineOver);
  CHECK(line_add(kLineOver - 1, 0) == kLineOver - 1 && line_add(kLineOver - 1, 1) == kLineOver);
  CHECK(line_places(uint64_t(1) << 40) == kLineOver && line_places(kLineOver - 1) == kLineOver - 1);
  CHECK(rows_add(kRowsMost, kRowsMost) == kRowsMost && rows_add(kRowsMost - 1, 0) == kRowsMost - 1);

  for (uint32_t parts : {1u, 2u, 36u, 148u, 296u, 592u})
    for (uint32_t total : {0u, 1u, 35u, 36u, 147u, 148u, 149u, 1000u, 4096u * 8u, 4000000000u, kLineOver - 1}) {
      uint32_t at = 0;
      for (uint32_t c = 0; c < parts; ++c) {
        const LinePart p = line_part(total, parts, c);
        CHECK(p.lo == at && p.hi >= p.lo);
        at = p.hi;
        if (p.lo == p.hi) continue;
        for (uint32_t x : {p.lo, p.lo + (p.hi - p.lo) / 2, p.hi - 1}) CHECK(line_owner(p.each, p.extra, parts, x) == c);
      }
      CHECK(at == total);
      // places past the line, as a unit that does not end on it would ask for
      const LinePart p = line_part(total, parts, 0);
      for (uint32_t past : {0u, 1u, 1000u, 100000u})
        if (total <= kLineOver - past) CHECK(line_owner(p.each, p.extra, parts, total + past) < parts);
    }
  std::puts("ok");
  return 0;
}
