// line.h -- a line of places of work that the thread blocks of a launch divide
// evenly (few-token attention, scores of few query rows).
//
// Places are unsigned 32-bit numbers: a 64-bit division takes some 500 clocks,
// and several stand between a launch and its first load.  The lengths that the
// line is made from are data, and contradictory ones (sequences that overlap)
// can add up to more places than the storage has tokens for.  Sums therefore
// stop at kLineOver instead of wrapping, which would give one place to two
// owners, or to none.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define BSA_LINE __host__ __device__ __forceinline__
#else
#define BSA_LINE inline
#endif

namespace bsa {

constexpr uint32_t kLineOver = 0xffffffffu;  // this many places, or more

BSA_LINE uint32_t line_add(uint32_t a, uint32_t b) {
  const uint32_t s = a + b;
  return s < a ? kLineOver : s;
}
BSA_LINE uint32_t line_places(uint64_t n) { return n < kLineOver ? uint32_t(n) : kLineOver; }

// index rows: up to 2^30 of them exist (the host refuses more), so sums stop there
constexpr uint32_t kRowsMost = uint32_t(1) << 30;
BSA_LINE uint32_t rows_add(uint32_t a, uint32_t b) {  // a, b <= kRowsMost
  return a + b < kRowsMost ? a + b : kRowsMost;
}

// part c of a line that is cut into `parts`: places [lo, hi); the first
// `extra` parts have each + 1 places, the others `each`
struct LinePart {
  uint32_t lo, hi, each, extra;
};
BSA_LINE LinePart line_part(uint32_t total, uint32_t parts, uint32_t c) {
  LinePart p;
  p.each = total / parts;
  p.extra = total % parts;
  p.lo = c * p.each + (c < p.extra ? c : p.extra);
  p.hi = p.lo + p.each + (c < p.extra ? 1u : 0u);
  return p;
}
// the part that holds place x, never past the last one
BSA_LINE uint32_t line_owner(uint32_t each, uint32_t extra, uint32_t parts, uint32_t x) {
  const uint32_t big = extra * (each + 1);
  const uint32_t c = x < big ? x / (each + 1) : each ? extra + (x - big) / each : parts;
  return c < parts ? c : parts - 1;
}

}  // namespace bsa
