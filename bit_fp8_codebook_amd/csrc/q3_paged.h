// Device-side reading of a batch's tables (gfx950 only).  Nothing that stands in
// them is trusted: whatever they hold, every address formed here is inside the
// tables, and a place that is not in the cache says so.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q3_internal.h"

namespace q3 {

// The sequence of a row, or b.sequences where it belongs to none: the number of
// entries q_start[1..] that are at most `row`.  One wave asks 64 entries at a
// time, so up to 63 sequences cost one load and up to 4095 two.
__device__ __forceinline__ int find_sequence(const BatchView& b, int row, int lane) {
  int lo = 0, hi = b.sequences;   // the count is in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + 63) / 64;
    const int at = lo + (lane + 1) * step - 1;   // entry 1 + at is asked
    const bool below = at < hi && b.q_start[1 + (at < hi ? at : 0)] <= row;
    const int c = __popcll(__ballot(below));
    const int first = lo + c * step;
    const int last = lo + (c + 1) * step - 1;
    lo = first < hi ? first : hi;
    hi = last < hi ? last : hi;
  }
  return lo < b.sequences && b.q_start[lo] <= row ? lo : b.sequences;
}

// The page of position p of a sequence (its row of the table), or -1.
__device__ __forceinline__ int64_t find_page(const BatchView& b, const CacheView& c, int sequence, int64_t p) {
  if (p < 0 || (p >> c.shift) >= b.table_pages) return -1;
  const int64_t page = b.table[(int64_t)sequence * b.ld_table + (p >> c.shift)];
  return page >= 0 && page < c.pages ? page : -1;
}

}  // namespace q3
