// The cache positions that a tile of rows sees, on the device and on the host: plain
// arithmetic on what a batch's tables say, whatever they say.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace q3 {

// Positions that attention sees stay below it, so that sums of a span's end with a
// step do not pass 2^31.
constexpr int kMaxKey = 0x7FFFF000;

// One below the first position that a token at `position` sees.
__host__ __device__ __forceinline__ int below_window(int32_t window, int position) {
  const int64_t low = window ? (int64_t)position - window : -1;
  return low > -1 ? (int)low : -1;
}

struct Span {
  int lo, hi;   // hi == lo: nothing
};
// What tokens at positions first..last see between them of a table of `pages` pages
// of 1 << shift positions.  Where they see nothing the span is [0, 0): a window may
// begin far behind the table's end, up to 2^31, where no step can be added.
__host__ __device__ __forceinline__ Span span_between(int first, int last, int32_t window, int64_t pages, int shift) {
  const int64_t held = pages << shift;   // the host keeps `pages` to 2^31
  int64_t hi = (int64_t)last + 1;
  if (hi > held) hi = held;
  if (hi > kMaxKey) hi = kMaxKey;
  const int64_t lo = below_window(window, first) + 1;
  if (hi <= lo) return {0, 0};
  return {(int)lo, (int)hi};
}

// A span is walked in steps of `step` positions (a power of two) from here on.
__host__ __device__ __forceinline__ int first_of(const Span& span, int step) { return span.lo & ~(step - 1); }
__host__ __device__ __forceinline__ int steps_of(const Span& span, int step) {
  return (span.hi - first_of(span, step) + step - 1) / step;
}

}  // namespace q3
