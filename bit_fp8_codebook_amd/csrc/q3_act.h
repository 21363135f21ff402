// The gate's activation and its derivative (fp32).
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/q3_block.h"

namespace q3 {

// Both activations have the form z / (1 + e^-v): silu with v = z, the tanh form
// of GELU with v = 2 sqrt(2/pi) (z + 0.044715 z^3), since 1/2 (1 + tanh(v/2)) =
// 1 / (1 + e^-v).  No cancellation for negative z; a finite z far enough out for
// e^-v to overflow gives -0 (z = -inf itself is NaN, as z times 0 is).
constexpr float kGelu2 = 1.5957691216057308f;   // 2 sqrt(2/pi)
constexpr float kGelu3 = 0.044715f;

__device__ __forceinline__ float act_value(int act, float z) {
  const float v = act == Q3_ACT_SILU ? z : kGelu2 * (z + kGelu3 * z * z * z);
  return z / (1.0f + expf(-v));
}

// act(z) and act'(z) = p + z p (1 - p) v'(z), p = 1 / (1 + e^-v).
__device__ __forceinline__ void act_both(int act, float z, float& a, float& da) {
  const bool silu = act == Q3_ACT_SILU;
  const float v = silu ? z : kGelu2 * (z + kGelu3 * z * z * z);
  const float dv = silu ? 1.0f : kGelu2 * (1.0f + 3.0f * kGelu3 * z * z);
  const float p = 1.0f / (1.0f + expf(-v));
  const float q = p * (1.0f - p);
  a = z * p;
  da = p + (q > 0.f ? z * q * dv : 0.f);   // far out z dv may overflow where q is 0
}

}  // namespace q3
