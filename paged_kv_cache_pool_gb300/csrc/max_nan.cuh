// The maximum that the joins of partial states take over the states' LSE.
#pragma once

namespace gk {

// the larger of two numbers; NaN where one of them is (fmaxf drops it)
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

}  // namespace gk
