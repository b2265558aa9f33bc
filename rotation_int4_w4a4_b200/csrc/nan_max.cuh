// Maxima in which NaN stays (fmaxf drops it): of the magnitudes that a quantisation scale is taken from, so that a row or
// head that holds a NaN gets a scale that is one.
#pragma once

namespace pq {

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

}  // namespace pq
