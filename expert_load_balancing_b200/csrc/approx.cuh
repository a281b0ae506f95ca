// approx.cuh -- the hardware's fast exponential and reciprocal, for results
// that are rounded to 8 or 16 bits or enter sums of many rows.
#pragma once

namespace kolibri {

// 2^x and 1 / x by the hardware's approximations, subnormal results flushed:
// about 2^-22 relative each.
constexpr float kLog2e = 1.44269504088896340736f;
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

}  // namespace kolibri
