// Sums in twice fp32 (fp64 arithmetic is slow on this GPU: its latency shows in short kernels).
#pragma once

#include <cfloat>

namespace fo {

// A number as the sum of two fp32 values, |lo| at most half a step of hi (sums of error-free
// transformations, Knuth).  Infinite or NaN: as the plain sum is, with lo = 0.
struct __align__(8) Wide {
  float hi, lo;
};
__device__ __forceinline__ Wide wide(float v) { return Wide{v, 0.f}; }
__device__ __forceinline__ Wide plus(const Wide& a, const Wide& b) {
  const float s = a.hi + b.hi, t = s - a.hi;
  const float lo = ((a.hi - (s - t)) + (b.hi - t)) + (a.lo + b.lo), hi = s + lo;
  return fabsf(s) <= FLT_MAX ? Wide{hi, lo - (hi - s)} : Wide{s, 0.f};
}
// Over a warp, in every lane
__device__ __forceinline__ Wide warp_sum(Wide v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    v = plus(v, Wide{__shfl_xor_sync(0xffffffffu, v.hi, o), __shfl_xor_sync(0xffffffffu, v.lo, o)});
  return v;
}

}  // namespace fo
