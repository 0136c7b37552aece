// fp64 functions for kernels where the general ones' length is what a wave waits for (not part of the C
// interface).
#pragma once

#include "moe_internal.h"

namespace moe {

// e^x in fp64 for x from -1100 (0) to 700 (1e304), clamped there; NaN stays NaN.  Reduction by n ln 2 in
// two parts and the Taylor series to the 13th power on |r| <= ln 2 / 2 (rest 4e-18): 23 operations
// against some 60 of the general function, which a wave that has little to do waits for one by one.
__device__ __forceinline__ double exp_clamped(double x) {
  x = x < -1100.0 ? -1100.0 : x > 700.0 ? 700.0 : x;
  const double n = rint(x * 1.4426950408889634);
  double r = fma(n, -0.6931471805599453, x);
  r = fma(n, -2.3190468138462996e-17, r);
  double p = 1.0 / 6227020800.0;
  constexpr double kInverse[] = {1.0 / 479001600.0, 1.0 / 39916800.0, 1.0 / 3628800.0, 1.0 / 362880.0,
                                 1.0 / 40320.0,     1.0 / 5040.0,     1.0 / 720.0,     1.0 / 120.0,
                                 1.0 / 24.0,        1.0 / 6.0,        0.5,             1.0,
                                 1.0};
#pragma unroll
  for (int i = 0; i < 13; ++i) p = fma(p, r, kInverse[i]);
  return ldexp(p, (int)n);
}
// 1 / d for finite d >= 1 (or NaN): two steps of Newton's from the instruction's estimate
__device__ __forceinline__ double reciprocal(double d) {
  double r = __builtin_amdgcn_rcp(d);
  r = fma(r, fma(-d, r, 1.0), r);
  return fma(r, fma(-d, r, 1.0), r);
}

}  // namespace moe
