// The INT8 step of a largest magnitude; shared by the quantizers and the forward products' rows.
#pragma once

#include "s3r_internal.h"

namespace s3r {
namespace {

// |v| as ordered bits: for non-negative floats uint order == float order, and
// NaN (> 0x7F800000) wins every max, so a NaN anywhere reaches the step.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Step from amax bits: Delta = fl(a/127), inv = fl(127/a) (a == 0: 1 and 0).
struct Step { float delta, inv, inv24; uint32_t flag; };
__device__ __forceinline__ Step make_step(uint32_t abits) {
  const float a = __uint_as_float(abits);
  Step s;
  s.flag = 0;
  if (abits == 0) { s.delta = 1.f; s.inv = 0.f; s.inv24 = 0.f; return s; }
  s.delta = __fdiv_rn(a, 127.f);
  s.inv = __fdiv_rn(127.f, a);
  s.inv24 = s.inv * 16777216.f;
  if (!(abits < 0x7F800000u)) s.flag |= S3R_FLAG_NONFINITE;
  else if (!(__float_as_uint(s.inv24) < 0x7F800000u)) s.flag |= S3R_FLAG_TINY_STEP;
  return s;
}

}  // namespace
}  // namespace s3r
