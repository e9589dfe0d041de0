// Scalar functions of the step operators (selective scan, RMS norm), fp32, defined for
// every input: infinities and NaN come out as the formulas have them.
#pragma once
#include "gdn_common.h"

namespace gdn {

// exp(x), x <= 0: 2^(x log2 e) with the product's rounding error and log2 e's own tail
// carried along (an exponent of 20 rounded to 24 bits alone would cost 2^-20), on the
// hardware's 2^x.  Below -104 the result is 0 in any case.
__device__ __forceinline__ float step_exp_nonpos(float x) {
  x = x < -104.0f ? -104.0f : x;   // (a NaN stays)
  const float hi = x * 1.4426950408889634f;
  const float lo = fmaf(x, 1.925963033500e-08f, fmaf(x, 1.4426950408889634f, -hi));
  const float e = __builtin_amdgcn_exp2f(hi);
  return fmaf(e, lo * 0.6931471805599453f, e);
}
// log(1 + exp(z))
__device__ __forceinline__ float step_softplus(float z) {
  return (z > 0.0f ? z : 0.0f) + gate_log1p_unit(step_exp_nonpos(-fabsf(z)));
}
// z / (1 + exp(-z)).  The exponential's argument is rounded once, which is worth |z| 2^-23 of
// the result at most (2^-19 at z = -20, where silu is 4e-8); past exp's range the result is -0.
// Held to few instructions: the gated norm is bound by them (170 -> 127 us at 32768 x 32 x 128).
__device__ __forceinline__ float step_silu(float z) {
  return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.4426950408889634f));
}

}  // namespace gdn
