// gate.h -- the gate of the gated linear recurrence on the device.
//
//   a = sigmoid(f),  w = 1 - a = sigmoid(-f):  e = exp(-f), a = 1 / (1 + e),
//   w = e a (1 where e overflows)
//
// so that both keep their relative precision, and a product with a is taken
// from the smaller of the two: a near 1 (long memory) as 1 - w.
#pragma once

#include "m3_device.h"

namespace m3 {

constexpr float kLog2e = 1.44269504088896341f;

// exp(-v) on the hardware exponential: v log2(e) in two floats, the second
// applied to first order, so the result's error does not grow with |v|.
__device__ __forceinline__ float exp_neg(float v) {
  const float hi = -v * kLog2e;
  // what the rounded product left out, in units of the exponent
  const float lo = __builtin_fmaf(-v, kLog2e, -hi) + -v * 1.925963033500e-8f;
  const float e = __builtin_amdgcn_exp2f(hi);
  const float c = e * (lo * 0.6931471805599453f);
  // an infinite v leaves no correction (inf - inf)
  return (c == c && e < 3.0e38f) ? e + c : e;
}

struct Gate {
  float a, w;
};
__device__ __forceinline__ Gate gate_of(float f) {
  const float e = exp_neg(f);
  const float a = 1.f / (1.f + e);
  return Gate{a, e > 3.0e38f ? 1.f : e * a};
}

// a v: from the smaller of a and w, so that neither a long memory (a near 1,
// held as w) nor a short one loses digits.  a = 0 does not look at v.
__device__ __forceinline__ float gate_decay(Gate q, float v) {
  const float s = q.w < 0.5f ? __builtin_fmaf(-q.w, v, v) : q.a * v;
  return q.a == 0.f ? 0.f : s;
}
// a h + w x; w = 0 does not look at x.
__device__ __forceinline__ float gate_step(Gate q, float h, float x) {
  return __builtin_fmaf(q.w, q.w == 0.f ? 0.f : x, gate_decay(q, h));
}

__device__ __forceinline__ float sigmoid_of(float v) { return 1.f / (1.f + exp_neg(v)); }

}  // namespace m3
