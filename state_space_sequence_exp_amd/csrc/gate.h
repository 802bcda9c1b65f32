// gate.h -- the gate of the gated linear recurrence on the device.
//
//   a = sigmoid(f) = 1 / (1 + e),  w = 1 - a = e / (1 + e),  e = exp(-f)
//
// A gate is kept as one float z, the smaller of a and w with a's sign bit
// set: z = w where e <= 1, z = -a where e > 1.  Either value follows from it
// with its relative precision (a long memory is its distance w from 1, a
// short one a itself), so does the slope a w = |z| (1 - |z|), and the masks
// are exact: +0 passes the state on, -0 drops it.  Not looking at what a mask
// hides (it may be NaN) takes some selects a step, which the waves that hold
// no mask leave out (kMask).
#pragma once

#include "m3_device.h"

namespace m3 {

constexpr float kLog2e = 1.44269504088896341f;

// exp(-v) on the hardware exponential; the rounding of v log2(e) makes its
// relative error up to (2 + 1.3 |v|) 2^-24.
__device__ __forceinline__ float exp_neg(float v) { return __builtin_amdgcn_exp2f(v * -kLog2e); }

__device__ __forceinline__ float sigmoid_of(float v) {
  return __builtin_amdgcn_rcpf(1.f + exp_neg(v));
}

__device__ __forceinline__ float gate_of(float f) {
  const float e = exp_neg(f), a = __builtin_amdgcn_rcpf(1.f + e);
  return e > 1.f ? -a : e * a;
}

__device__ __forceinline__ bool gate_cut(float z) { return __float_as_int(z) < 0; }
__device__ __forceinline__ bool gate_drops(float z) { return __float_as_uint(z) == 0x80000000u; }
__device__ __forceinline__ bool gate_passes(float z) { return __float_as_uint(z) == 0u; }

// Whether some gate may be a mask, from the smallest |z|.
__device__ __forceinline__ bool gate_masks(float least) { return least < 1e-30f; }

// w
__device__ __forceinline__ float gate_w(float z) { return z + (gate_cut(z) ? 1.f : 0.f); }
// a v.  kMask: a gate that drops the state does not look at v.
template <bool kMask>
__device__ __forceinline__ float gate_keep(float z, float v) {
  if constexpr (kMask) v = gate_drops(z) ? 0.f : v;
  return __builtin_fmaf(-z, v, gate_cut(z) ? 0.f : v);
}
// a h + w x.  kMask: nor does one that passes it look at x.
template <bool kMask>
__device__ __forceinline__ float gate_step(float z, float h, float x) {
  if constexpr (kMask) x = gate_passes(z) ? 0.f : x;
  return __builtin_fmaf(gate_w(z), x, gate_keep<kMask>(z, h));
}

constexpr float kLeastA = 1.40129846e-45f;  // 2^-149

// A run of steps as a map of the state before it: h -> A h + B.  A is 0 only
// where a gate of the run dropped the state (then h is not looked at): a
// product that underflows stays at the smallest float, so that a NaN state
// that is merely forgotten is NaN after the run as well.
struct Run {
  float A, B;
};
__device__ __forceinline__ float run_apply(Run r, float h) {
  return __builtin_fmaf(r.A, r.A == 0.f ? 0.f : h, r.B);
}
// The factor A of a run with one more gate.  `least`: the smallest that it may
// be, kLeastA to begin with, 0 from a gate on that drops the state (also behind
// a NaN gate, which makes no number of A).
template <bool kMask>
__device__ __forceinline__ float run_factor(float z, float A, float& least) {
  if constexpr (kMask) least = gate_drops(z) ? 0.f : least;
  return fmaxf(gate_keep<false>(z, A), least);
}
// `first`, then `then`.
__device__ __forceinline__ Run run_join(Run first, Run then) {
  const float p = first.A * then.A;
  const bool none = first.A == 0.f || then.A == 0.f;
  return Run{none ? 0.f : (p < kLeastA ? kLeastA : p), run_apply(then, first.B)};
}

}  // namespace m3
