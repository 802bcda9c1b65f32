// slots.h -- entries of a batch that name their states in a pool.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace m3 {

// The slot of entry i, or -1 when it is idle.
__device__ __forceinline__ int slot_of(const int32_t* slots, int n_slots, int i) {
  const int s = slots ? slots[i] : i;
  return (s < 0 || s >= n_slots) ? -1 : s;
}
// Whether this thread sees an entry before i that names the same slot: the NT
// threads of a workgroup look at all of them, 8 a thread in flight.
template <int NT>
__device__ __forceinline__ int named_before(const int32_t* slots, int i, int slot) {
  int same = 0;
  if (slots)
    for (int j0 = threadIdx.x; j0 < i; j0 += 8 * NT) {
      int s[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) s[q] = j0 + q * NT < i ? slots[j0 + q * NT] : -1;
#pragma unroll
      for (int q = 0; q < 8; ++q) same |= s[q] == slot ? 1 : 0;
    }
  return same;
}

}  // namespace m3
