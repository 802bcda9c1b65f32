// vec_io.h -- runs of V neighbouring elements between memory and float
// registers.  A run needs element alignment only: it is moved as one access
// (gfx950 takes any address), but for a cut run at a row's end, which is moved
// element by element.
#pragma once

#include "m3_device.h"

namespace m3 {

template <typename T, int V>
struct Raw {
  static constexpr int kWords = V * (int)sizeof(T) / 4;
  uint32_t w[kWords];
};

// The first n of V elements at p; zeros behind them.
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> load_run(const T* p, int n) {
  Raw<T, V> r;
  if (n >= V) {
    __builtin_memcpy(r.w, p, sizeof r.w);
    return r;
  }
#pragma unroll
  for (int i = 0; i < r.kWords; ++i) r.w[i] = 0u;
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (i < n) {
      if constexpr (sizeof(T) == 2)
        r.w[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << (16 * (i & 1));
      else
        r.w[i] = reinterpret_cast<const uint32_t*>(p)[i];
    }
  return r;
}
template <typename T, int V>
__device__ __forceinline__ void store_run(T* p, int n, const Raw<T, V>& r) {
  if (n >= V) {
    __builtin_memcpy(p, r.w, sizeof r.w);
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (i < n) {
      if constexpr (sizeof(T) == 2)
        reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(r.w[i / 2] >> (16 * (i & 1)));
      else
        reinterpret_cast<uint32_t*>(p)[i] = r.w[i];
    }
}

template <typename T, int V>
__device__ __forceinline__ Raw<T, V> no_run() {
  Raw<T, V> r;
#pragma unroll
  for (int i = 0; i < r.kWords; ++i) r.w[i] = 0u;
  return r;
}

// Element i as a float.
template <int V>
__device__ __forceinline__ float run_at(const Raw<bf16, V>& r, int i) {
  return __uint_as_float(i & 1 ? r.w[i / 2] & 0xffff0000u : r.w[i / 2] << 16);
}
template <int V>
__device__ __forceinline__ float run_at(const Raw<float, V>& r, int i) {
  return __uint_as_float(r.w[i]);
}

// V floats, each rounded once.
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> to_run(const float (&v)[V]) {
  Raw<T, V> r;
  if constexpr (sizeof(T) == 2) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int i = 0; i < r.kWords; ++i)
      r.w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{v[2 * i], v[2 * i + 1]}), bf16x2));
  } else {
#pragma unroll
    for (int i = 0; i < r.kWords; ++i) r.w[i] = __float_as_uint(v[i]);
  }
  return r;
}

// The first n of four floats that are next read much later: they need not stay in the
// caches.
__device__ __forceinline__ void store_for_later(float* p, int n, const float (&v)[4]) {
  typedef f32x4 unaligned __attribute__((aligned(4)));
  if (n >= 4)
    __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, reinterpret_cast<unaligned*>(p));
  else
    store_run<float, 4>(p, n, to_run<float, 4>(v));
}

}  // namespace m3
