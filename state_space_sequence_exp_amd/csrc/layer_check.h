// layer_check.h -- what the host checks of the layer operators share: types,
// alignment, leading dimensions, launch sizes, and whether two arrays of a call
// share memory.  Nothing here touches a device.
#pragma once

#include <limits.h>
#include <string.h>

#include "layer_internal.h"

namespace m3 {
namespace check {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// An enum argument's bits (a C caller may pass any int).
inline int enum_bits(const void* e) {
  int v;
  memcpy(&v, e, sizeof v);
  return v;
}
inline bool dtype_ok(const m3_dtype* d) {
  const int v = enum_bits(d);
  return v == M3_F32 || v == M3_BF16;
}
inline bool code_ok(const m3_code* c) {
  const int v = enum_bits(c);
  return v == M3_CODE_INT8 || v == M3_CODE_E4M3;
}
inline size_t esize_of(m3_dtype d) { return d == M3_BF16 ? 2 : 4; }

// Non-null and aligned to `a` bytes / null or aligned.
inline bool need(const void* p, uintptr_t a) { return p && aligned(p, a); }
inline bool maybe(const void* p, uintptr_t a) { return !p || aligned(p, a); }

// A leading dimension: 0 stands for the row length.
inline bool ld_ok(int64_t ld, int64_t n) { return ld == 0 || ld >= n; }
inline int64_t ld_of(int64_t ld, int64_t n) { return ld ? ld : n; }

inline m3_status done(hipError_t e) { return e == hipSuccess ? M3_SUCCESS : M3_ERR_HIP; }

// Elements of the largest array, kept where byte offsets fit 63 bits.
constexpr double kMaxElements = 1.0e18;

// A launch holds fewer than 2^32 threads: workgroups of 512 and of 256.
constexpr double kMaxGroups512 = 8388607.0, kMaxGroups256 = 16777215.0;

// The memory of one array of a call: `rows` rows of `row` bytes, `pitch` bytes
// apart (a null array has none).
struct Span {
  uintptr_t at;
  uintptr_t rows, row, pitch;
};
inline Span rows_of(const void* p, int64_t rows, int64_t n, int64_t ld, size_t es) {
  if (!p || rows < 1) return Span{};
  const uintptr_t row = (uintptr_t)n * es;
  return Span{reinterpret_cast<uintptr_t>(p), (uintptr_t)rows, row, rows > 1 ? (uintptr_t)ld * es : row};
}
inline Span bytes_of(const void* p, size_t n) {
  return p && n ? Span{reinterpret_cast<uintptr_t>(p), 1, n, n} : Span{};
}

// Whether two arrays share a byte.  Slices of one wider array (the same pitch)
// lie between each other's rows, and so may a dense array; arrays of different
// pitch whose extents meet are taken to share.
inline bool meet(const Span& a, const Span& b) {
  if (!a.row || !b.row) return false;
  const Span &lo = a.at <= b.at ? a : b, &hi = a.at <= b.at ? b : a;
  const uintptr_t off = hi.at - lo.at;
  if (off >= (lo.rows - 1) * lo.pitch + lo.row) return false;
  if (a.rows > 1 && b.rows > 1 && a.pitch != b.pitch) return true;
  const uintptr_t k = off / lo.pitch, at = off % lo.pitch;
  return at < lo.row || (at + hi.row > lo.pitch && k + 1 < lo.rows);
}
// The same, but one array in the place of the other is fine.
inline bool cross(const Span& a, const Span& b) {
  const bool same = a.at == b.at && a.rows == b.rows && a.row == b.row && a.pitch == b.pitch;
  return !same && meet(a, b);
}
// Whether an output lies over an input or another output.
template <size_t NO, size_t NI>
inline bool outputs_meet(const Span (&out)[NO], const Span (&in)[NI]) {
  for (size_t i = 0; i < NO; ++i) {
    for (size_t j = 0; j < i; ++j)
      if (meet(out[i], out[j])) return true;
    for (size_t j = 0; j < NI; ++j)
      if (meet(out[i], in[j])) return true;
  }
  return false;
}

// Whether [a, a + n) and [b, b + n) overlap without being the same.
inline bool partial_overlap(const void* a, const void* b, size_t n) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x != y && x < y + n && y < x + n;
}

}  // namespace check
}  // namespace m3
