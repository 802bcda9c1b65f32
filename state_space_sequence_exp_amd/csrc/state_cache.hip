// state_cache.hip -- recurrent states held in 8 bits: quantised as they are
// written, read back, and the decode step on them.
//
// A row of P values has one scale: amax = max |h|, scale = amax (1 / Q), code
// = round(h (Q / amax)), Q = 127 (int8) or 448 (e4m3); rows below 2^-100 are
// zeros, rows with an infinity or NaN get scale NaN.
//
// A code is a whole number, and a difference in the last bit of a state value
// that lies next to a border changes it for good.  So the decode step is
// defined operation by operation, each rounded to float, none fused:
//   h  = code scale
//   h += ((1 - lam) dt) (sum_r B_prev[r] x_prev[r])
//   h  = (cos h_0 - sin h_1, sin h_0 + cos h_1)           per row pair
//   h  = alpha h + (lam dt) (sum_r B[r] x[r])             r in order
// and any evaluation of these gets the same cache.  A product of two bfloat16
// values is a float, so that in bfloat16 the sums over r are fused all the
// same (4 operations at R = 4 instead of 7, twice an element); the sums of y,
// which is rounded once and not kept, are fused in either type.
//
// Store and load are bound by memory (256 x 32 states of 128 x 64: 66 and 68 us,
// 5 TB/s), the decode step by its vector operations: at R = 4 those that its
// definition asks for, one by one, take 40 us of 256 x 32 units, N = 128, P =
// 64, where the bytes take 34 (at a copy's 5.4 TB/s).
//
// A workgroup owns one (sequence, head).  Its threads request their codes,
// then put the coefficients of the row pairs into the LDS, a pair's together;
// a thread updates 8 columns of its row pairs in registers; a row's largest
// magnitude comes from the lanes that share the row.
#include "layer_internal.h"
#include "m3_device.h"

// For the whole file: a fused operation is one rounding less, which is another
// code now and then (the product h (Q / amax), say, is rounded before the sum
// that rounds it to a whole number).
#pragma clang fp contract(off)

namespace m3 {
namespace {

constexpr int kThreads = 256;
constexpr float kTinyRow = 7.8886090522101181e-31f;  // 2^-100

// The 8 codes of a lane as two words, and back.
template <int kCode>
struct Code;
template <>
struct Code<M3_CODE_INT8> {
  static constexpr float kMax = 127.f;
  __device__ __forceinline__ static void unpack4(uint32_t w, float* v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (float)(int8_t)(w >> (8 * i));
  }
  // |v| <= 127 (1 + 2^-23): beside 1.5 x 2^23 a float's last place is one, so
  // the sum's low byte is v rounded to even, in two's complement
  __device__ __forceinline__ static uint32_t pack4(const float* v) {
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(v[i] + 12582912.f);
    const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000c0cu);
    return lo | hi;
  }
};
template <>
struct Code<M3_CODE_E4M3> {
  static constexpr float kMax = 448.f;
  __device__ __forceinline__ static void unpack4(uint32_t w, float* v) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
    const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    v[0] = lo.x; v[1] = lo.y; v[2] = hi.x; v[3] = hi.y;
  }
  // |v| <= 448 (1 + 2^-23), which rounds to 448: nothing to clamp
  __device__ __forceinline__ static uint32_t pack4(const float* v) {
    int w = 0;
    w = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], w, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], w, true);
    return (uint32_t)w;
  }
};

// A row's scale and the factor that takes it to codes, from its largest
// magnitude (NaN where the row holds one).
template <int kCode>
__device__ __forceinline__ void row_scale(float amax, float* scale, float* inv) {
  const bool held = amax >= kTinyRow && amax < __builtin_inff();
  *inv = held ? Code<kCode>::kMax / amax : 0.f;
  *scale = held ? amax * (1.f / Code<kCode>::kMax) : amax < kTinyRow ? 0.f : __uint_as_float(0x7fc00000u);
}

// Codes of 8 values of a row.
template <int kCode>
__device__ __forceinline__ uint2 quantise8(const float (&h)[8], float amax, float inv) {
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = h[e] * inv;
  // rare, so a branch of the whole wave: 0 x infinity is no code
  const bool bad = !(amax < __builtin_inff());
  if (__builtin_expect(__any(bad), 0)) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = bad ? 0.f : v[e];
  }
  return make_uint2(Code<kCode>::pack4(v), Code<kCode>::pack4(v + 4));
}

// The larger of two magnitudes; NaN if one is.
__device__ __forceinline__ float max_abs(float a, float b) {
  return __builtin_elementwise_maximum(__builtin_fabsf(a), __builtin_fabsf(b));
}
__device__ __forceinline__ float top8(const float (&h)[8]) {
  const float a = max_abs(max_abs(h[0], h[1]), h[2]), b = max_abs(max_abs(h[3], h[4]), h[5]);
  return max_abs(max_abs(a, b), max_abs(h[6], h[7]));
}
__device__ __forceinline__ float top16(const float (&h)[16]) {
  float t = max_abs(h[0], h[1]);
#pragma unroll
  for (int e = 2; e < 16; e += 2) t = max_abs(max_abs(t, h[e]), h[e + 1]);
  return t;
}
// a = (a of lanes 0-31, b of lanes 0-31), b = (a of 32-63, b of 32-63).
__device__ __forceinline__ void swap_halves(float& a, float& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  a = __uint_as_float(r[0]);
  b = __uint_as_float(r[1]);
}
// The same in quarters: a keeps its lanes 0-15 and 32-47 and gets b's of them
// in 16-31 and 48-63; b gets a's of 16-31 and 48-63 in 0-15 and 32-47.
__device__ __forceinline__ void swap_rows(float& a, float& b) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  a = __uint_as_float(r[0]);
  b = __uint_as_float(r[1]);
}
template <int kCode>
__device__ __forceinline__ void unpack16(const uint4& w, float scale, float (&v)[16]) {
  Code<kCode>::unpack4(w.x, v);
  Code<kCode>::unpack4(w.y, v + 4);
  Code<kCode>::unpack4(w.z, v + 8);
  Code<kCode>::unpack4(w.w, v + 12);
#pragma unroll
  for (int e = 0; e < 16; ++e) v[e] *= scale;
}
// Codes of 16 values of a row.
template <int kCode>
__device__ __forceinline__ uint4 quantise16(const float (&h)[16], float amax, float inv) {
  float v[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) v[e] = h[e] * inv;
  const bool bad = !(amax < __builtin_inff());
  if (__builtin_expect(__any(bad), 0)) {
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = bad ? 0.f : v[e];
  }
  return make_uint4(Code<kCode>::pack4(v), Code<kCode>::pack4(v + 4), Code<kCode>::pack4(v + 8),
                    Code<kCode>::pack4(v + 12));
}

// Maximum over the `lanes` (2, 4, 8 or 16) consecutive lanes of a row, by lane
// moves inside the 16 lanes of a DPP row: lane xor 1, xor 2, then (all four of
// a quad being equal) the mirrored half row and row.
__device__ __forceinline__ float row_top(float top, int lanes) {
  top = max_abs(top, dpp_move<0xb1>(top));
  if (lanes > 2) top = max_abs(top, dpp_move<0x4e>(top));
  if (lanes > 4) top = max_abs(top, dpp_move<0x141>(top));
  if (lanes > 8) top = max_abs(top, dpp_move<0x140>(top));
  return top;
}

// The slot of entry i, or -1 when it is idle.
__device__ __forceinline__ int slot_of(const CacheArgs& a, int i) {
  const int s = a.slots ? a.slots[i] : i;
  return (s < 0 || s >= a.n_slots) ? -1 : s;
}
// Whether this thread sees an entry before i that names the same slot: the NT
// threads of a workgroup look at all of them, 8 a thread in flight.
template <int NT>
__device__ __forceinline__ int named_before(const CacheArgs& a, int i, int slot) {
  int same = 0;
  if (a.slots)
    for (int j0 = threadIdx.x; j0 < i; j0 += 8 * NT) {
      int s[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) s[q] = j0 + q * NT < i ? a.slots[j0 + q * NT] : -1;
#pragma unroll
      for (int q = 0; q < 8; ++q) same |= s[q] == slot ? 1 : 0;
    }
  return same;
}

template <int kCode>
__global__ void __launch_bounds__(kThreads) store_kernel(CacheArgs a) {
  const int i = blockIdx.x / a.H, head = blockIdx.x % a.H;
  const int slot = slot_of(a, i);
  if (slot < 0 || __syncthreads_or(named_before<kThreads>(a, i, slot))) return;
  const int lanes = a.P / 8;
  const float* h = a.h_in + ((size_t)i * a.H + head) * a.N * a.P;
  const size_t unit = (size_t)slot * a.H + head;
  uint2* codes = reinterpret_cast<uint2*>(static_cast<unsigned char*>(a.codes) + unit * a.N * a.P);
  for (int p0 = 0; p0 < a.N * lanes; p0 += kThreads) {  // every lane of a row together
    const int p = p0 + threadIdx.x;
    const bool in = p < a.N * lanes;
    float v[8];
    const float4 lo = in ? reinterpret_cast<const float4*>(h)[2 * p] : make_float4(0, 0, 0, 0);
    const float4 hi = in ? reinterpret_cast<const float4*>(h)[2 * p + 1] : make_float4(0, 0, 0, 0);
    v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
    v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
    const float top = row_top(top8(v), lanes);
    float scale, inv;
    row_scale<kCode>(top, &scale, &inv);
    if (in) {
      codes[p] = quantise8<kCode>(v, top, inv);
      if (p % lanes == 0) a.scales[unit * a.N + p / lanes] = scale;
    }
  }
}

// A thread reads the codes of one 16-byte vector of the output at a time (4
// floats, 8 bfloat16), so that a wave writes whole lines, and has four in
// flight: 68 us for 256 x 32 states of 128 x 64 into floats (4.9 TB/s), 41 us
// into bfloat16.  (With 8 columns a thread, two vectors side by side, 92 and 46.)
template <int kCode, typename T>
__global__ void __launch_bounds__(kThreads) load_kernel(CacheArgs a) {
  constexpr int E = 16 / (int)sizeof(T), W = E / 4, K = 4;
  struct Words {
    uint32_t w[W];
  };
  typedef T Out __attribute__((ext_vector_type(E)));
  const int i = blockIdx.x / a.H, head = blockIdx.x % a.H;
  const int slot = slot_of(a, i);
  const int lanes = a.P / E, all = a.N * lanes;
  Out* h = reinterpret_cast<Out*>(static_cast<T*>(a.h_out) + ((size_t)i * a.H + head) * a.N * a.P);
  if (slot < 0) {
    for (int p = threadIdx.x; p < all; p += kThreads) h[p] = Out(from_f32<T>(0.f));
    return;
  }
  const size_t unit = (size_t)slot * a.H + head;
  const Words* codes =
      reinterpret_cast<const Words*>(static_cast<const unsigned char*>(a.codes) + unit * a.N * a.P);
  for (int p0 = threadIdx.x; p0 < all; p0 += K * kThreads) {
    Words w[K];
    float scale[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int p = min(p0 + k * kThreads, all - 1);
      w[k] = codes[p];
      scale[k] = a.scales[unit * a.N + p / lanes];
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      Out o;
#pragma unroll
      for (int j = 0; j < W; ++j) {
        float v[4];
        Code<kCode>::unpack4(w[k].w[j], v);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[4 * j + e] = from_f32<T>(v[e] * scale[k]);
      }
      if (p0 + k * kThreads < all) h[p0 + k * kThreads] = o;
    }
  }
}

// 8 consecutive inputs as floats.
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const bf16* p, float (&v)[8]) {
  // the pointers are aligned to four elements
  const uint2 a = reinterpret_cast<const uint2*>(p)[0], b = reinterpret_cast<const uint2*>(p)[1];
  const uint32_t w[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// A row pair's coefficients in the LDS: cos, sin, 2 unused, then B_prev, B
// and C of row 0 (R each) and of row 1.
template <int R>
struct PairCoef {
  float cs, sn, pad[R == 2 ? 6 : 2];
  float bp[2][R], b[2][R], c[2][R];
};

template <typename T, int R, bool kTrap, bool kRot, int NT>
__device__ __forceinline__ void pair_coefficients(const CacheArgs& a, size_t in, int npair, float d,
                                                  PairCoef<R>* s_pair) {
  for (int kp = threadIdx.x; kp < npair; kp += NT) {
    PairCoef<R>& q = s_pair[kp];
    if constexpr (kRot) {
      const float psi = d * a.theta[in * npair + kp];
      sincosf(psi, &q.sn, &q.cs);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const size_t at = (in * R + r) * (2 * npair) + 2 * kp;
      const float2 b = load_pair(static_cast<const T*>(a.B_t) + at);
      const float2 c = load_pair(static_cast<const T*>(a.C_t) + at);
      q.b[0][r] = b.x; q.b[1][r] = b.y;
      q.c[0][r] = c.x; q.c[1][r] = c.y;
      if constexpr (kTrap) {
        const float2 p = load_pair(static_cast<const T*>(a.B_prev) + at);
        q.bp[0][r] = p.x; q.bp[1][r] = p.y;
      }
    }
  }
}

// sum_r b[r] x[r][e] in order, each product and sum rounded (a product of two
// bfloat16 values is exact, so there the fused form is the same).
template <typename T, int R>
__device__ __forceinline__ float rank_sum(const float (&b)[R], const float (&x)[R][8], int e) {
  float t = b[0] * x[0][e];
#pragma unroll
  for (int r = 1; r < R; ++r) {
    if constexpr (sizeof(T) == 2)
      t = __builtin_fmaf(b[r], x[r][e], t);
    else
      t = t + b[r] * x[r][e];
  }
  return t;
}

// What a thread reads of one row pair.
struct PairIn {
  uint2 w0, w1;
  float s0, s1;
};

// NT threads own a unit: row pair rg + k NT / lanes is the k-th of the thread
// in lane group rg.  The next pair is requested before the present one is
// worked on.
template <typename T, int R, int kCode, bool kTrap, bool kRot, int NT>
__global__ void __launch_bounds__(NT) decode_kernel(CacheArgs a) {
  extern __shared__ __align__(16) float dsm[];
  const int i = blockIdx.x / a.H, head = blockIdx.x % a.H;
  const int slot = slot_of(a, i);
  if (slot < 0) return;
  const int N = a.N, P = a.P, npair = N / 2, lanes = P / 8;
  const int tid = threadIdx.x, c8 = tid % lanes, rg = tid / lanes, groups = NT / lanes;
  const size_t in = (size_t)i * a.H + head;       // this token's inputs
  const size_t unit = (size_t)slot * a.H + head;  // its state
  PairCoef<R>* s_pair = reinterpret_cast<PairCoef<R>*>(dsm);
  float* s_y = dsm;  // [groups][R][P], in the coefficients' place at the end

  char* codes = static_cast<char*>(a.codes) + unit * N * P;
  float* scales = a.scales + unit * N;
  // pair kp's codes: row 2 kp at byte 2 kp P, its second row P bytes on
  // (past the last pair: the last pair's, unused)
  const auto request = [&](int kp) {
    kp = kp < npair ? kp : npair - 1;
    const uint32_t at = 2 * kp * P + 8 * c8;
    return PairIn{*reinterpret_cast<const uint2*>(codes + at),
                  *reinterpret_cast<const uint2*>(codes + at + P), scales[2 * kp], scales[2 * kp + 1]};
  };
  PairIn cur = request(rg);
  float xc[R][8], xq[R][8], yp[R][8];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const size_t at = (in * R + r) * P + 8 * c8;
    load8(static_cast<const T*>(a.x_t) + at, xc[r]);
    if constexpr (kTrap) load8(static_cast<const T*>(a.x_prev) + at, xq[r]);
#pragma unroll
    for (int e = 0; e < 8; ++e) yp[r][e] = 0.f;
  }
  const float d = a.dt[in], la = kTrap ? a.lam[in] : 1.f;
  const float alpha = expf(d * a.A[head]);
  const float cu = (1.f - la) * d, cv = la * d;
  pair_coefficients<T, R, kTrap, kRot, NT>(a, in, npair, d, s_pair);
  // of entries with one slot the first takes it; also the barrier before the
  // coefficients are read
  if (__syncthreads_or(named_before<NT>(a, i, slot))) return;

  for (int kp = rg; kp < npair; kp += groups) {  // the lanes of a row together
    const PairCoef<R>& q = s_pair[kp];
    float v0[8], v1[8];
    Code<kCode>::unpack4(cur.w0.x, v0);
    Code<kCode>::unpack4(cur.w0.y, v0 + 4);
    Code<kCode>::unpack4(cur.w1.x, v1);
    Code<kCode>::unpack4(cur.w1.y, v1 + 4);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v0[e] = v0[e] * cur.s0;
      v1[e] = v1[e] * cur.s1;
    }
    cur = request(kp + groups);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float h0 = v0[e], h1 = v1[e];
      if constexpr (kTrap) {
        h0 = h0 + cu * rank_sum<T, R>(q.bp[0], xq, e);
        h1 = h1 + cu * rank_sum<T, R>(q.bp[1], xq, e);
      }
      if constexpr (kRot) {
        const float n0 = q.cs * h0 - q.sn * h1, n1 = q.sn * h0 + q.cs * h1;
        h0 = n0;
        h1 = n1;
      }
      v0[e] = alpha * h0 + cv * rank_sum<T, R>(q.b[0], xc, e);
      v1[e] = alpha * h1 + cv * rank_sum<T, R>(q.b[1], xc, e);
#pragma unroll
      for (int r = 0; r < R; ++r)
        yp[r][e] = __builtin_fmaf(q.c[0][r], v0[e], __builtin_fmaf(q.c[1][r], v1[e], yp[r][e]));
    }
    // the even lanes of a row pair take the first row's scale, the odd ones
    // the second's: one division for both
    const float t0 = row_top(top8(v0), lanes), t1 = row_top(top8(v1), lanes);
    float scale, inv;
    row_scale<kCode>(c8 & 1 ? t1 : t0, &scale, &inv);
    const float i0 = dpp_move<0xa0>(inv), i1 = dpp_move<0xf5>(inv);  // of lanes 0, 0, 2, 2 / 1, 1, 3, 3
    const uint32_t at = 2 * kp * P + 8 * c8;
    *reinterpret_cast<uint2*>(codes + at) = quantise8<kCode>(v0, t0, i0);
    *reinterpret_cast<uint2*>(codes + at + P) = quantise8<kCode>(v1, t1, i1);
    if (c8 < 2) scales[2 * kp + c8] = scale;
  }
  __syncthreads();  // the coefficients are read
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float4* o = reinterpret_cast<float4*>(s_y + (rg * R + r) * P + 8 * c8);
    o[0] = make_float4(yp[r][0], yp[r][1], yp[r][2], yp[r][3]);
    o[1] = make_float4(yp[r][4], yp[r][5], yp[r][6], yp[r][7]);
  }
  __syncthreads();
  T* y = static_cast<T*>(a.y) + in * R * P;
  for (int o = tid; o < R * P; o += NT) {
    float sum = 0.f;
    for (int g = 0; g < groups; ++g) sum += s_y[g * R * P + o];
    y[o] = from_f32<T>(sum);
  }
}

template <typename T, int R, int kCode, bool kTrap, bool kRot, int NT>
hipError_t launch_decode_nt(const CacheArgs& a, hipStream_t stream) {
  const size_t coef = sizeof(PairCoef<R>) * (a.N / 2);
  const size_t part = sizeof(float) * (size_t)(NT / (a.P / 8)) * R * a.P;
  const size_t lds = coef > part ? coef : part;
  const hipError_t e = lds_limit(
      reinterpret_cast<const void*>(&decode_kernel<T, R, kCode, kTrap, kRot, NT>), lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((decode_kernel<T, R, kCode, kTrap, kRot, NT>), dim3(a.S * a.H), dim3(NT), lds,
                     stream, a);
  return hipGetLastError();
}

// The same step with the sums over r on the matrix units, a wave a unit, for
// bfloat16 inputs, states of 64 columns and whole sets of 16 row pairs.
//
// A 16x16x1 instruction takes one r of the outer product of 16 rows with 64
// columns and rounds each sum once, as a fused multiply-add does, so R of them
// in order are rank_sum (a sum of zeros is +0 here, whatever their signs: the
// cache holds the same values).  Lane (g, c) = (lane / 16, lane % 16) gets row
// c's columns 16 g + 4 b + j as value j of block b, so that a lane has 16
// consecutive columns where the x given to row 4 g + j of block b is that
// column's.  The c are 16 row pairs, one product for the pair's first rows and
// one for the second.
//
// What is left to the vector units is 17 operations an element at R = 4
// instead of 23.5, and a row's scale costs half as much (four lanes share a
// row, not eight).  Measured in turn on 256 x 32 units, N = 128, R = 4: 55 us
// against 58.5 (int8) and 62.5 (e4m3); 128 x 64, N = 64, R = 1: 24.5 against
// 26; R = 2: 27.5 against 30; 2048 units, N = 128, R = 4: 17.2 against 20.2;
// 1024: 11.7 against 15.0.  Below 1024 units four waves a unit are faster (512:
// 9.1 against 11.4), and with four waves this form is not (9.4); with 17 pairs
// instead of 16 it takes 21 us against 19 (8192 units, R = 1).  165 registers at R = 4
// let three waves run on a SIMD (unbounded it takes 207, two waves and 64 us).
template <int R>
__device__ __forceinline__ void outer(const float (&x)[R], const float (&b)[R], float (&v)[16]) {
  typedef float f32x16 __attribute__((ext_vector_type(16)));
  f32x16 t = f32x16(0.f);
#pragma unroll
  for (int r = 0; r < R; ++r) t = __builtin_amdgcn_mfma_f32_16x16x1f32(x[r], b[r], t, 0, 0, 0);
#pragma unroll
  for (int e = 0; e < 16; ++e) v[e] = t[e];
}

template <int R, int kCode, bool kTrap, bool kRot>
__global__ void __launch_bounds__(kWave, R > 2 ? 3 : 4) decode_outer_kernel(CacheArgs a) {
  constexpr int P = 64, kRound = R < 2 ? R : 2, kPitch = kRound * P + 4;
  extern __shared__ __align__(16) float dsm[];
  const int i = blockIdx.x / a.H, head = blockIdx.x % a.H;
  const int slot = slot_of(a, i);
  if (slot < 0) return;
  const int N = a.N, npair = N / 2;
  const int lane = threadIdx.x, g = lane / 16, c = lane % 16;
  const size_t in = (size_t)i * a.H + head;       // this token's inputs
  const size_t unit = (size_t)slot * a.H + head;  // its state
  PairCoef<R>* s_pair = reinterpret_cast<PairCoef<R>*>(dsm);

  char* codes = static_cast<char*>(a.codes) + unit * N * P;
  float* scales = a.scales + unit * N;
  struct In {
    uint4 w0, w1;
    float s0, s1;
  };
  // this lane's pair of the 16 from k0 on (behind the last: of the last ones, unused)
  const auto request = [&](int k0) {
    const int kp = min(k0, npair - 16) + c;
    const uint32_t at = 2 * kp * P + 16 * g;
    return In{*reinterpret_cast<const uint4*>(codes + at),
              *reinterpret_cast<const uint4*>(codes + at + P), scales[2 * kp], scales[2 * kp + 1]};
  };
  In cur = request(0);
  float xc[R], xq[R], yp[R][16];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const size_t at = (in * R + r) * P + 16 * (c / 4) + 4 * g + c % 4;
    xc[r] = to_f32(static_cast<const bf16*>(a.x_t)[at]);
    if constexpr (kTrap) xq[r] = to_f32(static_cast<const bf16*>(a.x_prev)[at]);
#pragma unroll
    for (int e = 0; e < 16; ++e) yp[r][e] = 0.f;
  }
  const float d = a.dt[in], la = kTrap ? a.lam[in] : 1.f;
  const float alpha = expf(d * a.A[head]);
  const float cu = (1.f - la) * d, cv = la * d;
  pair_coefficients<bf16, R, kTrap, kRot, kWave>(a, in, npair, d, s_pair);
  if (__syncthreads_or(named_before<kWave>(a, i, slot))) return;

  for (int k0 = 0; k0 < npair; k0 += 16) {
    const int kp = k0 + c;
    const PairCoef<R>& q = s_pair[kp];
    // one outer product at a time, behind the vector work that does not need
    // it, kept in this order (the compiler's own takes more registers)
    float v0[16], v1[16], o[16];
    if constexpr (kTrap) outer<R>(xq, q.bp[0], o);
    unpack16<kCode>(cur.w0, cur.s0, v0);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (kTrap) {
#pragma unroll
      for (int e = 0; e < 16; ++e) v0[e] = v0[e] + cu * o[e];
      outer<R>(xq, q.bp[1], o);
    }
    unpack16<kCode>(cur.w1, cur.s1, v1);
    __builtin_amdgcn_sched_barrier(0);
    cur = request(k0 + 16);
    if constexpr (kTrap) {
#pragma unroll
      for (int e = 0; e < 16; ++e) v1[e] = v1[e] + cu * o[e];
    }
    outer<R>(xc, q.b[0], o);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float h0 = v0[e], h1 = v1[e];
      if constexpr (kRot) {
        const float n0 = q.cs * h0 - q.sn * h1, n1 = q.sn * h0 + q.cs * h1;
        h0 = n0;
        h1 = n1;
      }
      v0[e] = alpha * h0;
      v1[e] = alpha * h1;
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int e = 0; e < 16; ++e) v0[e] = v0[e] + cv * o[e];
    outer<R>(xc, q.b[1], o);
    float top = top16(v0);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < 16; ++e) yp[r][e] = __builtin_fmaf(q.c[0][r], v0[e], yp[r][e]);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int e = 0; e < 16; ++e) v1[e] = v1[e] + cv * o[e];
    float top1 = top16(v1);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < 16; ++e) yp[r][e] = __builtin_fmaf(q.c[1][r], v1[e], yp[r][e]);
    // lanes 0-31 take the first rows' scales, 32-63 the second rows': one
    // division for both
    swap_halves(top, top1);
    top = max_abs(top, top1);
    top1 = top;
    swap_rows(top, top1);
    top = max_abs(top, top1);
    float scale, i0;
    row_scale<kCode>(top, &scale, &i0);
    float i1 = i0, t0 = top, t1 = top;
    swap_halves(i0, i1);
    swap_halves(t0, t1);
    const uint32_t at = 2 * kp * P + 16 * g;
    *reinterpret_cast<uint4*>(codes + at) = quantise16<kCode>(v0, t0, i0);
    *reinterpret_cast<uint4*>(codes + at + P) = quantise16<kCode>(v1, t1, i1);
    if (g % 2 == 0) scales[2 * kp + g / 2] = scale;
  }
  // y: each lane's sums over its row pairs, then those of the 16 lanes that
  // share its columns, up to two r at a time
#pragma unroll
  for (int r0 = 0; r0 < R; r0 += kRound) {
    __syncthreads();  // the coefficients or the sums before these are read
#pragma unroll
    for (int r = 0; r < kRound; ++r)
#pragma unroll
      for (int e = 0; e < 16; e += 4)
        *reinterpret_cast<float4*>(dsm + c * kPitch + r * P + 16 * g + e) =
            make_float4(yp[r0 + r][e], yp[r0 + r][e + 1], yp[r0 + r][e + 2], yp[r0 + r][e + 3]);
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kRound; ++r) {
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < 16; ++k) sum += dsm[k * kPitch + r * P + lane];
      static_cast<bf16*>(a.y)[(in * R + r0 + r) * P + lane] = from_f32<bf16>(sum);
    }
  }
}

template <int R, int kCode, bool kTrap, bool kRot>
hipError_t launch_outer(const CacheArgs& a, hipStream_t stream) {
  const size_t coef = sizeof(PairCoef<R>) * (a.N / 2);
  const size_t part = sizeof(float) * 16 * ((R < 2 ? R : 2) * 64 + 4);
  const size_t lds = coef > part ? coef : part;
  const hipError_t e = lds_limit(
      reinterpret_cast<const void*>(&decode_outer_kernel<R, kCode, kTrap, kRot>), lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((decode_outer_kernel<R, kCode, kTrap, kRot>), dim3(a.S * a.H), dim3(kWave), lds,
                     stream, a);
  return hipGetLastError();
}

// The matrix units where they serve; else one wave a unit once there is a wave
// for every SIMD, four before that; from
// 2048 units on where a wave takes 16 turns or more (a workgroup of four then
// pays longer), and always where a wave holds the whole unit.  Measured, us for
// one wave / four: N = 128, P = 64, R = 4, bfloat16: 12.4 / 6.8 with 256 units,
// 13.8 / 13.6 with 1024, 18.9 / 22.1 with 2048, 57.3 / 74.9 with 8192; N = P =
// 64, R = 1: 6.1 / 4.4, 6.9 / 6.8, 9.0 / 10.2, 22.9 / 30.6; N = P = 128, R = 4,
// float: 25.1 / 10.4, 28.5 / 21.8, 37.5 / 37.2, 114.6 / 130.2; N = 64, P = 16,
// R = 2, a whole unit: 4.3 / 5.9, 4.5 / 6.8, 5.7 / 12.2, 13.2 / 38.0.
template <typename T, int R, int kCode, bool kTrap, bool kRot>
hipError_t launch_decode_form(const CacheArgs& a, hipStream_t stream) {
  const int groups = kWave / (a.P / 8), turns = (a.N / 2 + groups - 1) / groups;
  const int64_t units = (int64_t)a.S * a.H;
  if constexpr (sizeof(T) == 2)
    if (a.P == 64 && a.N % 32 == 0 && units >= 1024)
      return launch_outer<R, kCode, kTrap, kRot>(a, stream);
  if (turns <= 1 || units >= (turns >= 16 ? 2048 : 1024))
    return launch_decode_nt<T, R, kCode, kTrap, kRot, 64>(a, stream);
  return launch_decode_nt<T, R, kCode, kTrap, kRot, 256>(a, stream);
}

template <typename T, int R, int kCode>
hipError_t launch_decode_r(const CacheArgs& a, hipStream_t stream) {
  if (a.lam)
    return a.theta ? launch_decode_form<T, R, kCode, true, true>(a, stream)
                   : launch_decode_form<T, R, kCode, true, false>(a, stream);
  return a.theta ? launch_decode_form<T, R, kCode, false, true>(a, stream)
                 : launch_decode_form<T, R, kCode, false, false>(a, stream);
}

template <typename T, int kCode>
hipError_t launch_decode_t(const CacheArgs& a, hipStream_t stream) {
  switch (a.R) {
    case 1: return launch_decode_r<T, 1, kCode>(a, stream);
    case 2: return launch_decode_r<T, 2, kCode>(a, stream);
    case 4: return launch_decode_r<T, 4, kCode>(a, stream);
    default: return hipErrorInvalidValue;
  }
}

template <int kCode>
hipError_t launch_load_t(const CacheArgs& a, m3_dtype dtype, hipStream_t stream) {
  if (dtype == M3_BF16)
    hipLaunchKernelGGL((load_kernel<kCode, bf16>), dim3(a.S * a.H), dim3(kThreads), 0, stream, a);
  else
    hipLaunchKernelGGL((load_kernel<kCode, float>), dim3(a.S * a.H), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_state_store(const CacheArgs& a, m3_code code, hipStream_t stream) {
  if (code == M3_CODE_INT8)
    hipLaunchKernelGGL(store_kernel<M3_CODE_INT8>, dim3(a.S * a.H), dim3(kThreads), 0, stream, a);
  else
    hipLaunchKernelGGL(store_kernel<M3_CODE_E4M3>, dim3(a.S * a.H), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_state_load(const CacheArgs& a, m3_code code, m3_dtype dtype,
                             hipStream_t stream) {
  return code == M3_CODE_INT8 ? launch_load_t<M3_CODE_INT8>(a, dtype, stream)
                              : launch_load_t<M3_CODE_E4M3>(a, dtype, stream);
}

hipError_t launch_decode_cached(const CacheArgs& a, m3_code code, m3_dtype dtype,
                                hipStream_t stream) {
  if (dtype == M3_BF16)
    return code == M3_CODE_INT8 ? launch_decode_t<bf16, M3_CODE_INT8>(a, stream)
                                : launch_decode_t<bf16, M3_CODE_E4M3>(a, stream);
  return code == M3_CODE_INT8 ? launch_decode_t<float, M3_CODE_INT8>(a, stream)
                              : launch_decode_t<float, M3_CODE_E4M3>(a, stream);
}

}  // namespace m3
