// layer_norm.hip -- layer norm with the residual sum, and its gradients:
//
//   s = x + residual,  q = (s - mean) rstd,  y = q weight + bias
//   dx = rstd (p - mean(p) - q mean(p q)) + dsum,  p = dy weight
//   dweight = sum_rows dy q,  dbias = sum_rows dy
//
// Bound by memory: each array is read or written once.  A row belongs to a
// team of 64 to 1024 threads that keeps it in registers, NV 16-byte
// vectors a thread, between the sum, the centred squares and the output; the
// threads keep their columns of the weights while their team walks rows.  The
// sums go by lane moves in a wave and by the LDS between waves.  (Rows above
// 8192 channels ask for more than the 128 registers that 1024 threads leave a
// thread in the backward pass: it spills 3 to 13 of them for bfloat16, 11 or 27
// for float.)
//
// The backward pass keeps each column's dweight and dbias in the registers of
// the thread that owns it, over all rows of its workgroup (up to 256 groups of
// rows); the teams of a workgroup are joined in the LDS, the groups by a
// second kernel, both in a fixed order.
//
// 8192 x 2048 bfloat16 with the residual and its gradient: forward 26 us (5.1
// TB/s), backward 29 and 4 for the joining kernel (4.6 without it).  Rows that
// are not 16-byte aligned run at 0.6 to 0.9 of that.  A row that leaves its team
// idle costs more in the backward pass, which has one workgroup a compute unit:
// 16384 x 2100 bfloat16 (263 vectors in a team of 512) 102 us, x 2047 63.  Above
// 8192 channels, 2048 rows with the residual's gradient, bfloat16 / float: 12288
// wide 65 / 102 us (its bytes take 37 / 75), 16384 wide 89 / 136 (50 / 100), 16383
// wide 118 / 174; 8192 wide, which does not spill, 52 / 62 (25 / 50).
#include <algorithm>

#include "layer_internal.h"
#include "m3_device.h"

namespace m3 {
namespace {

template <typename T>
constexpr int kE = 16 / (int)sizeof(T);  // elements of a vector

struct Vec {
  uint32_t w[4];
};

template <typename T>
__device__ __forceinline__ void unpack(const Vec& p, float (&v)[kE<T>]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2) {
      v[2 * i] = __uint_as_float(p.w[i] << 16);
      v[2 * i + 1] = __uint_as_float(p.w[i] & 0xffff0000u);
    } else {
      v[i] = __uint_as_float(p.w[i]);
    }
  }
}
template <typename T>
__device__ __forceinline__ Vec pack(const float (&v)[kE<T>]) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  Vec p;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2)
      p.w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{v[2 * i], v[2 * i + 1]}), bf16x2));
    else
      p.w[i] = __float_as_uint(v[i]);
  }
  return p;
}

// n of a vector's elements at p (n <= 0: none; the rest zeros).  kVec: rows
// are 16-byte aligned and n is a whole vector or <= 0; else elements are
// aligned and the last vector of a row may be cut.
//
// A cut vector of bfloat16 (`wide`) is loaded as the row's last 8 elements, and
// trim moves its own down when they are used, not before: guarded loads of
// single elements are put together as they arrive and so wait for each other
// in every row, and for the row that was requested ahead.  16384 rows with the
// residual, forward / backward: 2047 wide 48 / 63 us against 52 / 86, 2100 wide
// 61 / 102 against 96 / 100, 4095 wide 117 / 141 against 198 / 210.  One element
// alone waits for nobody (4097 wide: 143 / 216 against 117 / 183), nor do
// floats, each of which has a register (4095 wide: 228 / 252 against 224 / 209).
// Rows of such widths have kernels of their own (kCut), without the registers
// of the other form: in one kernel with it, 4097 wide took 132 us forward and
// 12281 wide (4096 rows) 161 backward, against 118 and 138.  (The other way round it
// does not pay: a kernel that knows `wide` spills at 1024 threads, 8191 wide
// 257 us forward against 242.)
template <typename T>
__host__ __device__ __forceinline__ bool loads_whole(int D) {
  return sizeof(T) == 2 && D >= kE<T> && D % kE<T> != 1;
}
template <typename T, bool kVec>
__device__ __forceinline__ Vec load_vec(const T* p, int n, bool wide) {
  constexpr int E = kE<T>;
  Vec r = {{0u, 0u, 0u, 0u}};
  if constexpr (kVec) {
    if (n >= E) {
      const uint4 u = *reinterpret_cast<const uint4*>(p);
      r.w[0] = u.x; r.w[1] = u.y; r.w[2] = u.z; r.w[3] = u.w;
    }
  } else if (wide) {
    if (n > 0) __builtin_memcpy(r.w, p - (n < E ? E - n : 0), 16);
  } else if (n >= E) {
    __builtin_memcpy(r.w, p, 16);
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (i < n) {
        if constexpr (sizeof(T) == 2)
          r.w[i / 2] |= (uint32_t)__builtin_bit_cast(uint16_t, p[i]) << (16 * (i & 1));
        else
          r.w[i] = __builtin_bit_cast(uint32_t, p[i]);
      }
  }
  return r;
}
template <typename T, bool kVec>
__device__ __forceinline__ void trim(Vec& r, int n, bool wide) {
  constexpr int E = kE<T>, W = 4 / (int)sizeof(T);
  if (!kVec && sizeof(T) == 2 && wide && n > 0 && n < E) {
    const int by = E - n;
#pragma unroll
    for (int step = 2; step > 0; step /= 2)  // whole words
#pragma unroll
      for (int i = 0; i < 4; ++i)
        r.w[i] = by & (step * W) ? (i + step < 4 ? r.w[i + step] : 0u) : r.w[i];
    if constexpr (W == 2)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        r.w[i] = by & 1 ? r.w[i] >> 16 | (i < 3 ? r.w[i + 1] << 16 : 0u) : r.w[i];
  }
}
template <typename T, bool kVec>
__device__ __forceinline__ void store_vec(T* p, int n, const Vec& r) {
  if (n >= kE<T>) {
    if constexpr (kVec)
      *reinterpret_cast<uint4*>(p) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
    else
      __builtin_memcpy(p, r.w, 16);
  } else if constexpr (!kVec) {
#pragma unroll
    for (int i = 0; i < kE<T>; ++i)
      if (i < n) {
        if constexpr (sizeof(T) == 2)
          p[i] = __builtin_bit_cast(T, (uint16_t)(r.w[i / 2] >> (16 * (i & 1))));
        else
          p[i] = __builtin_bit_cast(T, r.w[i]);
      }
  }
}
// A vector's weights (zeros without p or past the row).
template <int E>
__device__ __forceinline__ void load_weights(const float* p, int n, float (&w)[E]) {
  if (p && n >= E) {
    __builtin_memcpy(w, p, sizeof w);
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) w[i] = p && i < n ? p[i] : 0.f;
  }
}

__device__ __forceinline__ float wave_sum(float v) { return wave_read_lane(wave_incl_scan(v), 63); }

// Sum of v over the TPR threads of a team, the same in each.  `s` holds one
// float a wave; teams of several waves must not use the same `s` in two sums
// one after the other.
template <int TPR>
__device__ __forceinline__ float team_sum(float v, float* s) {
  v = wave_sum(v);
  if constexpr (TPR > kWave) {
    const int wave = threadIdx.x / kWave, w0 = wave / (TPR / kWave) * (TPR / kWave);
    if ((threadIdx.x & 63) == 0) s[wave] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / kWave; ++i) v += s[w0 + i];
  }
  return v;
}

// Waves a SIMD that the forward kernel's registers allow (bfloat16 rows off the
// vectors' alignment in teams of 1024 spill one).  The launch has as
// many workgroups as that makes, each walking as many rows as the others: with
// more, those that find no place start when the rest is done (1000 x 4097
// float with the residual: 16.2 us for four a compute unit where two fit, 13.8
// for two; 1000 x 6001: 21.1 and 18.2).
template <typename T, int TPR, int NV, bool kVec>
constexpr int kNormWaves = NV == 1 ? (sizeof(T) == 2 && TPR == 512 && !kVec ? 6 : 8)
                           : TPR == 512 && NV == 2 ? 6
                           : sizeof(T) == 4 && NV == 2 && kVec ? 8 : 4;

template <typename T, int TPR, int NV, bool kVec, bool kCut>
__global__ void __launch_bounds__(TPR > 256 ? TPR : 256, (kNormWaves<T, TPR, NV, kVec>)) norm_kernel(NormArgs a) {
  constexpr int E = kE<T>, NT = TPR > 256 ? TPR : 256, kTeams = NT / TPR;
  __shared__ float s_sum[2][NT / kWave];
  const int t = threadIdx.x % TPR, team = threadIdx.x / TPR;
  const bool wide = !kCut && loads_whole<T>(a.D);
  const float inv = 1.f / (float)a.D;
  float w[NV][E], b[NV][E];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e0 = (j * TPR + t) * E;
    load_weights<E>(a.weight + e0, a.D - e0, w[j]);
    load_weights<E>(a.bias ? a.bias + e0 : nullptr, a.D - e0, b[j]);
  }
  // the next row is requested while this one is worked on, where the
  // registers hold both
  constexpr bool kAhead = NV == 1;
  const int64_t step = (int64_t)gridDim.x * kTeams;
  int64_t r = (int64_t)blockIdx.x * kTeams + team;
  Vec x[NV], res[NV], next_x[NV], next_res[NV];
  const auto request = [&](int64_t row, Vec(&p)[NV], Vec(&q)[NV]) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e0 = (j * TPR + t) * E, n = row < a.rows ? a.D - e0 : 0;
      p[j] = load_vec<T, kVec>(static_cast<const T*>(a.x) + row * a.ld_x + e0, n, wide);
      if (a.residual)
        q[j] = load_vec<T, kVec>(static_cast<const T*>(a.residual) + row * a.ld_res + e0, n, wide);
    }
  };
  if constexpr (kAhead) request(r, next_x, next_res);
  // every team makes the same number of rounds (they share the barriers)
  for (int64_t r0 = (int64_t)blockIdx.x * kTeams; r0 < a.rows; r0 += step, r += step) {
    if constexpr (kAhead) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        x[j] = next_x[j];
        res[j] = next_res[j];
      }
      request(r + step, next_x, next_res);
    } else {
      request(r, x, res);
    }
    float v[NV][E], sum = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int n = a.D - (j * TPR + t) * E;
      trim<T, kVec>(x[j], n, wide);
      unpack<T>(x[j], v[j]);
      if (a.residual) {
        float q[E];
        trim<T, kVec>(res[j], n, wide);
        unpack<T>(res[j], q);
#pragma unroll
        for (int i = 0; i < E; ++i) v[j][i] += q[i];
        x[j] = pack<T>(v[j]);
        unpack<T>(x[j], v[j]);  // the statistics are those of the stored sum
      }
#pragma unroll
      for (int i = 0; i < E; ++i) sum += v[j][i];
    }
    const float mean = team_sum<TPR>(sum, s_sum[0]) * inv;
    float sq = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int n = a.D - (j * TPR + t) * E;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const float c = v[j][i] - mean;
        v[j][i] = c;
        if (kVec ? n > 0 : i < n) sq = __builtin_fmaf(c, c, sq);
      }
    }
    const float rstd = 1.f / sqrtf(team_sum<TPR>(sq, s_sum[1]) * inv + a.eps);
    if (r >= a.rows) continue;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e0 = (j * TPR + t) * E;
      if (a.sum) store_vec<T, kVec>(static_cast<T*>(a.sum) + r * a.ld_sum + e0, a.D - e0, x[j]);
#pragma unroll
      for (int i = 0; i < E; ++i) v[j][i] = __builtin_fmaf(v[j][i] * rstd, w[j][i], b[j][i]);
      store_vec<T, kVec>(static_cast<T*>(a.y) + r * a.ld_y + e0, a.D - e0, pack<T>(v[j]));
    }
    if (t == 0) {
      if (a.mean) a.mean[r] = mean;
      if (a.rstd) a.rstd[r] = rstd;
    }
  }
}

constexpr int kBwThreads = 1024;
constexpr int kMaxGroups = 256;

// A row's inputs in the backward pass.
template <typename T, int NV>
struct BwRow {
  Vec s[NV], dy[NV], ds[NV];
  float mean, rstd;
};
template <typename T, int TPR, int NV, bool kVec, bool kCut>
__device__ __forceinline__ void load_bw(const NormArgs& a, int64_t r, int t, BwRow<T, NV>& q) {
  const bool wide = !kCut && loads_whole<T>(a.D);
  if (r >= a.rows) {  // a row of zeros adds nothing
#pragma unroll
    for (int j = 0; j < NV; ++j) q.s[j] = q.dy[j] = q.ds[j] = Vec{{0u, 0u, 0u, 0u}};
    q.mean = q.rstd = 0.f;
    return;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e0 = (j * TPR + t) * kE<T>, n = a.D - e0;
    q.s[j] = load_vec<T, kVec>(static_cast<const T*>(a.sum) + r * a.ld_sum + e0, n, wide);
    q.dy[j] = load_vec<T, kVec>(static_cast<const T*>(a.dy) + r * a.ld_dy + e0, n, wide);
    q.ds[j] = a.dsum ? load_vec<T, kVec>(static_cast<const T*>(a.dsum) + r * a.ld_dsum + e0, n, wide)
                     : Vec{{0u, 0u, 0u, 0u}};
  }
  q.mean = a.mean[r];
  q.rstd = a.rstd[r];
}

template <typename T, int TPR, int NV, bool kVec, bool kCut>
__global__ void __launch_bounds__(kBwThreads) norm_backward_kernel(NormArgs a, int rounds) {
  constexpr int E = kE<T>, kTeams = kBwThreads / TPR, C = TPR * NV * E;  // columns of a team
  __shared__ float s_p[2][kBwThreads / kWave], s_pq[2][kBwThreads / kWave];
  extern __shared__ __align__(16) float s_acc[];  // [teams][2][C] at the end
  const int t = threadIdx.x % TPR, team = threadIdx.x / TPR;
  const float inv = 1.f / (float)a.D;
  float w[NV][E], dw[NV][E], db[NV][E];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e0 = (j * TPR + t) * E;
    load_weights<E>(a.weight + e0, a.D - e0, w[j]);
#pragma unroll
    for (int i = 0; i < E; ++i) dw[j][i] = db[j][i] = 0.f;
  }
  // every team makes the same number of rounds (they share the barriers)
  const int64_t step = (int64_t)gridDim.x * kTeams;
  int64_t r = (int64_t)blockIdx.x * kTeams + team;
  // the next row is requested while this one is worked on, where the
  // registers hold both
  constexpr bool kAhead = NV == 1;
  BwRow<T, NV> cur, next;
  if constexpr (kAhead) load_bw<T, TPR, NV, kVec, kCut>(a, r, t, next);
  for (int k = 0; k < rounds; ++k, r += step) {
    if constexpr (kAhead) {
      cur = next;
      load_bw<T, TPR, NV, kVec, kCut>(a, k + 1 < rounds ? r + step : a.rows, t, next);
    } else {
      load_bw<T, TPR, NV, kVec, kCut>(a, r, t, cur);
    }
    float q[NV][E], g[NV][E], sp = 0.f, spq = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int n = a.D - (j * TPR + t) * E;
      trim<T, kVec>(cur.s[j], n, !kCut && loads_whole<T>(a.D));
      trim<T, kVec>(cur.dy[j], n, !kCut && loads_whole<T>(a.D));
      trim<T, kVec>(cur.ds[j], n, !kCut && loads_whole<T>(a.D));
      unpack<T>(cur.s[j], q[j]);
      unpack<T>(cur.dy[j], g[j]);
#pragma unroll
      for (int i = 0; i < E; ++i) {
        q[j][i] = (q[j][i] - cur.mean) * cur.rstd;  // past the row dy and the weight are 0
        dw[j][i] = __builtin_fmaf(g[j][i], q[j][i], dw[j][i]);
        db[j][i] += g[j][i];
        g[j][i] *= w[j][i];
        sp += g[j][i];
        spq = __builtin_fmaf(g[j][i], q[j][i], spq);
      }
    }
    sp = wave_sum(sp);
    spq = wave_sum(spq);
    if constexpr (TPR > kWave) {
      const int wave = threadIdx.x / kWave, w0 = wave / (TPR / kWave) * (TPR / kWave);
      if ((threadIdx.x & 63) == 0) {
        s_p[k & 1][wave] = sp;
        s_pq[k & 1][wave] = spq;
      }
      __syncthreads();
      sp = spq = 0.f;
#pragma unroll
      for (int i = 0; i < TPR / kWave; ++i) {
        sp += s_p[k & 1][w0 + i];
        spq += s_pq[k & 1][w0 + i];
      }
    }
    const float mp = sp * inv, mpq = spq * inv;
    if (r < a.rows) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int e0 = (j * TPR + t) * E;
        float v[E];
#pragma unroll
        for (int i = 0; i < E; ++i)
          v[i] = cur.rstd * (g[j][i] - mp - q[j][i] * mpq);
        if (a.dsum) {
          float d[E];
          unpack<T>(cur.ds[j], d);
#pragma unroll
          for (int i = 0; i < E; ++i) v[i] += d[i];
        }
        store_vec<T, kVec>(static_cast<T*>(a.dx) + r * a.ld_dx + e0, a.D - e0, pack<T>(v));
      }
    }
  }
  // the teams' sums, in the order of the teams
  float* out = a.partial + (int64_t)blockIdx.x * 2 * a.D;
  if constexpr (kTeams > 1) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < E; ++i) {
        s_acc[(team * 2) * C + (j * TPR + t) * E + i] = dw[j][i];
        s_acc[(team * 2 + 1) * C + (j * TPR + t) * E + i] = db[j][i];
      }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * C; c += kBwThreads) {
      float v = 0.f;
#pragma unroll
      for (int m = 0; m < kTeams; ++m) v += s_acc[m * 2 * C + c];
      if (c % C < a.D) out[c / C * a.D + c % C] = v;
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int c = (j * TPR + t) * E + i;
        if (c < a.D) {
          out[c] = dw[j][i];
          out[a.D + c] = db[j][i];
        }
      }
  }
}

// dweight and dbias from the groups' partials: 32 columns a workgroup, the
// groups dealt to its 32 half waves, 8 in flight a thread, joined in a fixed
// order.
__global__ void __launch_bounds__(1024) norm_weights_kernel(NormArgs a, int groups) {
  constexpr int kCols = 32, kParts = 1024 / kCols, kFly = kMaxGroups / kParts;
  __shared__ float s_part[kParts][kCols];
  const int col = threadIdx.x % kCols, part = threadIdx.x / kCols;
  const int64_t c = (int64_t)blockIdx.x * kCols + col;  // of 2 D
  float v[kFly], sum = 0.f;
#pragma unroll
  for (int i = 0; i < kFly; ++i) {
    const int g = i * kParts + part;
    v[i] = c < 2 * (int64_t)a.D && g < groups ? a.partial[(int64_t)g * 2 * a.D + c] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < kFly; ++i) sum += v[i];
  s_part[part][col] = sum;
  __syncthreads();
  if (part == 0 && c < 2 * (int64_t)a.D) {
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < kParts; ++i) sum += s_part[i][col];
    if (c < a.D) a.dweight[c] = sum;
    else if (a.dbias) a.dbias[c - a.D] = sum;
  }
}

bool vec16(const void* p, int64_t ld, size_t es) {
  return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (size_t)ld * es % 16 == 0);
}

template <typename T, int TPR, int NV, bool kVec, bool kCut>
hipError_t launch_fwd_v(const NormArgs& a, hipStream_t stream) {
  constexpr int NT = TPR > 256 ? TPR : 256, kTeams = NT / TPR;
  const int64_t most = 256 * (kNormWaves<T, TPR, NV, kVec> * 4 * kWave / NT);
  const dim3 grid((unsigned)std::min<int64_t>((a.rows + kTeams - 1) / kTeams, most));
  hipLaunchKernelGGL((norm_kernel<T, TPR, NV, kVec, kCut>), grid, dim3(NT), 0, stream, a);
  return hipGetLastError();
}
template <typename T, int TPR, int NV>
hipError_t launch_fwd(const NormArgs& a, bool vec, hipStream_t stream) {
  if (vec) return launch_fwd_v<T, TPR, NV, true, false>(a, stream);
  if constexpr (sizeof(T) == 2)
    if (!loads_whole<T>(a.D)) return launch_fwd_v<T, TPR, NV, false, true>(a, stream);
  return launch_fwd_v<T, TPR, NV, false, false>(a, stream);
}

// The team for a row of `vecs` vectors: one a thread up to 1024; wide float
// rows two or three a thread in teams of 512, so that four rows are under way
// in a compute unit instead of two (1003 x 4097: 10.4 us against 12.8, 1003 x
// 4096: 8.8 against 9.6, 8192 x 4096 with the residual: 98.3 against 98.7).
// Not for bfloat16, whose vectors hold twice as many weights (1000 x 8192: 17.5
// against 16.6 us, 256 x 8192: 6.3 against 5.7; 8192 x 8192: 97 against 102).
template <typename T>
hipError_t launch_fwd_t(const NormArgs& a, hipStream_t stream) {
  constexpr size_t es = sizeof(T);
  const bool vec = a.D % kE<T> == 0 && vec16(a.x, a.ld_x, es) && vec16(a.residual, a.ld_res, es) &&
                   vec16(a.sum, a.ld_sum, es) && vec16(a.y, a.ld_y, es);
  const int vecs = (a.D + kE<T> - 1) / kE<T>;
  if (vecs <= 64) return launch_fwd<T, 64, 1>(a, vec, stream);
  if (vecs <= 128) return launch_fwd<T, 128, 1>(a, vec, stream);
  if (vecs <= 256) return launch_fwd<T, 256, 1>(a, vec, stream);
  if (vecs <= 512) return launch_fwd<T, 512, 1>(a, vec, stream);
  if constexpr (sizeof(T) == 4) {
    if (vecs <= 1024) return launch_fwd<T, 512, 2>(a, vec, stream);
    if (vecs <= 1536) return launch_fwd<T, 512, 3>(a, vec, stream);
  } else {
    if (vecs <= 1024) return launch_fwd<T, 1024, 1>(a, vec, stream);
  }
  if (vecs <= 2048) return launch_fwd<T, 1024, 2>(a, vec, stream);
  if constexpr (sizeof(T) == 4) return launch_fwd<T, 1024, 4>(a, vec, stream);
  return hipErrorInvalidValue;
}

template <typename T, int TPR, int NV, bool kVec, bool kCut>
hipError_t launch_bw_v(const NormArgs& a, int groups, hipStream_t stream) {
  constexpr int kTeams = kBwThreads / TPR;
  const size_t lds = kTeams > 1 ? sizeof(float) * (size_t)kTeams * 2 * TPR * NV * kE<T> : 0;
  const hipError_t e = lds_limit(reinterpret_cast<const void*>(&norm_backward_kernel<T, TPR, NV, kVec, kCut>), lds);
  if (e != hipSuccess) return e;
  const int64_t step = (int64_t)groups * kTeams;
  const int rounds = (int)((a.rows + step - 1) / step);
  hipLaunchKernelGGL((norm_backward_kernel<T, TPR, NV, kVec, kCut>), dim3(groups), dim3(kBwThreads), lds,
                     stream, a, rounds);
  return hipGetLastError();
}
template <typename T, int TPR, int NV>
hipError_t launch_bw(const NormArgs& a, bool vec, int groups, hipStream_t stream) {
  if (vec) return launch_bw_v<T, TPR, NV, true, false>(a, groups, stream);
  if constexpr (sizeof(T) == 2)
    if (!loads_whole<T>(a.D)) return launch_bw_v<T, TPR, NV, false, true>(a, groups, stream);
  return launch_bw_v<T, TPR, NV, false, false>(a, groups, stream);
}

template <typename T>
hipError_t launch_bw_t(const NormArgs& a, int groups, hipStream_t stream) {
  constexpr size_t es = sizeof(T);
  const bool vec = a.D % kE<T> == 0 && vec16(a.sum, a.ld_sum, es) && vec16(a.dy, a.ld_dy, es) &&
                   vec16(a.dsum, a.ld_dsum, es) && vec16(a.dx, a.ld_dx, es);
  const int vecs = (a.D + kE<T> - 1) / kE<T>;
  if (vecs <= 64) return launch_bw<T, 64, 1>(a, vec, groups, stream);
  if (vecs <= 128) return launch_bw<T, 128, 1>(a, vec, groups, stream);
  if (vecs <= 256) return launch_bw<T, 256, 1>(a, vec, groups, stream);
  if (vecs <= 512) return launch_bw<T, 512, 1>(a, vec, groups, stream);
  if (vecs <= 1024) return launch_bw<T, 1024, 1>(a, vec, groups, stream);
  if (vecs <= 2048) return launch_bw<T, 1024, 2>(a, vec, groups, stream);
  if constexpr (sizeof(T) == 4) return launch_bw<T, 1024, 4>(a, vec, groups, stream);
  return hipErrorInvalidValue;
}

// Teams of a backward workgroup for rows of D channels (the table above).
int bw_teams(int D, int esize) {
  const int e = 16 / esize, vecs = (D + e - 1) / e;
  return vecs <= 64 ? 16 : vecs <= 128 ? 8 : vecs <= 256 ? 4 : vecs <= 512 ? 2 : 1;
}

}  // namespace

int norm_backward_groups(int64_t rows, int D, int esize) {
  const int teams = bw_teams(D, esize);
  return (int)std::min<int64_t>((rows + teams - 1) / teams, kMaxGroups);
}

hipError_t launch_norm(const NormArgs& a, m3_dtype dtype, hipStream_t stream) {
  return dtype == M3_BF16 ? launch_fwd_t<bf16>(a, stream) : launch_fwd_t<float>(a, stream);
}

hipError_t launch_norm_backward(const NormArgs& a, m3_dtype dtype, hipStream_t stream) {
  const int groups = norm_backward_groups(a.rows, a.D, dtype == M3_BF16 ? 2 : 4);
  if (groups > 0) {
    const hipError_t e = dtype == M3_BF16 ? launch_bw_t<bf16>(a, groups, stream)
                                          : launch_bw_t<float>(a, groups, stream);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(norm_weights_kernel, dim3((2 * a.D + 31) / 32), dim3(1024), 0, stream,
                     a, groups);
  return hipGetLastError();
}

}  // namespace m3
