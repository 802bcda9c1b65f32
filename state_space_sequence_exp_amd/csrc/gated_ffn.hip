// gated_ffn.hip -- gated feed-forward projections, h = silu(x Wg^T) * (x Wu^T),
// and their gradients
//
//   du = dh silu(g), dg = dh u silu'(g),  dx = dg Wg + du Wu,
//   dWg = dg^T x, dWu = du^T x
//
// The products run on one kernel: C[m][n] = sum_k A(m, k) B(n, k), tile by tile
// through the LDS.  Forward, k is contiguous in both operands, and the B rows of a wave
// are its hidden units' rows of Wg, then of Wu, so that a lane ends with g and u of the
// same elements and the activation costs no memory.  Backward, one pass over dh, g and
// u writes [dg | du]; for dx the weights are read as they lie, k by k, for their own
// gradients [dg | du] and x are: such a tile lies in the LDS as it does in memory and
// is turned as its fragments are read.  (Transposed copies instead take 80 us more of
// 8192 x 2048 x 3824 in bfloat16, forward and gradients, which take 719; in float, 777 x
// 514 x 1001, 8 us less of 86.)
//
// Bound by the matrix units at the rate that the chip's power leaves them: 16384 x 2048
// x 4096 bfloat16 407 us, 1350 TFLOP/s (a product of that size alone, by the library,
// 1370 to 1470), the largest tile's waves reading their fragments of the next half tile
// from the LDS between the matrix instructions of this one (those of 32 x 32 take as many
// cycles at a lower clock, 8% more time); float 145 of 155 TFLOP/s.  A few rows are bound
// by the weights' bytes (few_kernel).
//
// (dg and du are rounded to the storage type, as the matrix units take it; g and u
// are kept in float, or each gradient would carry their rounding as well: 0.0031
// relative in bfloat16 instead of 0.0024, where rounding the result alone is 0.0017.)
#include <type_traits>

#include "ffn_plan.h"
#include "gate.h"
#include "layer_internal.h"
#include "vec_io.h"

namespace m3 {
namespace {

constexpr int kRowBytes = kPlanRowBytes, kChunks = kRowBytes / 16;  // of k in a tile's row

// ---- matrix products ---------------------------------------------------------

template <typename T>
struct GemmArgs {
  int M, N, K;                 // N: hidden units (dual), columns of C otherwise
  const T *A, *B, *B2;         // B2: the second weight matrix (dual, inputs)
  int64_t lda, ldb, ldb2;
  T* C;
  float *gate, *up;            // dual: g and u, unless null
  int64_t ldc, ld_gate, ld_up;
  T* C2;                       // weights: where A's columns from `split` on go
  int64_t ldc2;
  int split, rows;             // inputs, weights: each half of [dg | du] is `split` wide, `rows` of it used
  int parts, each;             // inputs, weights: k is cut into `parts` of `each`, and where they are more
  float* part;                 // than one their sums go to part [parts, M, N]
  const T* zeros;              // 16 bytes of them (inputs, weights)
  int gridM, gridN;
};
// dual: x by both weights.  inputs: [dg | du] by the weights one above the other.
// weights: [dg | du] by x, k over the rows of both.
enum Mode { kDual, kInputs, kWeights };

// acc[n 4g..4g+3][m l%16] += sum over the chunks' k: a lane's 16 bytes of a row are
// 8 bfloat16 or 4 float k, any order of k being the same for both operands.
__device__ __forceinline__ f32x4 mma_chunk(u32x4 n, u32x4 m, f32x4 c, bf16) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, n), __builtin_bit_cast(bf16x8, m), c,
                                                 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma_chunk(u32x4 n, u32x4 m, f32x4 c, float) {
  const f32x4 a = __builtin_bit_cast(f32x4, n), b = __builtin_bit_cast(f32x4, m);
#pragma unroll
  for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
  return c;
}

template <typename T>
__device__ __forceinline__ u32x4 load_chunk(const T* p, int n) {
  return __builtin_bit_cast(u32x4, load_run<T, 16 / (int)sizeof(T)>(p, n));
}

// A tile's row is 128 bytes of k (a cache line: rows of 64 bytes take twice the
// requests), its 16-byte chunks permuted by the row so that eight rows read together
// lie on different banks.
__device__ __forceinline__ int chunk_at(int row, int chunk) { return row * kChunks + (chunk ^ (row & 7)); }

// 16 bytes a lane from base + off (elements of T) straight into the LDS, lane
// after lane from byte address `lds` on.  The compiler does not know of the write:
// wait_loads, then a barrier, come before any read of it.  (Its own load to the LDS
// it waits for whole before the next read of any LDS array.)
template <typename T>
__device__ __forceinline__ void load_to_lds(uint32_t lds, const T* base, uint32_t off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "s"(lds), "v"(off * (uint32_t)sizeof(T)), "s"(base)
               : "memory", "m0");
}
// The same from an address of each lane's own.
template <typename T>
__device__ __forceinline__ void load_to_lds_from(uint32_t lds, const T* p) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" : : "s"(lds), "v"(p) : "memory", "m0");
}
// Until at most n of this wave's loads are outstanding.
template <int n>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(n) : "memory");
}

// A tile of an operand whose rows are k and whose columns are the product's R rows or
// columns from col0 on: BK rows of R elements, as they lie in memory but for units of
// 32 bytes (float: 64) permuted by the row, so that what a fragment reads from several
// rows at once lies on different banks.
template <typename T, int R, int NT>
struct TurnedTile {
  static constexpr int E = 16 / (int)sizeof(T), BK = kRowBytes / (int)sizeof(T);
  static constexpr int kRow = R * (int)sizeof(T), kAcross = kRow / 16;    // a row's bytes, its chunks
  static constexpr int kPass = NT * 16 / kRow, kPasses = BK / kPass;      // rows at once
  static_assert(kPasses * kPass == BK && kPass % 8 == 0, "passes are whole, and alike to the permutation");
  // The permutation of a row's units, for a chunk of it.
  __device__ __forceinline__ static int permuted(int k, int chunk) {
    if constexpr (sizeof(T) == 4) return (((chunk >> 2) ^ ((k >> 2) & 1)) << 2) | (chunk & 3);
    return (((chunk >> 1) ^ (kAcross >= 8 ? k & 3 : (k >> 1) & 1)) << 1) | (chunk & 1);
  }
  int k, col;  // of this thread's first chunk

  __device__ __forceinline__ TurnedTile(int tid, int col0) {
    k = tid / kAcross;
    col = col0 + permuted(k, tid % kAcross) * E;
  }
  // Where this thread's chunks lie, from the tile's first row on, rows being ld elements
  // apart; columns past the end, whole chunks, stand for the last.
  __device__ __forceinline__ void offsets(uint32_t (&off)[kPasses], uint32_t ld, int cols) const {
#pragma unroll
    for (int i = 0; i < kPasses; ++i) off[i] = (i * kPass + k) * ld + min(col, cols - E);
  }
  // The rows of the matrix at p, `left` of them, straight into the LDS at byte `lds` (this
  // wave's); the rows behind them are zeros, from 16 bytes of them in memory (so that
  // every tile is as many loads).
  __device__ __forceinline__ void bring(uint32_t lds, const T* p, const uint32_t (&off)[kPasses], int left,
                                        const T* zeros) const {
    if (left >= BK) {
#pragma unroll
      for (int i = 0; i < kPasses; ++i) load_to_lds(lds + i * kPass * kRow, p, off[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kPasses; ++i)
        load_to_lds_from(lds + i * kPass * kRow, i * kPass + k < left ? p + off[i] : zeros);
    }
  }
  // Fragment f (columns 16 f on) of half a tile's rows.  bfloat16: a lane names 8 bytes,
  // four columns of row l16 / 4 of its group's eight, and gets its own column's four
  // rows; twice.  float: four rows' elements.
  __device__ __forceinline__ static u32x4 get(const u32x4* tile, int f, int half, int l16, int l4) {
    const char* s = reinterpret_cast<const char*>(tile);
    if constexpr (sizeof(T) == 2) {
      typedef short s16x4 __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) s16x4* Lds;
      const int r = l16 >> 2, k0 = half * 32 + 8 * l4 + r;
      const char* at = s + k0 * kRow + (f ^ (kAcross >= 8 ? r & 3 : (r >> 1) & 1)) * 32 + (l16 & 3) * 8;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)at);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(at + 4 * kRow));
      const uint2 a = __builtin_bit_cast(uint2, lo), b = __builtin_bit_cast(uint2, hi);
      return u32x4{a.x, a.y, b.x, b.y};
    } else {
      const char* at = s + (half * 16 + 4 * l4) * kRow + (f ^ (l4 & 1)) * 64 + l16 * 4;
      u32x4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = *reinterpret_cast<const uint32_t*>(at + e * kRow);
      return v;
    }
  }
  static constexpr int kReads = sizeof(T) == 2 ? 2 : 4;  // LDS reads a fragment
};

// kDirect: rows of both operands start at multiples of 4 bytes; their tiles go straight
// into the LDS, as many ahead as its stages hold (two of the largest tile, four of the
// small ones, whose products take less than a load does).  Otherwise (dual) they pass
// through registers, two ahead.
template <typename T, int WM, int WN, int FM, int FN, Mode kMode, bool kDirect>
__global__ void __launch_bounds__(WM* WN* kWave) __attribute__((amdgpu_waves_per_eu(2, 2)))
gemm_kernel(GemmArgs<T> g) {
  constexpr int NT = WM * WN * kWave, BM = WM * FM * 16, BN = WN * FN * 16, E = 16 / (int)sizeof(T);
  constexpr int BK = kRowBytes / (int)sizeof(T), kPass = NT / kChunks;  // rows a pass loads
  constexpr int NA = BM / kPass, NB = BN / kPass, kStages = kDirect && BM + BN <= 128 ? 4 : 2;
  __shared__ u32x4 s_tile[kStages][(BM + BN) * kChunks];
  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, l4 = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave / WN, wn = wave % WN;

  // Neighbouring tiles on one XCD; eight rows of tiles side by side, so that a
  // chip's worth of tiles shares few rows of both operands.
  const int groups = (int)gridDim.x, x = blockIdx.x & 7, q = groups >> 3, rest = groups & 7;
  int at = x * q + min(x, rest) + (int)(blockIdx.x >> 3);
  int part = 0;
  if constexpr (kMode != kDual) {
    part = at / (g.gridM * g.gridN);
    at -= part * g.gridM * g.gridN;
    g.A += (int64_t)part * g.each * (kMode == kWeights ? g.lda : 1);
    if constexpr (kMode == kWeights) g.B += (int64_t)part * g.each * g.ldb;
    g.K = min(g.each, g.K - part * g.each);
    g.part += (int64_t)part * g.M * g.N;
  }
  const int band = at / (8 * g.gridN), inBand = at - band * 8 * g.gridN, high = min(8, g.gridM - band * 8);
  const int m0 = (band * 8 + inBand % high) * BM;
  const int n0 = inBand / high * (kMode == kDual ? BN / 2 : BN);

  constexpr bool kTurnA = kMode == kWeights, kTurnB = kMode != kDual;
  // What this thread brings of an operand with k contiguous: one chunk of every kPass-th
  // row, rows past the end standing for the last.  Straight loads put lane after lane,
  // so that it is the lane's chunk of memory that is permuted.
  const int row = tid / kChunks;
  const int chunk = kDirect ? (tid % kChunks) ^ (row & 7) : tid % kChunks;
  const T* const baseA = g.A + (kTurnA ? 0 : (int64_t)m0 * g.lda);
  uint32_t offA[NA], offB[NB];
  if constexpr (!kTurnA) {
#pragma unroll
    for (int i = 0; i < NA; ++i)
      offA[i] = (uint32_t)min(i * kPass + row, g.M - 1 - m0) * (uint32_t)g.lda + chunk * E;
  }
  // (whether a wave's rows of pass i are the second matrix's)
  const auto second = [&](int i) { return (i * kPass + wave * (kWave / kChunks)) % (FN * 16) >= FN * 8; };
  const T* const base1 = g.B + (kTurnB ? 0 : (int64_t)n0 * g.ldb);
  const T* const base2 = kMode == kDual ? g.B2 + (int64_t)n0 * g.ldb2 : g.B2;
  const auto baseB = [&](int i) { return second(i) ? base2 : base1; };
  if constexpr (!kTurnB) {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int r = i * kPass + row, col = r / (FN * 16) * FN * 8 + r % (FN * 8);
      offB[i] = (uint32_t)min(col, g.N - 1 - n0) * (uint32_t)(second(i) ? g.ldb2 : g.ldb) + chunk * E;
    }
  }
  // ... and of operands read k by k.
  const TurnedTile<T, BM, NT> turnA(tid, m0);
  const TurnedTile<T, BN, NT> turnB(tid, n0);
  uint32_t turnedA[NA], turnedB[NB], turnedB2[NB];
  const int colsB = (g.N + E - 1) / E * E;
  if constexpr (kTurnA) turnA.offsets(turnedA, (uint32_t)g.lda, 2 * g.split);
  if constexpr (kTurnB) turnB.offsets(turnedB, (uint32_t)g.ldb, colsB);
  if constexpr (kMode == kInputs) turnB.offsets(turnedB2, (uint32_t)g.ldb2, colsB);

  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  struct Frags {
    u32x4 a[FM], b[FN];
  };
  const int get_at[2] = {chunk_at(l16, l4), chunk_at(l16, 4 + l4)};
  const auto get = [&](Frags& f, int stage, int half) {  // of a tile's 128 bytes of k
    const u32x4* s = s_tile[stage];
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      if constexpr (kTurnB) f.b[j] = turnB.get(s + BM * kChunks, wn * FN + j, half, l16, l4);
      else f.b[j] = s[get_at[half] + (BM + (wn * FN + j) * 16) * kChunks];
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      if constexpr (kTurnA) f.a[i] = turnA.get(s, wm * FM + i, half, l16, l4);
      else f.a[i] = s[get_at[half] + (wm * FM + i) * 16 * kChunks];
    }
  };
  const auto multiply = [&](const Frags& f) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = mma_chunk(f.b[j], f.a[i], acc[i][j], T());
  };
  struct Moved {  // through registers
    u32x4 a[NA], b[NB];
  };
  const auto request = [&](Moved& r, int k0) {
    const int n = g.K - k0 - chunk * E;  // elements from this thread's chunk to the row's end
#pragma unroll
    for (int i = 0; i < NA; ++i) r.a[i] = load_chunk<T>(baseA + k0 + offA[i], n);
#pragma unroll
    for (int i = 0; i < NB; ++i) r.b[i] = load_chunk<T>(baseB(i) + k0 + offB[i], n);
  };
  const int put_at = chunk_at(row, chunk);  // (kPass is a multiple of 8)
  const auto put = [&](const Moved& r, int stage) {
    u32x4* const s = s_tile[stage];
#pragma unroll
    for (int i = 0; i < NA; ++i) s[put_at + i * kPass * kChunks] = r.a[i];
#pragma unroll
    for (int i = 0; i < NB; ++i) s[put_at + (BM + i * kPass) * kChunks] = r.b[i];
  };

  int done = 0;  // tiles multiplied
  if constexpr (kDirect) {
    // (read k by k, a last tile of fewer rows is filled with zeros)
    const int whole = kTurnB ? (g.K + BK - 1) / BK : g.K / BK;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) u32x4*)&s_tile[0][0];
    const uint32_t lds = __builtin_amdgcn_readfirstlane(lds0 + wave * (kWave * 16));
    const auto bring = [&](int t) {
      const int last = min(t, whole - 1);
      const uint32_t to = lds + (t & (kStages - 1)) * (uint32_t)sizeof s_tile[0];
      const int k0 = last * BK;  // (past the end: a tile again, into a stage that no one reads)
      if constexpr (kTurnA) {
        turnA.bring(to, baseA + k0 * g.lda, turnedA, g.K - k0, g.zeros);
      } else {
#pragma unroll
        for (int i = 0; i < NA; ++i) load_to_lds(to + i * kPass * kRowBytes, baseA + k0, offA[i]);
      }
      const uint32_t toB = to + BM * kRowBytes;
      if constexpr (kMode == kInputs) {  // (a half of [dg | du] is whole tiles wide)
        const int k = part * g.each + k0;
        if (k < g.split) turnB.bring(toB, base1 + k * g.ldb, turnedB, g.rows - k, g.zeros);
        else turnB.bring(toB, base2 + (k - g.split) * g.ldb2, turnedB2, g.rows - (k - g.split), g.zeros);
      } else if constexpr (kMode == kWeights) {
        turnB.bring(toB, base1 + k0 * g.ldb, turnedB, g.K - k0, g.zeros);
      } else {
#pragma unroll
        for (int i = 0; i < NB; ++i) load_to_lds(toB + i * kPass * kRowBytes, baseB(i) + k0, offB[i]);
      }
    };
    // the fragments' reads one by one between the products
    const auto order = [] {
      constexpr int kReads = FM * (kTurnA ? TurnedTile<T, BM, NT>::kReads : 1) +
                             FN * (kTurnB ? TurnedTile<T, BN, NT>::kReads : 1);
      constexpr int kProducts = FM * FN * (sizeof(T) == 2 ? 1 : 4);
      constexpr int kEach = kProducts < kReads ? 1 : kProducts / kReads;
#pragma unroll
      for (int i = 0; i < kReads; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, kEach, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    if (whole > 0) {
#pragma unroll
      for (int t = 0; t < kStages; ++t) bring(t);
      wait_loads<(kStages - 1) * (NA + NB)>();
      lds_barrier();
      Frags f0, f1;
      get(f0, 0, 0);
      for (; done < whole; ++done) {
        __builtin_amdgcn_sched_barrier(0);
        get(f1, done & (kStages - 1), 1);
        multiply(f0);
        order();
        wait_loads<(kStages - 2) * (NA + NB)>();  // the next tile has come, and every wave has read this one
        lds_barrier();
        bring(done + kStages);
        __builtin_amdgcn_sched_barrier(0);
        get(f0, (done + 1) & (kStages - 1), 0);
        multiply(f1);
        order();
      }
      wait_loads<0>();
      lds_barrier();
    }
    if (kMode == kDual && done * BK < g.K) {
      Moved r;
      request(r, done * BK);
      put(r, 0);
      lds_barrier();
      Frags rest;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        get(rest, 0, half);
        multiply(rest);
      }
    }
  } else {
    Moved next, later;
    request(next, 0);
    request(later, BK);
    for (int k0 = 0; k0 < g.K; k0 += BK, done ^= 1) {
      put(next, done);
      lds_barrier();
      next = later;
      request(later, k0 + 2 * BK);
      Frags f;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        get(f, done, half);
        multiply(f);
      }
    }
  }

#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int m = m0 + (wm * FM + i) * 16 + l16;
    if (m >= g.M) continue;
    if constexpr (kMode == kDual) {
#pragma unroll
      for (int j = 0; j < FN / 2; ++j) {
        const int n = n0 + (wn * (FN / 2) + j) * 16 + 4 * l4, left = g.N - n;
        if (left <= 0) continue;
        float gv[4], uv[4], hv[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          gv[e] = acc[i][j][e];
          uv[e] = acc[i][j + FN / 2][e];
          hv[e] = gv[e] * sigmoid_of(gv[e]) * uv[e];
        }
        store_run<T, 4>(g.C + (int64_t)m * g.ldc + n, left, to_run<T, 4>(hv));
        if (g.gate) {
          store_for_later(g.gate + (int64_t)m * g.ld_gate + n, left, gv);
          store_for_later(g.up + (int64_t)m * g.ld_up + n, left, uv);
        }
      }
    } else {
      T* c = g.C + (int64_t)m * g.ldc;
      if constexpr (kMode == kWeights) {
        const bool second = m >= g.split;
        const int r = second ? m - g.split : m;
        if (r >= g.rows) continue;
        if (second) c = g.C2 + (int64_t)r * g.ldc2;
      }
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int n = n0 + (wn * FN + j) * 16 + 4 * l4, left = g.N - n;
        if (left <= 0) continue;
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = acc[i][j][e];
        if (g.parts > 1)
          store_run<float, 4>(g.part + (int64_t)m * g.N + n, left, to_run<float, 4>(v));
        else
          store_run<T, 4>(c + n, left, to_run<T, 4>(v));
      }
    }
  }
}

// C = the sum of the parts, in order.
template <typename T, Mode kMode>
__global__ void __launch_bounds__(256) join_kernel(GemmArgs<T> g) {
  const int64_t all = (int64_t)g.M * g.N;
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < all; i += (int64_t)gridDim.x * 1024) {
    const int n = (int)min((int64_t)4, all - i);
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    for (int p = 0; p < g.parts; ++p) {
      const Raw<float, 4> r = load_run<float, 4>(g.part + p * all + i, n);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += run_at(r, e);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      int64_t row = (i + e) / g.N;
      const int64_t col = (i + e) - row * g.N;
      T* c = g.C;
      int64_t ld = g.ldc;
      if constexpr (kMode == kWeights) {
        if (row >= g.split) {
          row -= g.split;
          c = g.C2;
          ld = g.ldc2;
        }
        if (row >= g.rows) continue;
      }
      if (e < n) c[row * ld + col] = from_f32<T>(v[e]);
    }
  }
}

template <typename T, int WM, int WN, int FM, int FN, Mode kMode>
void launch_gemm_tile(GemmArgs<T> g, bool direct, hipStream_t stream) {
  constexpr int BM = WM * FM * 16, BN = WN * FN * 16 / (kMode == kDual ? 2 : 1);
  g.gridM = (g.M + BM - 1) / BM;
  g.gridN = (g.N + BN - 1) / BN;
  const dim3 grid((unsigned)g.gridM * g.gridN * g.parts), block(WM * WN * kWave);
  if constexpr (kMode == kDual && sizeof(T) == 2)  // (float rows are aligned, the others' are made so)
    if (!direct) {
      hipLaunchKernelGGL((gemm_kernel<T, WM, WN, FM, FN, kMode, false>), grid, block, 0, stream, g);
      return;
    }
  hipLaunchKernelGGL((gemm_kernel<T, WM, WN, FM, FN, kMode, true>), grid, block, 0, stream, g);
}
bool rows4(const void* p, int64_t ld, int es) {
  return reinterpret_cast<uintptr_t>(p) % 4 == 0 && ld * es % 4 == 0;
}
template <typename T, Mode kMode>
void launch_gemm(GemmArgs<T> g, hipStream_t stream) {
  constexpr int es = (int)sizeof(T);
  const bool direct =
      kMode != kDual || (rows4(g.A, g.lda, es) && rows4(g.B, g.ldb, es) && rows4(g.B2, g.ldb2, es));
  const Plan plan = plan_gemm(g.M, (kMode == kDual ? 2 : 1) * (int64_t)g.N, g.K, (int)sizeof(T), kMode != kDual);
  g.parts = plan.parts;
  g.each = plan.each;
  if (plan.tile == 0) {
    if constexpr (sizeof(T) == 2) launch_gemm_tile<T, 2, 4, 8, 4, kMode>(g, direct, stream);
  } else if (plan.tile == 1) {
    launch_gemm_tile<T, 2, 2, 4, 4, kMode>(g, direct, stream);
  } else if (plan.tile == 2) {
    launch_gemm_tile<T, 2, 2, 2, 2, kMode>(g, direct, stream);
  } else {
    launch_gemm_tile<T, 2, 2, 1, 2, kMode>(g, direct, stream);
  }
  if constexpr (kMode != kDual)
    if (g.parts > 1) {
      const int64_t quads = ((int64_t)g.M * g.N + 3) / 4, groups = (quads + 255) / 256;
      hipLaunchKernelGGL((join_kernel<T, kMode>), dim3((unsigned)(groups < 2048 ? groups : 2048)), dim3(256), 0, stream, g);
    }
}

// ---- few rows ------------------------------------------------------------------
// Up to 16 FM rows (a decode batch): the weights are read once, straight into the
// matrix units' layout (4 x 2048 x 4096 bfloat16: 7 us, 4.8 TB/s, 16 rows 8.0, 32 rows
// 10.0, on inputs that the caches hold; 33 rows, in tiles, take 8.1, but 40 beside 36 of
// 4096 x 64 in float).  A workgroup owns 16 hidden units; its eight waves share
// out k and add their parts in the LDS, in order.
constexpr int kFewWaves = 8;

template <typename T, int FM>
__global__ void __launch_bounds__(kFewWaves * kWave) few_kernel(GemmArgs<T> g) {
  constexpr int E = 16 / (int)sizeof(T), KS = 4 * E;  // k of a step
  __shared__ f32x4 s_part[kFewWaves][2 * FM][kWave];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l16 = lane & 15, l4 = lane >> 4;
  const int n0 = blockIdx.x * 16;
  const T* pg = g.B + (int64_t)min(n0 + l16, g.N - 1) * g.ldb;
  const T* pu = g.B2 + (int64_t)min(n0 + l16, g.N - 1) * g.ldb2;
  const T* px[FM];
#pragma unroll
  for (int i = 0; i < FM; ++i) px[i] = g.A + (int64_t)min(i * 16 + l16, g.M - 1) * g.lda;
  const int steps = (g.K + KS - 1) / KS, each = (steps + kFewWaves - 1) / kFewWaves;
  const int s0 = wave * each, s1 = min(s0 + each, steps);
  f32x4 acc[FM][2];
#pragma unroll
  for (int i = 0; i < FM; ++i) acc[i][0] = acc[i][1] = f32x4{0.f, 0.f, 0.f, 0.f};
  const auto some = [&](auto count, int s) {
    constexpr int U = decltype(count)::value;
    u32x4 wg[U], wu[U], xv[U][FM];
#pragma unroll
    for (int v = 0; v < U; ++v) {
      const int k = (s + v) * KS + l4 * E, n = g.K - k;
      wg[v] = load_chunk<T>(pg + k, n);
      wu[v] = load_chunk<T>(pu + k, n);
#pragma unroll
      for (int i = 0; i < FM; ++i) xv[v][i] = load_chunk<T>(px[i] + k, n);
    }
#pragma unroll
    for (int v = 0; v < U; ++v)
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        acc[i][0] = mma_chunk(wg[v], xv[v][i], acc[i][0], T());
        acc[i][1] = mma_chunk(wu[v], xv[v][i], acc[i][1], T());
      }
  };
  int s = s0;
  for (; s + 4 <= s1; s += 4) some(std::integral_constant<int, 4>{}, s);
  for (; s < s1; ++s) some(std::integral_constant<int, 1>{}, s);
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    s_part[wave][2 * i][lane] = acc[i][0];
    s_part[wave][2 * i + 1][lane] = acc[i][1];
  }
  __syncthreads();
  if (wave >= FM) return;
  f32x4 gv = s_part[0][2 * wave][lane], uv = s_part[0][2 * wave + 1][lane];
#pragma unroll
  for (int w = 1; w < kFewWaves; ++w) {
    gv += s_part[w][2 * wave][lane];
    uv += s_part[w][2 * wave + 1][lane];
  }
  const int m = wave * 16 + l16, n = n0 + 4 * l4, left = g.N - n;
  if (m >= g.M || left <= 0) return;
  float gs[4], us[4], hs[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    gs[e] = gv[e];
    us[e] = uv[e];
    hs[e] = gs[e] * sigmoid_of(gs[e]) * us[e];
  }
  store_run<T, 4>(g.C + (int64_t)m * g.ldc + n, left, to_run<T, 4>(hs));
  if (g.gate) {
    store_for_later(g.gate + (int64_t)m * g.ld_gate + n, left, gs);
    store_for_later(g.up + (int64_t)m * g.ld_up + n, left, us);
  }
}

// ---- the backward pass ------------------------------------------------------------

constexpr int kSide = 64;  // the halves of [dg | du] are a multiple of this wide

// What the gradients' products read of the inputs: themselves, or copies whose rows are
// whole 16-byte chunks (`pitch` elements), in as many workgroups each.
template <typename T>
struct Copies {
  T *wg, *wu, *x;
  int pitch;
  unsigned slopes, weights, inputs;
};

template <typename T>
__device__ __forceinline__ void copy_chunk(unsigned group, const void* from, int64_t ld, int rows, int cols, T* to,
                                           int pitch) {
  constexpr int E = 16 / (int)sizeof(T);
  const int64_t across = pitch / E, at = (int64_t)group * 256 + threadIdx.x, r = at / across;
  const int c = (int)(at - r * across) * E;
  if (r >= rows) return;
  const Raw<T, E> v = load_run<T, E>(static_cast<const T*>(from) + r * ld + c, cols - c);
  __builtin_memcpy(to + r * pitch + c, v.w, 16);
}

// [dg | du], Fp columns each, zeros from F on, a chunk of each a thread; then the copies.
template <typename T>
__global__ void __launch_bounds__(256) operands_kernel(FfnArgs a, u32x4* zeros, T* both, int Fp, Copies<T> o) {
  constexpr int E = 16 / (int)sizeof(T);
  unsigned group = blockIdx.x;
  if (group >= o.slopes) {
    group -= o.slopes;
    if (group < o.weights) copy_chunk<T>(group, a.wg, a.ld_wg, a.F, a.K, o.wg, o.pitch);
    else if (group < 2 * o.weights) copy_chunk<T>(group - o.weights, a.wu, a.ld_wu, a.F, a.K, o.wu, o.pitch);
    else copy_chunk<T>(group - 2 * o.weights, a.x, a.ld_x, a.M, a.K, o.x, o.pitch);
    return;
  }
  const int64_t across = Fp / E, at = (int64_t)group * 256 + threadIdx.x;
  if (at == 0) *zeros = u32x4{0u, 0u, 0u, 0u};
  const int64_t m = at / across;
  const int f = (int)(at - m * across) * E, n = a.F - f;
  if (m >= a.M) return;
  const Raw<T, E> dh = load_run<T, E>(static_cast<const T*>(a.dh) + m * a.ld_dh + f, n);
  const Raw<float, E> g = load_run<float, E>(a.gate + m * a.ld_gate + f, n);
  const Raw<float, E> u = load_run<float, E>(a.up + m * a.ld_up + f, n);
  float dg[E], du[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const float gv = run_at(g, e), d = run_at(dh, e), sg = sigmoid_of(gv);
    du[e] = d * (gv * sg);
    dg[e] = d * run_at(u, e) * (sg * __builtin_fmaf(gv, 1.f - sg, 1.f));
  }
  T* p = both + m * 2 * Fp + f;
  const Raw<T, E> rg = to_run<T, E>(dg), ru = to_run<T, E>(du);
  __builtin_memcpy(p, rg.w, 16);
  __builtin_memcpy(p + Fp, ru.w, 16);
}

int64_t padded(int64_t n) { return (n + kSide - 1) / kSide * kSide; }
size_t area_bytes(int64_t n, int es) { return ((size_t)n * es + 255) / 256 * 256; }
// Whether the workspace has room for copies of x and the weights: where their rows may
// not be whole 16-byte chunks at multiples of 4 bytes.  (For bfloat16 always: its size
// is promised for any distances between rows and any pointers, which it is not told.)
bool copies_kept(int64_t K, int es) { return es == 2 || K % 4 != 0; }

template <typename T>
hipError_t launch_ffn_t(const FfnArgs& a, hipStream_t stream) {
  GemmArgs<T> g = {};
  g.M = a.M;
  g.N = a.F;
  g.K = a.K;
  g.A = static_cast<const T*>(a.x);
  g.B = static_cast<const T*>(a.wg);
  g.B2 = static_cast<const T*>(a.wu);
  g.lda = a.ld_x;
  g.ldb = a.ld_wg;
  g.ldb2 = a.ld_wu;
  g.C = static_cast<T*>(a.h);
  g.gate = a.gate;
  g.up = a.up;
  g.ldc = a.ld_h;
  g.ld_gate = a.ld_gate;
  g.ld_up = a.ld_up;
  const dim3 few((unsigned)((a.F + 15) / 16));
  if (a.M <= 16) hipLaunchKernelGGL((few_kernel<T, 1>), few, dim3(kFewWaves * kWave), 0, stream, g);
  else if (a.M <= 32) hipLaunchKernelGGL((few_kernel<T, 2>), few, dim3(kFewWaves * kWave), 0, stream, g);
  else launch_gemm<T, kDual>(g, stream);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_ffn_backward_t(const FfnArgs& a, hipStream_t stream) {
  const int Fp = (int)padded(a.F), es = (int)sizeof(T);
  constexpr int E = 16 / (int)sizeof(T);
  char* ws = static_cast<char*>(a.workspace);
  u32x4* const zeros = reinterpret_cast<u32x4*>(ws);                // 256 bytes, the first 16 zeros
  ws += 256;
  const auto area = [&](int64_t n) {
    T* p = reinterpret_cast<T*>(ws);
    ws += area_bytes(n, es);
    return p;
  };
  T* const both = area((int64_t)a.M * 2 * Fp);                      // [M, 2 Fp]
  Copies<T> o = {};
  o.pitch = (a.K + E - 1) / E * E;
  const auto groups = [](int64_t rows, int64_t cols) { return (unsigned)((rows * (cols / E) + 255) / 256); };
  o.slopes = groups(a.M, Fp);
  FfnArgs in = a;
  if (copies_kept(a.K, es)) {
    o.wg = area((int64_t)a.F * o.pitch);
    o.wu = area((int64_t)a.F * o.pitch);
    o.x = area((int64_t)a.M * o.pitch);
    const FfnCopies made = ffn_copies(a, es);
    if (a.dx && made.weights) {
      o.weights = groups(a.F, o.pitch);
      in.wg = o.wg;
      in.wu = o.wu;
      in.ld_wg = in.ld_wu = o.pitch;
    }
    if (a.dwg && made.inputs) {
      o.inputs = groups(a.M, o.pitch);
      in.x = o.x;
      in.ld_x = o.pitch;
    }
  }
  float* const part = reinterpret_cast<float*>(ws);                 // dx's parts, then the weights' gradients'
  hipLaunchKernelGGL((operands_kernel<T>), dim3(o.slopes + 2 * o.weights + o.inputs), dim3(256), 0, stream, a, zeros,
                     both, Fp, o);
  GemmArgs<T> g = {};
  g.zeros = reinterpret_cast<const T*>(zeros);
  g.A = both;
  g.lda = 2 * Fp;
  g.N = a.K;
  g.split = Fp;
  g.rows = a.F;
  g.part = part;
  if (a.dx) {
    g.M = a.M;
    g.K = 2 * Fp;
    g.B = static_cast<const T*>(in.wg);
    g.B2 = static_cast<const T*>(in.wu);
    g.ldb = in.ld_wg;
    g.ldb2 = in.ld_wu;
    g.C = static_cast<T*>(a.dx);
    g.ldc = a.ld_dx;
    launch_gemm<T, kInputs>(g, stream);
  }
  if (a.dwg) {
    g.M = 2 * Fp;
    g.K = a.M;
    g.B = static_cast<const T*>(in.x);
    g.ldb = in.ld_x;
    g.C = static_cast<T*>(a.dwg);
    g.ldc = a.ld_dwg;
    g.C2 = static_cast<T*>(a.dwu);
    g.ldc2 = a.ld_dwu;
    launch_gemm<T, kWeights>(g, stream);
  }
  return hipGetLastError();
}

template <typename T>
__global__ void __launch_bounds__(256) zero_rows_kernel(T* p, int64_t ld, int R, int C) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < (int64_t)R * C; i += (int64_t)gridDim.x * 256)
    p[i / C * ld + i % C] = from_f32<T>(0.f);
}
template <typename T>
hipError_t launch_ffn_no_rows_t(const FfnArgs& a, hipStream_t stream) {
  const int64_t groups = ((int64_t)a.F * a.K + 255) / 256;
  const dim3 grid((unsigned)(groups < 4096 ? groups : 4096));
  hipLaunchKernelGGL((zero_rows_kernel<T>), grid, dim3(256), 0, stream, static_cast<T*>(a.dwg), a.ld_dwg, a.F, a.K);
  hipLaunchKernelGGL((zero_rows_kernel<T>), grid, dim3(256), 0, stream, static_cast<T*>(a.dwu), a.ld_dwu, a.F, a.K);
  return hipGetLastError();
}

}  // namespace

size_t ffn_backward_workspace(int64_t M, int64_t K, int64_t F, int esize) {
  if (M == 0) return 0;
  const int64_t Fp = padded(F);
  const int64_t inputs = plan_gemm(M, K, 2 * Fp, esize, true).parts, weights = plan_gemm(2 * Fp, K, M, esize, true).parts;
  const size_t x = inputs > 1 ? (size_t)inputs * M * K : 0, w = weights > 1 ? (size_t)weights * 2 * Fp * K : 0;
  const int64_t pitch = (K * esize + 15) / 16 * 16 / esize;
  const size_t copies = copies_kept(K, esize) ? 2 * area_bytes(F * pitch, esize) + area_bytes(M * pitch, esize) : 0;
  return 256 + area_bytes(M * 2 * Fp, esize) + copies + (x > w ? x : w) * sizeof(float);
}

FfnCopies ffn_copies(const FfnArgs& a, int esize) {
  const bool chunks = (int64_t)a.K * esize % 16 == 0;
  return FfnCopies{!(chunks && rows4(a.wg, a.ld_wg, esize) && rows4(a.wu, a.ld_wu, esize)),
                   !(chunks && rows4(a.x, a.ld_x, esize))};
}

double ffn_operand_groups(const FfnArgs& a, int esize) {
  const FfnCopies made = ffn_copies(a, esize);
  const double M = a.M, K = a.K + 8.0, F = a.F;
  const double elements = M * (double)padded(a.F) + (made.weights ? 2.0 * F * K : 0.0) + (made.inputs ? M * K : 0.0);
  return elements * esize / 16 / 256 + 4;
}

hipError_t launch_ffn(const FfnArgs& a, m3_dtype dtype, hipStream_t stream) {
  return dtype == M3_BF16 ? launch_ffn_t<bf16>(a, stream) : launch_ffn_t<float>(a, stream);
}
hipError_t launch_ffn_backward(const FfnArgs& a, m3_dtype dtype, hipStream_t stream) {
  if (a.M == 0)
    return dtype == M3_BF16 ? launch_ffn_no_rows_t<bf16>(a, stream) : launch_ffn_no_rows_t<float>(a, stream);
  return dtype == M3_BF16 ? launch_ffn_backward_t<bf16>(a, stream) : launch_ffn_backward_t<float>(a, stream);
}

}  // namespace m3
