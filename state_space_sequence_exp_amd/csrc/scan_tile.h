// scan_tile.h -- what the gated recurrence's forward and backward kernels
// share: the tile a workgroup owns and the chain between workgroups.
//
// A workgroup of 512 threads owns one chunk of 128 tokens of 256 bytes of
// channels (128 bfloat16, 64 float): lanes side by side read whole lines of a
// token, 4 channels a lane, and each thread holds 8 (bfloat16) or 4 (float)
// consecutive tokens of its lane's channels in registers: 64 bytes of each
// array.  So each input is read once and each output written once.  (Tiles of
// 128 bytes of channels and 256 tokens reach 4.1 TB/s where these reach 4.6;
// 8 channels a lane, in 16-byte bfloat16 vectors, take 32 registers more for
// the maps and spill.)  A thread's steps make one map h -> A h + B a channel;
// the maps of the threads of a wave that share channels are joined by lane
// moves, those of the waves in the LDS, those of the chunks through the
// workspace.
#pragma once

#include <hip/hip_runtime.h>

#include "gate.h"
#include "layer_internal.h"

namespace m3 {

constexpr int kV = 4;                                   // channels a lane
template <typename T>
constexpr int kAcross = 64 / (int)sizeof(T);            // lanes side by side in the channels
template <typename T>
constexpr int kC = kV * kAcross<T>;                     // channels of a tile
constexpr int kWindow = 8;                              // chunks a look-back spans (see the chain)
template <typename T>
constexpr int kTok = 16 / (int)sizeof(T);               // tokens a thread
constexpr int kScanThreads = 512;
constexpr int kScanWaves = kScanThreads / kWave;
static_assert(kScanThreads / kAcross<bf16> * kTok<bf16> == M3_SCAN_CHUNK &&
              kScanThreads / kAcross<float> * kTok<float> == M3_SCAN_CHUNK,
              "a workgroup owns one chunk");
template <typename T>
constexpr int kShare = kWave / kAcross<T>;              // threads of a wave that share a channel
template <typename T>
constexpr int kParts = kScanThreads / kC<T>;            // threads that look back for one channel
template <typename T>
constexpr int kHeads = kC<T> / kWave;                   // waves that join a tile's channels

// The kV channels of a lane as they are stored.  The kernels go through them
// word by word, so that a word of an output takes the registers of an input's
// that has been used.
template <typename T>
constexpr int kWords = kV * (int)sizeof(T) / 4;
template <typename T>
constexpr int kPerWord = 4 / (int)sizeof(T);  // channels of a word
template <typename T>
struct Pack {
  uint32_t w[kWords<T>];
};

__device__ __forceinline__ void unpack_word(uint32_t w, float (&v)[2]) {
  v[0] = __uint_as_float(w << 16);
  v[1] = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ void unpack_word(uint32_t w, float (&v)[1]) {
  v[0] = __uint_as_float(w);
}
__device__ __forceinline__ uint32_t pack_word(const float (&v)[2]) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{v[0], v[1]}), bf16x2));
}
__device__ __forceinline__ uint32_t pack_word(const float (&v)[1]) { return __float_as_uint(v[0]); }

// n of kV channels from p (n <= 0: none, zeros).  kVec: p is aligned to kV
// elements and n is kV or <= 0; else p has element alignment and the last
// lane of a row may hold fewer.
template <typename T, bool kVec>
__device__ __forceinline__ Pack<T> load_pack(const void* p, int n) {
  Pack<T> r;
  if (n >= kV) {
    if constexpr (kVec)
      r = *static_cast<const Pack<T>*>(__builtin_assume_aligned(p, kV * sizeof(T)));
    else
      __builtin_memcpy(r.w, p, sizeof r.w);
    return r;
  }
#pragma unroll
  for (int i = 0; i < kWords<T>; ++i) r.w[i] = 0u;
  if constexpr (!kVec) {
#pragma unroll
    for (int i = 0; i < kV; ++i)
      if (i < n) {
        if constexpr (sizeof(T) == 2)
          r.w[i / 2] |= (uint32_t) static_cast<const uint16_t*>(p)[i] << (16 * (i & 1));
        else
          r.w[i] = static_cast<const uint32_t*>(p)[i];
      }
  }
  return r;
}
template <typename T, bool kVec>
__device__ __forceinline__ void store_pack(void* p, int n, const Pack<T>& r) {
  if (n >= kV) {
    if constexpr (kVec)
      *static_cast<Pack<T>*>(__builtin_assume_aligned(p, kV * sizeof(T))) = r;
    else
      __builtin_memcpy(p, r.w, sizeof r.w);
  } else if constexpr (!kVec) {
#pragma unroll
    for (int i = 0; i < kV; ++i)
      if (i < n) {
        if constexpr (sizeof(T) == 2)
          static_cast<uint16_t*>(p)[i] = (uint16_t)(r.w[i / 2] >> (16 * (i & 1)));
        else
          static_cast<uint32_t*>(p)[i] = r.w[i];
      }
  }
}

// Hides a register's value from the compiler.  What was computed from it is
// then computed again, not kept (an unpacked copy of every value kept between
// the two walks of a tile would spill), and a result is computed here, not
// where it is stored (the values it comes from would be kept until then).
__device__ __forceinline__ void renew(uint32_t& v) { asm volatile("" : "+v"(v)); }
__device__ __forceinline__ void renew(float& v) { asm volatile("" : "+v"(v)); }
template <typename T, int K>
__device__ __forceinline__ void renew(Pack<T> (&p)[K]) {
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < kWords<T>; ++i) renew(p[k].w[i]);
}
template <int K>
__device__ __forceinline__ void renew(float (&z)[K][kV]) {
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int v = 0; v < kV; ++v) renew(z[k][v]);
}

// A thread's rows of an array in the tile whose first element is at `first`:
// row k is k rows on from a base that the workgroup shares (scalar), plus a
// 32-bit byte offset of the thread (M3_SCAN_CHUNK rows of an array span less
// than 4 GiB).
template <typename T>
struct Rows {
  char* base;
  int64_t step;
  uint32_t at;
  __device__ __forceinline__ Rows(const void* p, int64_t first, int64_t ld, int tok, int cl)
      : base(static_cast<char*>(const_cast<void*>(p)) + first * (int64_t)sizeof(T)),
        step(ld * (int64_t)sizeof(T)),
        at((uint32_t)((tok * (uint32_t)ld + cl) * sizeof(T))) {}
  __device__ __forceinline__ void* operator[](int k) const { return base + k * step + at; }
};

// ---- the chain -----------------------------------------------------------------
// A unit is one (sequence, channel tile); its chunks form a chain.  The
// workgroup takes its place in the chain from the unit's ticket counter, so
// it only ever waits for workgroups that already run, whatever the order of
// their start.
//
// What a chunk hands on are 64-bit words, one a channel, that validate
// themselves: the high half is A with its sign bit set (A is never negative),
// the low half B; an empty word is 0.  They are written and read by relaxed
// device-scope atomics, and no order between words is needed.  A chunk
// publishes its map as soon as it has it, and the state that leaves it (a word
// with A = 0) once it knows its entry.  Chunk k's entry is the state that left
// chunk k - 8 through the maps of chunks k - 7 .. k - 1, joined in this order,
// so that results do not depend on timing.  About as many chunks of a unit
// run at once, so the state waited for is there by then; a window that slides
// has no place where all have to wait for their neighbour's state, as groups
// have at their borders.  Counters and words are zero between calls: the
// unit's last workgroup to finish looking back clears them.
//
// Workspace, in 32-bit words: [0] unused, [1] error word (1: a wait ran out;
// 2: the counters were not zero), then from byte 256 two counters a unit,
// then (256-byte aligned) the 64-bit words: [unit][chunk][C] maps, then
// [unit][chunk][C] states.
struct ChainWs {
  int* err;
  int* counters;                 // [units][2]: ticket, finished
  unsigned long long* maps;      // [units][nC][C]
  unsigned long long* exits;     // [units][nC][C]
};

__device__ __forceinline__ unsigned long long word_of(float A, float B) {
  return ((unsigned long long)(__float_as_uint(A) | 0x80000000u) << 32) | __float_as_uint(B);
}
__device__ __forceinline__ Run run_of(unsigned long long w) {
  return Run{__uint_as_float((uint32_t)(w >> 32) & 0x7fffffffu), __uint_as_float((uint32_t)w)};
}
__device__ __forceinline__ void publish(unsigned long long* p, unsigned long long w) {
  __hip_atomic_store(p, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ unsigned long long peek(const unsigned long long* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// About a quarter of a second of sleeps.
constexpr int kScanSpins = 1 << 18;

// The word at p once it is there; a NaN state and error word 1 if it never is.
__device__ __forceinline__ unsigned long long await(const unsigned long long* p, int* err) {
  unsigned long long w = peek(p);
  for (int i = 0; w == 0 && i < kScanSpins; ++i) {
    __builtin_amdgcn_s_sleep(1);
    w = peek(p);
  }
  if (w == 0) {
    __hip_atomic_store(err, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    w = word_of(0.f, __uint_as_float(0x7fc00000u));
  }
  return w;
}

// A thread's K tokens of an array: `nt` of them inside the sequence and `n` of
// the lane's channels inside the row (`full`: all); what lies outside is
// filled with `fill` words.
template <typename T, bool kVec, int K>
__device__ __forceinline__ void load_rows(Pack<T> (&v)[K], const Rows<T>& r, bool full, int nt, int n,
                                          uint32_t fill) {
  if (full) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = load_pack<T, kVec>(r[k], kV);
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      v[k] = load_pack<T, kVec>(r[k], k < nt ? n : 0);
#pragma unroll
      for (int i = 0; i < kWords<T>; ++i) v[k].w[i] = k < nt ? v[k].w[i] : fill;
    }
  }
}
template <typename T, bool kVec, int K>
__device__ __forceinline__ void store_rows(const Pack<T> (&v)[K], const Rows<T>& r, bool full, int nt,
                                           int n) {
  if (full) {
#pragma unroll
    for (int k = 0; k < K; ++k) store_pack<T, kVec>(r[k], kV, v[k]);
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (k < nt) store_pack<T, kVec>(r[k], n, v[k]);
  }
}
// Gates behind the sequence pass the state on: f = +inf.
template <typename T>
constexpr uint32_t kPassGate = sizeof(T) == 2 ? 0x7f807f80u : 0x7f800000u;

// Whether every row of an array starts at a multiple of kV elements.
inline bool vec_rows(const void* p, int64_t ld, size_t es) {
  return !p || (reinterpret_cast<uintptr_t>(p) % (kV * es) == 0 && ld % kV == 0);
}

// This workgroup's place in its unit's chain, the same in every thread; nC
// when the counters were not zero (error word 2; the workgroup leaves).
__device__ __forceinline__ int chain_ticket(const ChainWs& ws, int unit, int nC, int* s_word) {
  if (threadIdx.x == 0) {
    const int k = __hip_atomic_fetch_add(ws.counters + 2 * unit, 1, __ATOMIC_RELAXED,
                                         __HIP_MEMORY_SCOPE_AGENT);
    if (k < 0 || k >= nC)
      __hip_atomic_store(ws.err, 2, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *s_word = k < 0 || k >= nC ? nC : k;
  }
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(*s_word);  // in a scalar register, as the addresses from it
}

// This part's share of the window of chunk k, joined: the state that left
// chunk k - kWindow (`start` where there is none) and the maps behind it.
template <typename T>
__device__ __forceinline__ Run chain_part(const ChainWs& ws, int unit, int nC, int k, int part,
                                          int ch, float start) {
  constexpr int C = kC<T>, kPer = kWindow / kParts<T>;
  const size_t base = ((size_t)unit * nC) * C + ch;
  unsigned long long w[kPer];
  const unsigned long long* from[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = part * kPer + j, c = k - kWindow + i;
    from[j] = (i == 0 ? ws.exits : ws.maps) + base + (int64_t)(c < 0 ? 0 : c) * C;
    w[j] = c >= 0 ? peek(from[j]) : 0;
  }
  Run r = Run{1.f, 0.f};
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = part * kPer + j, c = k - kWindow + i;
    if (c >= 0) {
      if (w[j] == 0) w[j] = await(from[j], ws.err);
      r = run_join(r, run_of(w[j]));
    } else if (i == 0) {
      r = Run{0.f, start};
    }
  }
  return r;
}

// Counts this wave as done with the unit's words: each wave that publishes
// (the first kHeads), after a barrier behind the look-back.  True in the
// unit's last.
template <typename T>
__device__ __forceinline__ bool chain_count(const ChainWs& ws, int unit, int nC) {
  // what this wave published has arrived before the count does
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  int old = 0;
  if ((threadIdx.x & 63) == 0)
    old = __hip_atomic_fetch_add(ws.counters + 2 * unit + 1, 1, __ATOMIC_RELAXED,
                                 __HIP_MEMORY_SCOPE_AGENT);
  return __builtin_amdgcn_readfirstlane(old) == nC * kHeads<T> - 1;
}
// The unit's last workgroup leaves its counters and words zero.  Nobody reads
// them any more in this launch, so ordinary 16-byte stores do: they are out
// by the end of the kernel.
template <typename T>
__device__ __forceinline__ void chain_clear(const ChainWs& ws, int unit, int nC) {
  const size_t n = (size_t)nC * kC<T> / 2;  // 16-byte vectors
  uint4* maps = reinterpret_cast<uint4*>(ws.maps) + unit * n;
  uint4* exits = reinterpret_cast<uint4*>(ws.exits) + unit * n;
  for (size_t i = threadIdx.x; i < n; i += kScanThreads) {
    maps[i] = make_uint4(0u, 0u, 0u, 0u);
    exits[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  if (threadIdx.x < 2) ws.counters[2 * unit + threadIdx.x] = 0;
}

// The thread maps of a wave joined over the threads that share a channel
// (kBack: from the last token to the first): r becomes the join up to and
// with this thread, `before` the join of those before it.
template <typename T, bool kBack>
__device__ __forceinline__ void wave_join(Run& r, Run& before) {
  constexpr int kStep = kAcross<T>;
  const int g = (threadIdx.x & 63) / kStep, place = kBack ? kShare<T> - 1 - g : g;
#pragma unroll
  for (int s = 1; s < kShare<T>; s *= 2) {
    Run o;
    o.A = kBack ? __shfl_down(r.A, s * kStep, kWave) : __shfl_up(r.A, s * kStep, kWave);
    o.B = kBack ? __shfl_down(r.B, s * kStep, kWave) : __shfl_up(r.B, s * kStep, kWave);
    if (s == 1) before = o;
    if (place >= s) r = run_join(o, r);
  }
  if constexpr (kShare<T> > 2) {
    before.A = kBack ? __shfl_down(r.A, kStep, kWave) : __shfl_up(r.A, kStep, kWave);
    before.B = kBack ? __shfl_down(r.B, kStep, kWave) : __shfl_up(r.B, kStep, kWave);
  }
  if (place == 0) before = Run{1.f, 0.f};
}

}  // namespace m3
