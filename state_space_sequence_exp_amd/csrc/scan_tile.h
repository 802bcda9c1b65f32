// scan_tile.h -- what the gated recurrence's forward and backward kernels
// share: the tile a workgroup owns and the chain between workgroups.
//
// A workgroup owns some tokens of 256 bytes of channels (128 bfloat16, 64
// float): lanes side by side read whole lines of a token, V channels a lane,
// and each thread holds K consecutive tokens of its lane's channels in
// registers, so each input is read once and each output written once.  A
// thread's steps make one map h -> A h + B a channel; the maps of the threads
// of a wave that share channels are joined by lane moves, those of the waves
// in the LDS, those of the tiles through the workspace.
//
// The kernels are bound by memory, and by how many of a compute unit's waves
// the registers let run.  Measured on B1 T16384 and B4 T2048, D4096, bfloat16
// with the output gate: tiles of 128 bytes of channels reach 4.1 TB/s where
// these reach 4.7; the forward pass with V = 2 and 64 tokens runs three
// workgroups a unit instead of two and is no faster (142 against 123 us when
// this was measured, now 113), as a
// long sequence then has twice the tiles to chain; the backward pass with V =
// 4 and 128 tokens fills its registers and runs two (126 against 116 us then,
// now 109).
#pragma once

#include <hip/hip_runtime.h>

#include "gate.h"
#include "layer_internal.h"

namespace m3 {

template <typename T_, int V_, int K_, int kTile_>
struct ScanCfg {
  typedef T_ T;
  static constexpr int V = V_;                                // channels a lane
  static constexpr int K = K_;                                // tokens a thread
  static constexpr int kTile = kTile_;                        // tokens a workgroup
  static constexpr int C = kScanTileBytes / (int)sizeof(T);   // channels of a tile
  static constexpr int kAcross = C / V;                       // lanes side by side in the channels
  static constexpr int kThreads = kTile / K * kAcross;
  static constexpr int kWaves = kThreads / kWave;
  static constexpr int kShare = kWave / kAcross;              // threads of a wave that share a channel
  static constexpr int kParts = kThreads / C;                 // threads that look back for one channel
  static constexpr int kHeads = C / kWave;                    // waves that join a tile's channels
  static constexpr int kPerWord = 4 / (int)sizeof(T);         // channels of a word
  static constexpr int kWords = V / kPerWord;                 // words of a lane's channels
};
template <typename T>
struct ScanForward;
template <>
struct ScanForward<bf16> : ScanCfg<bf16, 4, 8, kScanForwardTile> {};
template <>
struct ScanForward<float> : ScanCfg<float, 4, 4, kScanForwardTile> {};
template <typename T>
struct ScanBackward;
template <>
struct ScanBackward<bf16> : ScanCfg<bf16, 2, 8, kScanBackwardTile> {};
template <>
struct ScanBackward<float> : ScanCfg<float, 2, 4, kScanBackwardTile> {};

// V channels of a lane as they are stored.  The kernels go through them word
// by word, so that a word of an output takes the registers of an input's that
// has been used.
template <typename T, int V>
struct Pack {
  static constexpr int kWords = V * (int)sizeof(T) / 4;
  uint32_t w[kWords];
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

// Channel i of a pack becomes channel i - by (0 <= by), zeros behind.
template <typename T, int V>
__device__ __forceinline__ void move_down(Pack<T, V>& r, int by) {
  constexpr int W = 4 / (int)sizeof(T), kWords = Pack<T, V>::kWords;
#pragma unroll
  for (int step = kWords / 2; step > 0; step /= 2)  // whole words
#pragma unroll
    for (int i = 0; i < kWords; ++i)
      r.w[i] = by & (step * W) ? (i + step < kWords ? r.w[i + step] : 0u) : r.w[i];
  if constexpr (W == 2)
#pragma unroll
    for (int i = 0; i < kWords; ++i)
      r.w[i] = by & 1 ? r.w[i] >> 16 | (i + 1 < kWords ? r.w[i + 1] << 16 : 0u) : r.w[i];
#pragma unroll
  for (int i = 0; i < kWords; ++i) r.w[i] = by < V ? r.w[i] : 0u;
}

// n of V channels from p (n <= 0: none, zeros).  kVec: p is aligned to V
// elements and n is V or <= 0; else p has element alignment and the last lane
// of a row may hold fewer.
template <typename T, int V, bool kVec>
__device__ __forceinline__ Pack<T, V> load_pack(const void* p, int n) {
  Pack<T, V> r;
  if (n >= V) {
    if constexpr (kVec)
      r = *static_cast<const Pack<T, V>*>(__builtin_assume_aligned(p, V * sizeof(T)));
    else
      __builtin_memcpy(r.w, p, sizeof r.w);
    return r;
  }
#pragma unroll
  for (int i = 0; i < r.kWords; ++i) r.w[i] = 0u;
  if constexpr (!kVec) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) {
        if constexpr (sizeof(T) == 2)
          r.w[i / 2] |= (uint32_t) static_cast<const uint16_t*>(p)[i] << (16 * (i & 1));
        else
          r.w[i] = static_cast<const uint32_t*>(p)[i];
      }
  }
  return r;
}
template <typename T, int V, bool kVec>
__device__ __forceinline__ void store_pack(void* p, int n, const Pack<T, V>& r) {
  if (n >= V) {
    if constexpr (kVec)
      *static_cast<Pack<T, V>*>(__builtin_assume_aligned(p, V * sizeof(T))) = r;
    else
      __builtin_memcpy(p, r.w, sizeof r.w);
  } else if constexpr (!kVec) {
#pragma unroll
    for (int i = 0; i < V; ++i)
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
template <typename T, int V, int K>
__device__ __forceinline__ void renew(Pack<T, V> (&p)[K]) {
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < p[k].kWords; ++i) renew(p[k].w[i]);
}
template <int V, int K>
__device__ __forceinline__ void renew(float (&z)[K][V]) {
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int v = 0; v < V; ++v) renew(z[k][v]);
}

// A thread's rows of an array in the tile whose first element is at `first`:
// row k is k rows on from a base that the workgroup shares (scalar), plus a
// 32-bit byte offset of the thread (a tile's rows of an array span less than
// 4 GiB).
template <typename T>
struct Rows {
  char* base;
  int64_t step;
  uint32_t at;
  int tok, cl;
  __device__ __forceinline__ Rows(const void* p, int64_t first, int64_t ld, int tok, int cl)
      : base(static_cast<char*>(const_cast<void*>(p)) + first * (int64_t)sizeof(T)),
        step(ld * (int64_t)sizeof(T)),
        at((uint32_t)((tok * (uint32_t)ld + cl) * sizeof(T))),
        tok(tok),
        cl(cl) {}
  __device__ __forceinline__ void* operator[](int k) const { return base + k * step + at; }
  // row k (it may be negative: the tile's rows before the thread's), `less`
  // channels down
  __device__ __forceinline__ const void* below(int k, int less) const {
    return base + (int64_t)(cl - less) * (int64_t)sizeof(T) + (uint32_t)((tok + k) * (uint32_t)step);
  }
};

// A thread's K tokens of an array: `nt` of them inside the sequence and `n` of
// the lane's channels inside the row (`full`: all); what lies outside is
// filled with `fill` words, channels with zeros.
//
// Rows that are not vectors throughout: where a row has V channels at all
// (`wide`), a thread at an edge loads the last token again and the row's last
// V channels, and moves its own down once every load is under way.  (Guarded
// loads of a cut vector's channels wait for each other: B3 T777 D1023 bfloat16
// 17.2 us against 12.4, D1001 13.2 against 12.4.  Whole vectors, which are
// there or not, are faster under guards: D1000 10.7 against 11.3.)
template <bool kVec, typename T, int V, int K>
__device__ __forceinline__ void load_rows(Pack<T, V> (&v)[K], const Rows<T>& r, bool full, int nt,
                                          int n, bool wide, uint32_t fill) {
  if (full) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = load_pack<T, V, kVec>(r[k], V);
    return;
  }
  if (!kVec && wide) {
    const int less = n < V ? V - n : 0;
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = load_pack<T, V, kVec>(r.below(min(k, nt - 1), less), V);
#pragma unroll
    for (int k = 0; k < K; ++k) move_down<T, V>(v[k], less);
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = load_pack<T, V, kVec>(r[k], k < nt ? n : 0);
  }
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < v[k].kWords; ++i) v[k].w[i] = k < nt ? v[k].w[i] : fill;
}
template <bool kVec, typename T, int V, int K>
__device__ __forceinline__ void store_rows(const Pack<T, V> (&v)[K], const Rows<T>& r, bool full,
                                           int nt, int n) {
  if (full) {
#pragma unroll
    for (int k = 0; k < K; ++k) store_pack<T, V, kVec>(r[k], V, v[k]);
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (k < nt) store_pack<T, V, kVec>(r[k], n, v[k]);
  }
}
// Gates behind the sequence pass the state on: f = +inf.
template <typename T>
constexpr uint32_t kPassGate = sizeof(T) == 2 ? 0x7f807f80u : 0x7f800000u;

// Whether every row of an array starts at a multiple of V elements.
inline bool vec_rows(const void* p, int64_t ld, size_t es, int V) {
  return !p || (reinterpret_cast<uintptr_t>(p) % (V * es) == 0 && ld % V == 0);
}

// ---- the chain -----------------------------------------------------------------
// A unit is one (sequence, channel tile); its tiles in time form a chain.  The
// workgroup takes its place in the chain from the unit's ticket counter, so
// it only ever waits for workgroups that already run, whatever the order of
// their start.
//
// What a tile hands on are 64-bit words, one a channel, that validate
// themselves: the high half is A with its sign bit set (A is never negative),
// the low half B; an empty word is 0.  They are written and read by relaxed
// device-scope atomics, and no order between words is needed.  Place k
// publishes its map as soon as it has it, and the state that leaves it (a word
// with A = 0) once it knows its entry.  Its entry is the state that left place
// k - W (W = kWindow) through the maps of places k - W + 1 .. k - 1, joined in
// this order, so that results do not depend on timing.  A window that slides
// has no place where all have to wait for their neighbour's state, as groups
// have at their borders.
//
// Words are cleared as the chain moves on.  Besides the state it needs, place
// k waits until the states that left places k - 2 W + 1 .. k - W are all there
// (one lane looks at one word of each, and they are as good as always there):
// a place publishes its state after its look-back, so the look-backs of all
// places up to k - W are then over, by induction.  The map of place c is read
// by places up to c + W - 1 and its state's words by places up to c + 2 W - 1,
// so place k clears map k - 2 W + 1 and state k - 3 W + 1.  The rest, and the
// counters, are left to the unit's last workgroup: all is zero between calls.
// (All of it left to that one took 15 us of a B1 T16384 D4096 call.)
//
// Workspace, in 32-bit words: [0] unused, [1] error word (1: a wait ran out;
// 2: the counters were not zero), then from byte 256 two counters a unit,
// then (256-byte aligned) the 64-bit words: [unit][place][C] maps, then
// [unit][place][C] states.
struct ChainWs {
  int* err;
  int* counters;                 // [units][2]: ticket, finished
  unsigned long long* maps;      // [units][nP][C]
  unsigned long long* exits;     // [units][nP][C]
};
constexpr int kWindow = 8;

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

// The word at p once it is there; a NaN state and error word 1 if it never is
// (or, seen now and then, if another wait has run out already).
__device__ __forceinline__ unsigned long long await(const unsigned long long* p, int* err) {
  unsigned long long w = peek(p);
  for (int i = 1; w == 0 && i < kScanSpins; ++i) {
    __builtin_amdgcn_s_sleep(1);
    w = peek(p);
    if (i % 256 == 0 &&
        __hip_atomic_load(err, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) != 0)
      break;
  }
  if (w == 0) {
    int none = 0;  // the first error stays
    __hip_atomic_compare_exchange_strong(err, &none, 1, __ATOMIC_RELAXED, __ATOMIC_RELAXED,
                                         __HIP_MEMORY_SCOPE_AGENT);
    w = word_of(0.f, __uint_as_float(0x7fc00000u));
  }
  return w;
}

// A launch's unit of workgroup i: the units in turn, turned by one a round, so
// that a compute die does not keep to the same columns.
__device__ __forceinline__ int chain_unit(int units) {
  return (int)((blockIdx.x + blockIdx.x / units) % units);
}

// This workgroup's place in its unit's chain, the same in every thread; nP
// when the counters were not zero (error word 2; the workgroup leaves).
__device__ __forceinline__ int chain_ticket(const ChainWs& ws, int unit, int nP, int* s_word) {
  if (threadIdx.x == 0) {
    const int k = __hip_atomic_fetch_add(ws.counters + 2 * unit, 1, __ATOMIC_RELAXED,
                                         __HIP_MEMORY_SCOPE_AGENT);
    if (k < 0 || k >= nP)
      __hip_atomic_store(ws.err, 2, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *s_word = k < 0 || k >= nP ? nP : k;
  }
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(*s_word);  // in a scalar register, as the addresses from it
}

// This part's share of the window of place k, joined: the state that left
// place k - kWindow (`start` where there is none) and the maps behind it.
// `base`: the unit's first word.
template <typename Cfg>
__device__ __forceinline__ Run chain_part(const ChainWs& ws, size_t base, int k, int part, int ch,
                                          float start) {
  constexpr int C = Cfg::C, kPer = kWindow / Cfg::kParts;
  unsigned long long w[kPer];
  const unsigned long long* from[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = part * kPer + j, c = k - kWindow + i;
    from[j] = (i == 0 ? ws.exits : ws.maps) + base + (size_t)(c < 0 ? 0 : c) * C + ch;
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

// One wave of a workgroup waits for the states that left the window before.
__device__ __forceinline__ void chain_passed(const ChainWs& ws, size_t base, int C, int k) {
  const int lane = threadIdx.x & 63, c = k - 2 * kWindow + 1 + lane;
  if (lane < kWindow && c >= 0) {
    const unsigned long long* from = ws.exits + base + (size_t)c * C;
    if (peek(from) == 0) await(from, ws.err);
  }
}
// Clears what place k is the last to need, behind its look-back.  Nobody reads
// these words any more in this launch, so ordinary stores do: they are out by
// the end of the kernel.
template <typename Cfg>
__device__ __forceinline__ void chain_clear(const ChainWs& ws, size_t base, int k) {
  constexpr int C = Cfg::C;
  const int tid = threadIdx.x, m = k - 2 * kWindow + 1, e = k - 3 * kWindow + 1;
  if (tid < C) {
    if (m >= 0) ws.maps[base + (size_t)m * C + tid] = 0;
  } else if (tid < 2 * C) {
    if (e >= 0) ws.exits[base + (size_t)e * C + tid - C] = 0;
  }
}
// Counts this wave as done with the unit's words: each wave that publishes
// (the first kHeads), after a barrier behind the look-back.  True in the
// unit's last.
template <typename Cfg>
__device__ __forceinline__ bool chain_count(const ChainWs& ws, int unit, int nP) {
  // what this wave published has arrived before the count does
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  int old = 0;
  if ((threadIdx.x & 63) == 0)
    old = __hip_atomic_fetch_add(ws.counters + 2 * unit + 1, 1, __ATOMIC_RELAXED,
                                 __HIP_MEMORY_SCOPE_AGENT);
  return __builtin_amdgcn_readfirstlane(old) == nP * Cfg::kHeads - 1;
}
template <typename Cfg>
__device__ __forceinline__ void chain_clear_rest(const ChainWs& ws, size_t base, int unit, int nP) {
  constexpr int C = Cfg::C;
  const int m = nP - 2 * kWindow + 1, e = nP - 3 * kWindow + 1;
  for (int i = (m < 0 ? 0 : m) * C + (int)threadIdx.x; i < nP * C; i += Cfg::kThreads)
    ws.maps[base + i] = 0;
  for (int i = (e < 0 ? 0 : e) * C + (int)threadIdx.x; i < (nP - kWindow) * C; i += Cfg::kThreads)
    ws.exits[base + i] = 0;
  if (threadIdx.x < 2) ws.counters[2 * unit + threadIdx.x] = 0;
}

// The thread maps of a wave joined over the threads that share a channel
// (kBack: from the last token to the first): r becomes the join up to and
// with this thread, `before` the join of those before it.
template <typename Cfg, bool kBack>
__device__ __forceinline__ void wave_join(Run& r, Run& before) {
  constexpr int kStep = Cfg::kAcross, kShare = Cfg::kShare;
  before = Run{1.f, 0.f};
  if constexpr (kShare > 1) {
    const int g = (threadIdx.x & 63) / kStep, place = kBack ? kShare - 1 - g : g;
    Run o;
#pragma unroll
    for (int s = 1; s < kShare; s *= 2) {
      o.A = kBack ? __shfl_down(r.A, s * kStep, kWave) : __shfl_up(r.A, s * kStep, kWave);
      o.B = kBack ? __shfl_down(r.B, s * kStep, kWave) : __shfl_up(r.B, s * kStep, kWave);
      if (kShare == 2 && place > 0) before = o;
      if (place >= s) r = run_join(o, r);
    }
    if constexpr (kShare > 2) {
      o.A = kBack ? __shfl_down(r.A, kStep, kWave) : __shfl_up(r.A, kStep, kWave);
      o.B = kBack ? __shfl_down(r.B, kStep, kWave) : __shfl_up(r.B, kStep, kWave);
      if (place > 0) before = o;
    }
  }
}

}  // namespace m3
