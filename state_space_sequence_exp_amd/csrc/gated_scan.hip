// gated_scan.hip -- the gated linear recurrence, per channel
//
//   h_t = a_t h_{t-1} + w_t x_t,  a = sigmoid(f),  w = 1 - a,  y = h * silu(g)
//
// over whole sequences (one pass: see scan_tile.h) and for one token.
//
// Bound by memory: x, f and g are read once and y is written once.  B1 T16384
// D4096 bfloat16 with the gate takes 113 us (4.8 TB/s, 5.2 with the chain's
// words; copies reach 5.2 to 6.1).  What a short call takes is the latency of
// its steps: B1 D1024 bfloat16 6.9 us for one place of the chain (up to 128
// tokens), 8.1 for two, about 0.3 more for each further one (9.8 for 8, 12.1 for
// 16, 16.5 for 32); B3 T777 D1024 10.5.  Rows that are not vectors throughout add
// 2 us to that: a wave at an edge has its loads of f back before it requests x.
//
// A workgroup requests its chunk of x and f and walks each thread's tokens
// once, keeping for every token the map from the state before the thread's
// first (A and B, where x and f were); the threads' maps are joined and
// published, g is requested, and once the state that enters the chunk is known
// every state is A h + B.  (Walking the tokens a second time instead keeps
// one float a token less and takes 63 vector operations an element with the
// output gate, against 38: 139 us for B1 T16384 D4096 bf16 and bound by them.)
#include <type_traits>

#include "scan_tile.h"

namespace m3 {
namespace {

template <typename T, bool kGate, bool kVec>
__global__ void __launch_bounds__(ScanForward<T>::kThreads, 4) scan_kernel(ScanArgs a, ChainWs ws, int nTiles) {
  typedef ScanForward<T> Cfg;
  constexpr int C = Cfg::C, W = Cfg::kPerWord, K = Cfg::K, V = Cfg::V, NW = Cfg::kWaves;
  __shared__ Run s_wave[NW][C];           // each wave's map, then the join of those before
  __shared__ Run s_run[V][Cfg::kThreads];                   // the join of the maps before a thread's in its wave
  __shared__ Run s_part[Cfg::kParts][C];  // the look-back's parts
  __shared__ float s_entry[C];                    // the state entering the chunk
  __shared__ int s_word;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, nP = (int)((a.T + Cfg::kTile - 1) / Cfg::kTile);
  const int units = (int)a.B * nTiles, unit = chain_unit(units);
  const size_t words = (size_t)unit * nP * C;     // of this unit
  const int64_t b = unit / nTiles;
  const int d0 = unit % nTiles * C;
  const int cl = (lane % Cfg::kAcross) * V;       // this lane's first channel in the tile
  const int n = (int)a.D - d0 - cl;               // channels from there to the row's end
  const int k0 = nP > 1 ? chain_ticket(ws, unit, nP, &s_word) : 0;
  if (k0 >= nP) return;
  const int tok = (tid / Cfg::kAcross) * K;    // this thread's first token in the chunk
  const int nt = (int)(a.T - (int64_t)k0 * Cfg::kTile) - tok;  // tokens from there on
  const int64_t row0 = b * a.T + (int64_t)k0 * Cfg::kTile;
  const Rows<T> rf(a.f, row0 * a.ld_f + d0, a.ld_f, tok, cl), rx(a.x, row0 * a.ld_x + d0, a.ld_x, tok, cl);

  Pack<T, V> x[K], f[K], g[K];
  const bool full = nt >= K && n >= V;
  load_rows<kVec>(f, rf, full, nt, n, a.D >= V, kPassGate<T>);
  load_rows<kVec>(x, rx, full, nt, n, a.D >= V, 0u);
  // per token the map from the state before the thread's first; where a gate
  // dropped that state A is NaN, which stays so under the output gate (A is NaN
  // nowhere else: a NaN gate makes B NaN, and so does a NaN output gate)
  const float kDropped = __uint_as_float(0x7fc00000u);
  float A[K][V], B[K][V];
#pragma unroll
  for (int i = 0; i < Cfg::kWords; ++i) {
    float z[K][W], least = 1.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float fv[W];
      unpack_word(f[k].w[i], fv);
#pragma unroll
      for (int e = 0; e < W; ++e) {
        z[k][e] = gate_of(fv[e]);
        least = fminf(least, __builtin_fabsf(z[k][e]));
      }
    }
    Run whole[W];  // of the thread's tokens
    const auto walk = [&](auto mask) {
      constexpr bool kMask = decltype(mask)::value;
#pragma unroll
      for (int e = 0; e < W; ++e) {
        Run r = Run{1.f, 0.f};
        float least = kLeastA;
#pragma unroll
        for (int k = 0; k < K; ++k) {
          float xv[W];
          unpack_word(x[k].w[i], xv);
          r.A = run_factor<kMask>(z[k][e], r.A, least);
          r.B = gate_step<kMask>(z[k][e], r.B, xv[e]);
          A[k][i * W + e] = kMask && r.A == 0.f ? kDropped : r.A;
          B[k][i * W + e] = r.B;
        }
        whole[e] = r;
      }
    };
    if (__any(gate_masks(least))) walk(std::true_type{});
    else walk(std::false_type{});
#pragma unroll
    for (int e = 0; e < W; ++e) {
      const int v = i * W + e;
      Run r = whole[e], before;
      wave_join<Cfg, false>(r, before);
      s_run[v][tid] = before;
      if (lane / Cfg::kAcross == Cfg::kShare - 1) s_wave[wave][cl + v] = r;
    }
  }
  if constexpr (kGate) {
    const Rows<T> rg(a.g, row0 * a.ld_g + d0, a.ld_g, tok, cl);
    load_rows<kVec>(g, rg, full, nt, n, a.D >= V, 0u);
  }
  __syncthreads();
  Run total = Run{1.f, 0.f};
  if (tid < C) {
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const Run m = s_wave[w][tid];
      s_wave[w][tid] = total;
      total = run_join(total, m);
    }
    if (k0 + 1 < nP)
      publish(ws.maps + words + (size_t)k0 * C + tid, word_of(total.A, total.B));
  }
  if constexpr (kGate) {
    // the output gate goes into the maps while the neighbours publish theirs
#pragma unroll
    for (int i = 0; i < Cfg::kWords; ++i)
#pragma unroll
      for (int k = 0; k < K; ++k) {
        float gv[W];
        unpack_word(g[k].w[i], gv);
#pragma unroll
        for (int e = 0; e < W; ++e) {
          const float s = gv[e] * sigmoid_of(gv[e]);
          A[k][i * W + e] *= s;
          B[k][i * W + e] *= s;
          renew(A[k][i * W + e]);
          renew(B[k][i * W + e]);
        }
      }
  }
  const int ch = tid % C, part = tid / C;
  const float h0 = a.h0 && d0 + ch < a.D ? a.h0[b * a.D + d0 + ch] : 0.f;
  if (wave == NW - 1) chain_passed(ws, words, C, k0);
  s_part[part][ch] = chain_part<Cfg>(ws, words, k0, part, ch, h0);
  __syncthreads();
  if (tid < C) {
    float h = 0.f;
#pragma unroll
    for (int p = 0; p < Cfg::kParts; ++p) h = run_apply(s_part[p][tid], h);
    s_entry[tid] = h;
    const float out = run_apply(total, h);
    if (k0 + kWindow < nP)
      publish(ws.exits + words + (size_t)k0 * C + tid, word_of(0.f, out));
    if (d0 + tid < a.D) {
      if (a.states) {
        // one state a chunk: that before the chunk's first wave
        constexpr int kPerTile = Cfg::kTile / M3_SCAN_CHUNK, kStep = NW / kPerTile;
#pragma unroll
        for (int j = 0; j < kPerTile; ++j) {
          const int64_t c = (int64_t)k0 * kPerTile + j;
          if (c < a.nC) a.states[(b * a.nC + c) * a.D + d0 + tid] = run_apply(s_wave[j * kStep][tid], h);
        }
      }
      if (a.h_last && k0 == nP - 1) a.h_last[b * a.D + d0 + tid] = out;
    }
  }
  __syncthreads();
  bool final = false;
  if (nP > 1) {
    chain_clear<Cfg>(ws, words, k0);
    final = wave < Cfg::kHeads && chain_count<Cfg>(ws, unit, nP);
  }

#pragma unroll
  for (int i = 0; i < Cfg::kWords; ++i) {
    float h[W];
#pragma unroll
    for (int e = 0; e < W; ++e) {
      const int v = i * W + e;
      h[e] = run_apply(s_run[v][tid], run_apply(s_wave[wave][cl + v], s_entry[cl + v]));
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float y[W];
#pragma unroll
      for (int e = 0; e < W; ++e) {
        const float p = A[k][i * W + e], q = B[k][i * W + e];
        y[e] = p == p ? __builtin_fmaf(p, h[e], q) : q;
      }
      x[k].w[i] = pack_word(y);
      renew(x[k].w[i]);
    }
  }
  const Rows<T> ry(a.y, row0 * a.ld_y + d0, a.ld_y, tok, cl);
  store_rows<kVec>(x, ry, full, nt, n);
  if (nP > 1 && __syncthreads_or(final)) chain_clear_rest<Cfg>(ws, words, unit, nP);
}

// h_last of an empty sequence.
__global__ void __launch_bounds__(256) scan_empty_kernel(const float* h0, float* h_last, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < n) h_last[i] = h0 ? h0[i] : 0.f;
}

// One token: a lane takes 4 channels of a sequence.
template <typename T, bool kGate, bool kVec>
__global__ void __launch_bounds__(256) scan_step_kernel(ScanStepArgs a, int64_t packs) {
  constexpr int W = 4 / (int)sizeof(T), V = 4;
  const int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (j >= a.B * packs) return;
  const int64_t b = j / packs, d = j % packs * V;
  const int n = (int)(a.D - d);
  Pack<T, V> g;
  const Pack<T, V> f = load_pack<T, V, kVec>(static_cast<const T*>(a.f) + b * a.ld_f + d, n);
  Pack<T, V> x = load_pack<T, V, kVec>(static_cast<const T*>(a.x) + b * a.ld_x + d, n);
  if constexpr (kGate) g = load_pack<T, V, kVec>(static_cast<const T*>(a.g) + b * a.ld_g + d, n);
  Pack<float, V> h = load_pack<float, V, kVec>(a.h_in + b * a.D + d, n);
#pragma unroll
  for (int i = 0; i < f.kWords; ++i) {
    float xv[W], fv[W], gv[W], y[W];
    unpack_word(x.w[i], xv);
    unpack_word(f.w[i], fv);
    if constexpr (kGate) unpack_word(g.w[i], gv);
#pragma unroll
    for (int e = 0; e < W; ++e) {
      const int v = i * W + e;
      y[e] = gate_step<true>(gate_of(fv[e]), __uint_as_float(h.w[v]), xv[e]);
      h.w[v] = __float_as_uint(y[e]);
      if constexpr (kGate) y[e] = y[e] * (gv[e] * sigmoid_of(gv[e]));
    }
    x.w[i] = pack_word(y);
  }
  store_pack<float, V, kVec>(a.h_out + b * a.D + d, n, h);
  store_pack<T, V, kVec>(static_cast<T*>(a.y) + b * a.ld_y + d, n, x);
}


template <typename T>
hipError_t launch_scan_t(const ScanArgs& a, const ChainWs& ws, hipStream_t stream) {
  typedef ScanForward<T> Cfg;
  constexpr size_t es = sizeof(T);
  constexpr int V = Cfg::V;
  const int tiles = (int)scan_tiles(a.D, (int)es);
  const bool vec = a.D % V == 0 && vec_rows(a.x, a.ld_x, es, V) && vec_rows(a.f, a.ld_f, es, V) &&
                   vec_rows(a.g, a.ld_g, es, V) && vec_rows(a.y, a.ld_y, es, V);
  const dim3 grid((unsigned)(a.B * tiles * ((a.T + Cfg::kTile - 1) / Cfg::kTile)));
#define M3_SCAN_LAUNCH(G, VEC)                                                             \
  hipLaunchKernelGGL((scan_kernel<T, G, VEC>), grid, dim3(Cfg::kThreads), 0, stream, a, ws, tiles)
  if (a.g) {
    if (vec) M3_SCAN_LAUNCH(true, true);
    else M3_SCAN_LAUNCH(true, false);
  } else {
    if (vec) M3_SCAN_LAUNCH(false, true);
    else M3_SCAN_LAUNCH(false, false);
  }
#undef M3_SCAN_LAUNCH
  return hipGetLastError();
}

template <typename T>
hipError_t launch_step_t(const ScanStepArgs& a, hipStream_t stream) {
  constexpr size_t es = sizeof(T);
  const int64_t packs = (a.D + 3) / 4;
  const bool vec = a.D % 4 == 0 && vec_rows(a.x, a.ld_x, es, 4) && vec_rows(a.f, a.ld_f, es, 4) &&
                   vec_rows(a.g, a.ld_g, es, 4) && vec_rows(a.y, a.ld_y, es, 4) && vec_rows(a.h_in, a.D, 4, 4) &&
                   vec_rows(a.h_out, a.D, 4, 4);
  const dim3 grid((unsigned)((a.B * packs + 255) / 256));
#define M3_STEP_LAUNCH(G, VEC) \
  hipLaunchKernelGGL((scan_step_kernel<T, G, VEC>), grid, dim3(256), 0, stream, a, packs)
  if (a.g) {
    if (vec) M3_STEP_LAUNCH(true, true);
    else M3_STEP_LAUNCH(true, false);
  } else {
    if (vec) M3_STEP_LAUNCH(false, true);
    else M3_STEP_LAUNCH(false, false);
  }
#undef M3_STEP_LAUNCH
  return hipGetLastError();
}

}  // namespace

namespace {
// Counters (rounded up), then the words' count.
size_t chain_head(size_t units) { return 256 + (units * 8 + 255) / 256 * 256; }
size_t chain_words(size_t units, int64_t T, int tile, int esize) {
  return units * (size_t)((T + tile - 1) / tile) * (kScanTileBytes / esize);
}
}  // namespace

size_t scan_workspace(int64_t B, int64_t T, int64_t D, int tile, int esize) {
  if (T <= tile) return 0;
  const size_t units = (size_t)(B * scan_tiles(D, esize));
  return chain_head(units) + 2 * 8 * chain_words(units, T, tile, esize);
}

ChainWs scan_chain(void* workspace, int64_t B, int64_t T, int64_t D, int tile, int esize) {
  ChainWs w = {};
  if (!workspace || T <= tile) return w;
  const size_t units = (size_t)(B * scan_tiles(D, esize));
  unsigned char* p = static_cast<unsigned char*>(workspace);
  w.err = reinterpret_cast<int*>(p) + 1;
  w.counters = reinterpret_cast<int*>(p + 256);
  w.maps = reinterpret_cast<unsigned long long*>(p + chain_head(units));
  w.exits = w.maps + chain_words(units, T, tile, esize);
  return w;
}

hipError_t launch_scan_empty(const float* h0, float* h_last, int64_t n, hipStream_t stream) {
  hipLaunchKernelGGL(scan_empty_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, stream, h0,
                     h_last, n);
  return hipGetLastError();
}

hipError_t launch_scan(const ScanArgs& a, m3_dtype dtype, hipStream_t stream) {
  const ChainWs ws = scan_chain(a.workspace, a.B, a.T, a.D, kScanForwardTile, dtype == M3_BF16 ? 2 : 4);
  return dtype == M3_BF16 ? launch_scan_t<bf16>(a, ws, stream) : launch_scan_t<float>(a, ws, stream);
}

hipError_t launch_scan_step(const ScanStepArgs& a, m3_dtype dtype, hipStream_t stream) {
  return dtype == M3_BF16 ? launch_step_t<bf16>(a, stream) : launch_step_t<float>(a, stream);
}

}  // namespace m3
