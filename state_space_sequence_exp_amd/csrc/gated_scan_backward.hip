// gated_scan_backward.hip -- gradients of the gated linear recurrence:
//
//   G_t = dy_t silu(g_t) + u_t,  u_{t-1} = a_t G_t  (u_{T-1} = dh_last)
//   dx = G w,  df = G (h_{t-1} - x) a w,  dg = dy h silu'(g),  dh0 = u_{-1}
//
// Bound by memory: x, f, g, dy and the chunks' states are read once, dx, df and
// dg written once.  B4 T2048 D4096 bfloat16 with the gate takes 177 us with its
// forward pass (738 MB between the two, 4.2 TB/s).
//
// The tile and the chain are scan_tile.h's, the chain from the last chunk to
// the first.  The state that enters a chunk was kept by the forward pass, so
// only u has to come from another workgroup.  A thread's tokens make a map of
// the state before them and one of the u behind them; both have the same A.
// Behind the first gate that drops the state (and only there: a factor that
// underflows is no such gate) the state before the thread is not looked at.
#include "scan_tile.h"

namespace m3 {
namespace {

template <typename T, bool kGate, bool kVec>
__global__ void __launch_bounds__(ScanBackward<T>::kThreads, 4)
    scan_backward_kernel(ScanArgs a, ChainWs ws, int nTiles) {
  typedef ScanBackward<T> Cfg;
  constexpr int C = Cfg::C, W = Cfg::kPerWord, K = Cfg::K, V = Cfg::V, NW = Cfg::kWaves;
  __shared__ Run s_fore[NW][C];           // each wave's map of h, then the state entering it
  __shared__ Run s_back[NW][C];           // each wave's map of u, then the join of those behind
  __shared__ Run s_run[V][Cfg::kThreads], s_behind[V][Cfg::kThreads];  // the joins before / behind a thread in its wave
  __shared__ Run s_part[Cfg::kParts][C];  // the look-back's parts
  __shared__ float s_entry[C];                    // the u entering the chunk from behind
  __shared__ int s_word;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, nP = (int)((a.T + Cfg::kTile - 1) / Cfg::kTile);
  const int units = (int)a.B * nTiles, unit = chain_unit(units);
  const size_t words = (size_t)unit * nP * C;     // of this unit
  const int64_t b = unit / nTiles;
  const int d0 = unit % nTiles * C;
  const int cl = (lane % Cfg::kAcross) * V;
  const int n = (int)a.D - d0 - cl;
  const int k0 = nP > 1 ? chain_ticket(ws, unit, nP, &s_word) : 0;  // place in the chain
  if (k0 >= nP) return;
  const int c0 = nP - 1 - k0;                                       // the chunk
  const int tok = (tid / Cfg::kAcross) * K;
  const int nt = (int)(a.T - (int64_t)c0 * Cfg::kTile) - tok;
  const int64_t row0 = b * a.T + (int64_t)c0 * Cfg::kTile;
  const Rows<T> rf(a.f, row0 * a.ld_f + d0, a.ld_f, tok, cl), rx(a.x, row0 * a.ld_x + d0, a.ld_x, tok, cl);
  const Rows<T> rd(a.dy, row0 * a.ld_y + d0, a.ld_y, tok, cl), rg(a.g, row0 * a.ld_g + d0, a.ld_g, tok, cl);

  Pack<T, V> x[K], f[K], dy[K], g[K];
  const bool full = nt >= K && n >= V;
  load_rows<kVec>(f, rf, full, nt, n, a.D >= V, kPassGate<T>);
  load_rows<kVec>(x, rx, full, nt, n, a.D >= V, 0u);
  load_rows<kVec>(dy, rd, full, nt, n, a.D >= V, 0u);
  if constexpr (kGate) load_rows<kVec>(g, rg, full, nt, n, a.D >= V, 0u);
  // per token: the gate, the map from the state before the thread's first
  // token to that before this one, dL/dh without what comes from behind, and
  // dy silu'(g)
  float z[K][V], A[K][V], B[K][V], dh[K][V], dsilu[kGate ? K : 1][V];
  Run whole[V];  // of the thread's tokens
  int drop[V];   // the first token whose gate drops the state (K: none)
#pragma unroll
  for (int i = 0; i < Cfg::kWords; ++i) {
    Run r[W], u[W];
#pragma unroll
    for (int e = 0; e < W; ++e) {
      r[e] = u[e] = Run{1.f, 0.f};
      drop[i * W + e] = K;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float xv[W], fv[W];
      unpack_word(x[k].w[i], xv);
      unpack_word(f[k].w[i], fv);
#pragma unroll
      for (int e = 0; e < W; ++e) {
        const int v = i * W + e;
        const float q = gate_of(fv[e]);
        z[k][v] = q;
        A[k][v] = r[e].A;
        B[k][v] = r[e].B;
        r[e].A = gate_keep<false>(q, r[e].A);
        r[e].B = gate_step<true>(q, r[e].B, xv[e]);
      }
    }
#pragma unroll
    for (int k = K - 1; k >= 0; --k) {
      float dv[W], gv[W];
      unpack_word(dy[k].w[i], dv);
      if constexpr (kGate) unpack_word(g[k].w[i], gv);
#pragma unroll
      for (int e = 0; e < W; ++e) {
        const int v = i * W + e;
        dh[k][v] = dv[e];
        if constexpr (kGate) {
          const float sg = sigmoid_of(gv[e]);
          dh[k][v] = dv[e] * (gv[e] * sg);
          dsilu[k][v] = dv[e] * (sg * __builtin_fmaf(gv[e], 1.f - sg, 1.f));
        }
        u[e].B = gate_keep<true>(z[k][v], dh[k][v] + u[e].B);
        drop[v] = gate_drops(z[k][v]) ? k : drop[v];
      }
    }
#pragma unroll
    for (int e = 0; e < W; ++e) {
      const int v = i * W + e;
      Run o;
      // (A may be NaN where a gate before the one that dropped the state was)
      r[e].A = drop[v] < K ? 0.f : fmaxf(r[e].A, kLeastA);
      whole[v] = r[e];
      u[e].A = r[e].A;
      wave_join<Cfg, false>(r[e], o);
      s_run[v][tid] = o;
      if (lane / Cfg::kAcross == Cfg::kShare - 1) s_fore[wave][cl + v] = r[e];
      wave_join<Cfg, true>(u[e], o);
      s_behind[v][tid] = o;
      if (lane / Cfg::kAcross == 0) s_back[wave][cl + v] = u[e];
    }
  }
  renew(x);
  renew(z);
  renew(dh);
  if constexpr (kGate) renew(dsilu);
  __syncthreads();
  Run total = Run{1.f, 0.f};
  if (tid < C) {
#pragma unroll
    for (int w = NW - 1; w >= 0; --w) {
      const Run m = s_back[w][tid];
      s_back[w][tid] = total;
      total = run_join(total, m);
    }
    if (k0 + 1 < nP)
      publish(ws.maps + words + (size_t)k0 * C + tid, word_of(total.A, total.B));
  } else if (tid < 2 * C) {
    const int c = tid - C;
    float h = d0 + c < a.D ? a.states[(b * nP + c0) * a.D + d0 + c] : 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const Run m = s_fore[w][c];
      s_fore[w][c].B = h;
      h = run_apply(m, h);
    }
  }
  const int ch = tid % C, part = tid / C;
  const float last = a.dh_last && d0 + ch < a.D ? a.dh_last[b * a.D + d0 + ch] : 0.f;
  if (wave == NW - 1) chain_passed(ws, words, C, k0);
  s_part[part][ch] = chain_part<Cfg>(ws, words, k0, part, ch, last);
  __syncthreads();
  if (tid < C) {
    float v = 0.f;
#pragma unroll
    for (int p = 0; p < Cfg::kParts; ++p) v = run_apply(s_part[p][tid], v);
    s_entry[tid] = v;
    const float out = run_apply(total, v);
    if (k0 + kWindow < nP)
      publish(ws.exits + words + (size_t)k0 * C + tid, word_of(0.f, out));
    if (a.dh0 && k0 == nP - 1 && d0 + tid < a.D) a.dh0[b * a.D + d0 + tid] = out;
  }
  __syncthreads();
  bool final = false;
  if (nP > 1) {
    chain_clear<Cfg>(ws, words, k0);
    final = wave < Cfg::kHeads && chain_count<Cfg>(ws, unit, nP);
  }

#pragma unroll
  for (int i = 0; i < Cfg::kWords; ++i) {
    float h[W], after[W], u[W];  // the state before the thread, after a token; u from behind
#pragma unroll
    for (int e = 0; e < W; ++e) {
      const int v = i * W + e;
      h[e] = run_apply(s_run[v][tid], s_fore[wave][cl + v].B);
      after[e] = run_apply(whole[v], h[e]);
      u[e] = run_apply(s_behind[v][tid], run_apply(s_back[wave][cl + v], s_entry[cl + v]));
    }
#pragma unroll
    for (int k = K - 1; k >= 0; --k) {
      float xv[W], dx[W], df[W], dg[W];
      unpack_word(x[k].w[i], xv);
#pragma unroll
      for (int e = 0; e < W; ++e) {
        const int v = i * W + e;
        const float q = z[k][v], kept = __builtin_fmaf(A[k][v], h[e], B[k][v]);
        const float before = k > drop[v] ? B[k][v] : kept;
        if constexpr (kGate) dg[e] = dsilu[k][v] * after[e];
        const float G = dh[k][v] + u[e], s = __builtin_fabsf(q), slope = s * (1.f - s);
        dx[e] = gate_passes(q) ? 0.f : G * gate_w(q);
        df[e] = slope == 0.f ? 0.f : G * (before - xv[e]) * slope;
        u[e] = gate_keep<true>(q, G);
        after[e] = before;
      }
      x[k].w[i] = pack_word(dx);
      dy[k].w[i] = pack_word(df);
      renew(x[k].w[i]);
      renew(dy[k].w[i]);
      if constexpr (kGate) {
        g[k].w[i] = pack_word(dg);
        renew(g[k].w[i]);
      }
    }
  }
  const Rows<T> wx(a.dx, row0 * a.ld_dx + d0, a.ld_dx, tok, cl), wf(a.df, row0 * a.ld_df + d0, a.ld_df, tok, cl);
  const Rows<T> wg(a.dg, row0 * a.ld_dg + d0, a.ld_dg, tok, cl);
  store_rows<kVec>(x, wx, full, nt, n);
  store_rows<kVec>(dy, wf, full, nt, n);
  if constexpr (kGate) store_rows<kVec>(g, wg, full, nt, n);
  if (nP > 1 && __syncthreads_or(final)) chain_clear_rest<Cfg>(ws, words, unit, nP);
}

template <typename T>
hipError_t launch_t(const ScanArgs& a, const ChainWs& ws, hipStream_t stream) {
  typedef ScanBackward<T> Cfg;
  constexpr size_t es = sizeof(T);
  constexpr int V = Cfg::V;
  const int tiles = (int)scan_tiles(a.D, (int)es);
  const bool vec = a.D % V == 0 && vec_rows(a.x, a.ld_x, es, V) && vec_rows(a.f, a.ld_f, es, V) &&
                   vec_rows(a.g, a.ld_g, es, V) && vec_rows(a.dy, a.ld_y, es, V) && vec_rows(a.dx, a.ld_dx, es, V) &&
                   vec_rows(a.df, a.ld_df, es, V) && vec_rows(a.dg, a.ld_dg, es, V);
  const dim3 grid((unsigned)(a.B * tiles * ((a.T + Cfg::kTile - 1) / Cfg::kTile)));
#define M3_SCAN_LAUNCH(G, VEC)                                                                   \
  hipLaunchKernelGGL((scan_backward_kernel<T, G, VEC>), grid, dim3(Cfg::kThreads), 0, stream, a,  \
                     ws, tiles)
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

}  // namespace

hipError_t launch_scan_backward(const ScanArgs& a, m3_dtype dtype, hipStream_t stream) {
  const ChainWs ws = scan_chain(a.workspace, a.B, a.T, a.D, kScanBackwardTile, dtype == M3_BF16 ? 2 : 4);
  return dtype == M3_BF16 ? launch_t<bf16>(a, ws, stream) : launch_t<float>(a, ws, stream);
}

}  // namespace m3
