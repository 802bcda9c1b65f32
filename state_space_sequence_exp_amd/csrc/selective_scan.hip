// selective_scan.hip -- the selective state space scan: N states a channel, each
// with a decay of its own,
//
//   s = softplus(dt + dt_bias),  h[n] = exp(s A[n]) h[n] + (s x) B[n]
//   y = (sum_n C[n] h[n] + skip x) * silu(z)
//
// over whole sequences and for one token.
//
// A prompt is bound by vector operations: a state and token takes a product, an
// exponential, a product and two fused sums.  A lane owns the states n, n + 16,
// ... of one channel, so that the 16 lanes of a DPP row own a channel and a wave
// four of them: with a state a lane a layer of 4096 channels and 16 states is
// 1024 waves, one a SIMD, without cutting the sequence.  Steps s and s x lie one
// token a lane and reach the row as DPP operands, which cost nothing; the sums
// over n of 16 tokens are taken together, halving the tokens a lane keeps at each
// of four exchanges, so that lane i ends with token i's.
//
// A workgroup takes 16 channels through tiles of 64 tokens.  Four of its waves scan
// a tile while the other four make ready: they load the tiles after it as they lie in
// memory, four channels of a token each, compute their steps once, turn them in the
// LDS, and finish and store the outputs of the tile before.  Neighbouring workgroups,
// which share cache lines, run on one XCD.
//
// B1 T16384 D4096 N16 bfloat16 with the gate takes 384 us: its scanning waves alone 320,
// at one a SIMD, which issues an operation in about five cycles, not four; the vector
// units are busy for 85% of the cycles.  (With every wave doing both halves' work in turn,
// 589 us; the sums by matrix instructions, 586 and more: they wait for their operands
// and hold up the wave; the sums left to the other half's waves, 703.)  With more
// waves a state and token takes 0.31 to 0.34 ps (B4 T2048 D4096) instead of 0.36.
//
// With few channels (see select_segments) the tokens are cut into segments: a
// first launch takes each from a zero state to its end state and sum of steps
// (the decay of a whole segment is exp(A sum s)), the second joins those before
// its segment and scans on from there.
#include <type_traits>

#include "gate.h"
#include "layer_internal.h"
#include "slots.h"
#include "vec_io.h"

namespace m3 {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / kWave;  // of either half of a scan's workgroup
constexpr int kTile = 64;               // tokens
constexpr int kRow = 16;                // lanes of a DPP row: a channel's
constexpr int kChan = kWaves * kWave / kRow;  // channels of a workgroup
constexpr int kPitch = kTile + 4;       // of the LDS's token rows

// log(1 + exp(v)): with e = exp(-|v|), max(v, 0) + log1p(e), and log1p(e) = log(w)
// + (e - (w - 1)) / w for w the rounded 1 + e, which keeps a small e's digits.
__device__ __forceinline__ float softplus_of(float v) {
  const float e = exp_neg(__builtin_fabsf(v)), w = 1.f + e;
  const float low = (e - (w - 1.f)) * __builtin_amdgcn_rcpf(w);
  return fmaxf(v, 0.f) + __builtin_fmaf(__builtin_amdgcn_logf(w), 0.693147180559945309f, low);
}

// Lane i of every row of 16 lanes, in all of its lanes.
template <int i>
__device__ __forceinline__ float row_lane(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x150 + i, 0xf, 0xf, true));
}
template <int kCtrl>
__device__ __forceinline__ float swap_lanes(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), kCtrl, 0xf, 0xf, true));
}
// Lane i of a row: the sum of p[i] over its 16 lanes.  Four exchanges, each of which
// halves the tokens a lane keeps: with the lane 8 away, lane xor 7, xor 2 and xor 1.
// In the first two the lanes that keep the upper half of the tokens are whole banks
// of four, so that each sum is written for its own lanes alone, by the DPP's bank
// mask (33 operations for 16 tokens; with selects before the sums, 45).  A DPP
// operand is read two operations after it was written, at the earliest: what is
// written here is, and the two waits see to the rest.
__device__ __forceinline__ float row_sums(float (&p)[kRow]) {
  const unsigned long long odd2 = 0xccccccccccccccccull, odd1 = 0xaaaaaaaaaaaaaaaaull;  // lanes with bit 1, 0
  asm(
      "s_nop 1\n\t"
      "v_add_f32_dpp %0, %0, %0 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
      "v_add_f32_dpp %0, %8, %8 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
      "v_add_f32_dpp %1, %1, %1 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
      "v_add_f32_dpp %1, %9, %9 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
      "v_add_f32_dpp %2, %2, %2 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
      "v_add_f32_dpp %2, %10, %10 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
      "v_add_f32_dpp %3, %3, %3 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
      "v_add_f32_dpp %3, %11, %11 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
      "v_add_f32_dpp %4, %4, %4 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
      "v_add_f32_dpp %4, %12, %12 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
      "v_add_f32_dpp %5, %5, %5 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
      "v_add_f32_dpp %5, %13, %13 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
      "v_add_f32_dpp %6, %6, %6 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
      "v_add_f32_dpp %6, %14, %14 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
      "v_add_f32_dpp %7, %7, %7 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
      "v_add_f32_dpp %7, %15, %15 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
      "v_add_f32_dpp %0, %0, %0 row_half_mirror row_mask:0xf bank_mask:0x5\n\t"
      "v_add_f32_dpp %0, %4, %4 row_half_mirror row_mask:0xf bank_mask:0xa\n\t"
      "v_add_f32_dpp %1, %1, %1 row_half_mirror row_mask:0xf bank_mask:0x5\n\t"
      "v_add_f32_dpp %1, %5, %5 row_half_mirror row_mask:0xf bank_mask:0xa\n\t"
      "v_add_f32_dpp %2, %2, %2 row_half_mirror row_mask:0xf bank_mask:0x5\n\t"
      "v_add_f32_dpp %2, %6, %6 row_half_mirror row_mask:0xf bank_mask:0xa\n\t"
      "v_add_f32_dpp %3, %3, %3 row_half_mirror row_mask:0xf bank_mask:0x5\n\t"
      "v_add_f32_dpp %3, %7, %7 row_half_mirror row_mask:0xf bank_mask:0xa\n\t"
      "v_add_f32_dpp %0, %0, %0 quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
      "v_add_f32_dpp %2, %2, %2 quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
      "v_add_f32_dpp %1, %1, %1 quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
      "v_add_f32_dpp %3, %3, %3 quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
      "v_cndmask_b32_e64 %0, %0, %2, %16\n\t"
      "v_cndmask_b32_e64 %1, %1, %3, %16\n\t"
      "s_nop 1\n\t"
      "v_add_f32_dpp %0, %0, %0 quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
      "v_add_f32_dpp %1, %1, %1 quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
      "v_cndmask_b32_e64 %0, %0, %1, %17"
      : "+v"(p[0]), "+v"(p[1]), "+v"(p[2]), "+v"(p[3]), "+v"(p[4]), "+v"(p[5]), "+v"(p[6]), "+v"(p[7]),
        "+v"(p[8]), "+v"(p[9]), "+v"(p[10]), "+v"(p[11]), "+v"(p[12]), "+v"(p[13]), "+v"(p[14]), "+v"(p[15])
      : "s"(odd2), "s"(odd1));
  return p[0];
}

// The w-th workgroup's place when each of the 8 XCDs takes a run of neighbours.
__device__ __forceinline__ int xcd_place(int w, int groups) {
  const int x = w & 7, q = groups >> 3, rest = groups & 7;
  return x * q + min(x, rest) + (w >> 3);
}

// What one thread brings of a tile: four channels of one token, and its share of
// that token's B and C.
template <typename T, int NL, bool kLocal>
struct Piece {
  Raw<T, 4> x, dt, z, b[NL], c[NL];
};

template <int NL, bool kLocal>
struct Stage {
  static constexpr int kN = kRow * NL;  // states held, the last of them zeros where N is less
  float dt[kChan][kPitch], dx[kChan][kPitch];
  float b[kN][kPitch], c[kLocal ? 1 : kN][kPitch];
  float y[kLocal ? 1 : kTile][kChan + 4];
};

template <typename T, int NL, bool kLocal>
__global__ void __launch_bounds__(2 * kThreads)
select_kernel(SelectArgs a, int tiles, int segs, int64_t segLen, float* ends, float* sums) {
  __shared__ Stage<NL, kLocal> s_stage[2];
  const int tid = threadIdx.x & (kThreads - 1), lane = tid & 63, i = lane & (kRow - 1);
  const bool scans = __builtin_amdgcn_readfirstlane(threadIdx.x) < kThreads;
  const int place = xcd_place((int)blockIdx.x, (int)gridDim.x);
  const int launched = kLocal ? segs - 1 : segs;     // nothing follows the last segment's end
  const int tile0 = place % tiles, seg = place / tiles % launched;
  const int64_t bq = place / tiles / launched;
  const int64_t d0 = (int64_t)tile0 * kChan;
  const int N = a.N;
  const int64_t len = a.lengths ? min(max((int64_t)a.lengths[bq], (int64_t)0), a.T) : a.T;
  const int64_t t0 = seg * segLen, t1 = min(t0 + segLen, a.T);
  const int64_t tEnd = min(t1, len);                 // padding from there on
  const int nTiles = tEnd > t0 ? (int)((tEnd - t0 + kTile - 1) / kTile) : 0;

  if (scans) {
    const int ch = (tid >> 6) * (kWave / kRow) + (lane >> 4);
    const int64_t d = d0 + ch;
    float A2[NL], h[NL];
#pragma unroll
    for (int k = 0; k < NL; ++k) {
      const int n = i + kRow * k;
      const bool in = d < a.D && n < N;
      A2[k] = in ? a.A[d * N + n] * kLog2e : 0.f;
      h[k] = !kLocal && in && a.h0 ? a.h0[(bq * a.D + d) * N + n] : 0.f;
    }
    if constexpr (!kLocal) {
      // the segments before, eight at a time in flight (past the last: none, its decay 1)
      for (int s0 = 0; s0 < seg; s0 += 8) {
        float sum[8], end[8][NL];
#pragma unroll
        for (int v = 0; v < 8; ++v) {
          const int64_t at = (bq * (segs - 1) + min(s0 + v, seg - 1)) * a.D + min(d, a.D - 1);
          const bool in = s0 + v < seg;
          sum[v] = in ? sums[at] : 0.f;
#pragma unroll
          for (int k = 0; k < NL; ++k) end[v][k] = in ? ends[at * N + min(i + kRow * k, N - 1)] : 0.f;
        }
#pragma unroll
        for (int v = 0; v < 8; ++v)
#pragma unroll
          for (int k = 0; k < NL; ++k)
            h[k] = __builtin_fmaf(__builtin_amdgcn_exp2f(A2[k] * sum[v]), h[k], end[v][k]);
      }
#pragma unroll
      for (int k = 0; k < NL; ++k)  // lanes without a state hold none
        if (d >= a.D || i + kRow * k >= N) h[k] = 0.f;
    }
    float total = 0.f;  // of the steps of this lane's tokens
    lds_barrier();
    for (int q = 0; q < nTiles; ++q) {
      Stage<NL, kLocal>& st = s_stage[q & 1];
      for (int j = 0; j < kTile; j += kRow) {
        const float vdt = st.dt[ch][j + i], vdx = st.dx[ch][j + i];
        float p[kRow];
        if constexpr (kLocal) total += vdt;
        const auto four = [&](auto first) {  // tokens first .. first + 3 of the 16
          constexpr int f = decltype(first)::value;
          float4 b4[NL], c4[NL];
#pragma unroll
          for (int k = 0; k < NL; ++k) {
            b4[k] = *reinterpret_cast<const float4*>(&st.b[i + kRow * k][j + f]);
            if constexpr (!kLocal) c4[k] = *reinterpret_cast<const float4*>(&st.c[i + kRow * k][j + f]);
          }
          const auto one = [&](auto tok) {
            constexpr int e = decltype(tok)::value;
#pragma unroll
            for (int k = 0; k < NL; ++k) {
              const float decay = __builtin_amdgcn_exp2f(row_lane<f + e>(vdt) * A2[k]);
              h[k] = __builtin_fmaf(decay, h[k], row_lane<f + e>(vdx) * (&b4[k].x)[e]);
              if constexpr (!kLocal)
                p[f + e] = k ? __builtin_fmaf((&c4[k].x)[e], h[k], p[f + e]) : (&c4[k].x)[e] * h[k];
            }
          };
          one(std::integral_constant<int, 0>{});
          one(std::integral_constant<int, 1>{});
          one(std::integral_constant<int, 2>{});
          one(std::integral_constant<int, 3>{});
        };
        four(std::integral_constant<int, 0>{});
        four(std::integral_constant<int, 4>{});
        four(std::integral_constant<int, 8>{});
        four(std::integral_constant<int, 12>{});
        if constexpr (!kLocal) st.y[j + i][ch] = row_sums(p);
      }
      lds_barrier();
    }
    if constexpr (kLocal) {
      total += swap_lanes<0xb1>(total);
      total += swap_lanes<0x4e>(total);
      total += swap_lanes<0x141>(total);
      total += swap_lanes<0x140>(total);
      const int64_t at = (bq * (segs - 1) + seg) * a.D + d;
      if (d < a.D && i == 0) sums[at] = total;
#pragma unroll
      for (int k = 0; k < NL; ++k)
        if (d < a.D && i + kRow * k < N) ends[at * N + i + kRow * k] = h[k];
    } else if (a.h_last && seg == segs - 1) {
#pragma unroll
      for (int k = 0; k < NL; ++k)
        if (d < a.D && i + kRow * k < N) a.h_last[(bq * a.D + d) * N + i + kRow * k] = h[k];
    }
    return;
  }

  // what a thread of the other half brings and finishes
  const int tk = tid >> 2, part = tid & 3, c0 = part * 4;
  const int nc = (int)max((int64_t)0, min((int64_t)4, a.D - d0 - c0));
  float bias[4], skip[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    bias[e] = a.dt_bias && e < nc ? a.dt_bias[d0 + c0 + e] : 0.f;
    skip[e] = a.skip && e < nc ? a.skip[d0 + c0 + e] : 0.f;
  }
  // (addresses are walked, a tile at a time: a 64-bit product takes a wave as long as
  // sixteen of its other operations)
  const int64_t row0 = bq * a.T + t0 + tk;
  const T* px = static_cast<const T*>(a.x) + row0 * a.ld_x + d0 + c0;
  const T* pdt = static_cast<const T*>(a.dt) + row0 * a.ld_dt + d0 + c0;
  const T* pz = a.z ? static_cast<const T*>(a.z) + row0 * a.ld_z + d0 + c0 : px;
  const T* pb = static_cast<const T*>(a.Bt) + row0 * a.ld_b + part * NL * 4;
  const T* pc = static_cast<const T*>(a.Ct) + row0 * a.ld_c + part * NL * 4;
  T* py = static_cast<T*>(a.y) + row0 * a.ld_y + d0 + c0;
  int64_t toGo = tEnd - t0 - tk;  // tokens from this thread's next on
  const auto request = [&] {
    Piece<T, NL, kLocal> p = {};
    if (toGo > 0) {
      p.x = load_run<T, 4>(px, nc);
      p.dt = load_run<T, 4>(pdt, nc);
      if constexpr (!kLocal)
        if (a.z) p.z = load_run<T, 4>(pz, nc);
#pragma unroll
      for (int v = 0; v < NL; ++v) {
        const int n = (part * NL + v) * 4;
        p.b[v] = load_run<T, 4>(pb + 4 * v, N - n);
        if constexpr (!kLocal) p.c[v] = load_run<T, 4>(pc + 4 * v, N - n);
      }
    }
    px += kTile * a.ld_x;
    pdt += kTile * a.ld_dt;
    pz += kTile * a.ld_z;
    pb += kTile * a.ld_b;
    pc += kTile * a.ld_c;
    toGo -= kTile;
    return p;
  };
  const auto put = [&](int q, const Piece<T, NL, kLocal>& p) {
    Stage<NL, kLocal>& st = s_stage[q & 1];
    const bool live = t0 + (int64_t)q * kTile + tk < tEnd;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float v = run_at(p.dt, e) + bias[e];
      const float step = live ? (a.softplus ? softplus_of(v) : v) : 0.f;
      st.dt[c0 + e][tk] = step;
      st.dx[c0 + e][tk] = step * run_at(p.x, e);
    }
#pragma unroll
    for (int v = 0; v < NL; ++v)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        st.b[(part * NL + v) * 4 + e][tk] = run_at(p.b[v], e);
        if constexpr (!kLocal) st.c[(part * NL + v) * 4 + e][tk] = run_at(p.c[v], e);
      }
  };
  struct Held {
    Raw<T, 4> x, z;
  };
  const auto finish = [&](int q, const Held& v) {
    T* const to = py;
    py += kTile * a.ld_y;
    if (t0 + (int64_t)q * kTile + tk >= tEnd) return;
    const float4 sum = *reinterpret_cast<const float4*>(&s_stage[q & 1].y[kLocal ? 0 : tk][c0]);
    float y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      y[e] = __builtin_fmaf(skip[e], run_at(v.x, e), (&sum.x)[e]);
      if (a.z) {
        const float g = run_at(v.z, e);
        y[e] = y[e] * (g * sigmoid_of(g));
      }
    }
    store_run<T, 4>(to, nc, to_run<T, 4>(y));
  };

  // (two tiles' loads are in flight; the outputs are stored last, so that no wait
  // for loads is one for the stores too)
  Held before = {}, now = {};
  Piece<T, NL, kLocal> next = request(), later = request();
  if (nTiles > 0) put(0, next);
  now = Held{next.x, next.z};
  next = later;
  later = request();
  lds_barrier();
  for (int q = 0; q < nTiles; ++q) {
    const Held last = before;
    before = now;
    now = Held{next.x, next.z};
    if (q + 1 < nTiles) put(q + 1, next);
    next = later;
    later = request();
    if constexpr (!kLocal)
      if (q > 0) finish(q - 1, last);
    lds_barrier();
  }
  if constexpr (!kLocal) {
    if (nTiles > 0) finish(nTiles - 1, before);
    for (int64_t t = max(tEnd, t0) + tk; t < t1; t += kTile)
      store_run<T, 4>(static_cast<T*>(a.y) + (bq * a.T + t) * a.ld_y + d0 + c0, nc, no_run<T, 4>());
  }
}

// One token: a lane owns four neighbouring states, LQ lanes a channel; bound by
// the state's 8 bytes (256 x 4096 x 16 bfloat16: 31 us, 4.5 TB/s).  A thread takes
// kSteps channels (with 1, 36 us, with 4, 35), all requested before the rows before
// its own are searched for its slot.
constexpr int kSteps = 2;

template <typename T, int LQ>
__global__ void __launch_bounds__(kThreads) select_step_kernel(SelectArgs a, int tiles) {
  constexpr int kAcross = kThreads / LQ;  // channels side by side
  const int b = blockIdx.x / tiles, tile = blockIdx.x % tiles;
  const int slot = slot_of(a.slots, a.n_slots, b);
  if (slot < 0) return;
  const int q = threadIdx.x % LQ, n0 = 4 * q, N = a.N;
  const int64_t first = (int64_t)tile * kAcross * kSteps + threadIdx.x / LQ;
  const Raw<T, 4> Bv = load_run<T, 4>(static_cast<const T*>(a.Bt) + b * a.ld_b + n0, N - n0);
  const Raw<T, 4> Cv = load_run<T, 4>(static_cast<const T*>(a.Ct) + b * a.ld_c + n0, N - n0);
  Raw<float, 4> hv[kSteps], Av[kSteps];
  float x[kSteps], dt[kSteps], z[kSteps], skip[kSteps];
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int64_t d = first + s * kAcross;
    const bool in = d < a.D;
    hv[s] = load_run<float, 4>(a.h_last + ((int64_t)slot * a.D + d) * N + n0, in ? N - n0 : 0);
    Av[s] = load_run<float, 4>(a.A + d * N + n0, in ? N - n0 : 0);
    x[s] = in ? to_f32(static_cast<const T*>(a.x)[b * a.ld_x + d]) : 0.f;
    dt[s] = in ? to_f32(static_cast<const T*>(a.dt)[b * a.ld_dt + d]) : 0.f;
    if (a.dt_bias && in) dt[s] += a.dt_bias[d];
    z[s] = in && a.z ? to_f32(static_cast<const T*>(a.z)[b * a.ld_z + d]) : 0.f;
    skip[s] = in && a.skip ? a.skip[d] : 0.f;
  }
  if (__syncthreads_or(named_before<kThreads>(a.slots, b, slot))) return;
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int64_t d = first + s * kAcross;
    const float step = a.softplus ? softplus_of(dt[s]) : dt[s], dx = step * x[s];
    float h[4], y = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float decay = __builtin_amdgcn_exp2f(step * (run_at(Av[s], e) * kLog2e));
      h[e] = __builtin_fmaf(decay, run_at(hv[s], e), dx * run_at(Bv, e));
      y = __builtin_fmaf(run_at(Cv, e), h[e], y);
    }
    if constexpr (LQ > 1) y += swap_lanes<0xb1>(y);
    if constexpr (LQ > 2) y += swap_lanes<0x4e>(y);
    if constexpr (LQ > 4) y += swap_lanes<0x141>(y);
    if constexpr (LQ > 8) y += swap_lanes<0x140>(y);
    if (d >= a.D) continue;
    store_for_later(a.h_last + ((int64_t)slot * a.D + d) * N + n0, N - n0, h);
    y = __builtin_fmaf(skip[s], x[s], y);
    if (a.z) y = y * (z[s] * sigmoid_of(z[s]));
    if (q == 0) static_cast<T*>(a.y)[b * a.ld_y + d] = from_f32<T>(y);
  }
}

int64_t channel_tiles(int64_t D) { return (D + kChan - 1) / kChan; }
int64_t segment_tokens(int64_t T, int segs) {
  const int64_t n = (T + segs - 1) / segs;
  return (n + kTile - 1) / kTile * kTile;
}
int lanes_of(int N) { return N <= 4 ? 1 : N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }

template <typename T, int NL>
void launch_select_n(const SelectArgs& a, hipStream_t stream) {
  const int tiles = (int)channel_tiles(a.D), segs = select_segments(a.B, a.T, a.D);
  const int64_t len = segment_tokens(a.T, segs);
  float* ends = static_cast<float*>(a.workspace);
  float* sums = ends + a.B * (segs - 1) * a.D * a.N;
  const unsigned units = (unsigned)(a.B * tiles);
  if (segs > 1)
    hipLaunchKernelGGL((select_kernel<T, NL, true>), dim3(units * (segs - 1)), dim3(2 * kThreads), 0, stream, a,
                       tiles, segs, len, ends, sums);
  hipLaunchKernelGGL((select_kernel<T, NL, false>), dim3(units * segs), dim3(2 * kThreads), 0, stream, a, tiles,
                     segs, len, ends, sums);
}
template <typename T>
hipError_t launch_select_t(const SelectArgs& a, hipStream_t stream) {
  if (a.N <= kRow) launch_select_n<T, 1>(a, stream);
  else if (a.N <= 2 * kRow) launch_select_n<T, 2>(a, stream);
  else launch_select_n<T, 4>(a, stream);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_select_step_t(const SelectArgs& a, hipStream_t stream) {
  const int lq = lanes_of(a.N), each = kThreads / lq * kSteps;
  const int tiles = (int)((a.D + each - 1) / each);
  const dim3 grid((unsigned)select_step_groups(a.B, a.D, a.N));
#define M3_STEP_LAUNCH(LQ) \
  hipLaunchKernelGGL((select_step_kernel<T, LQ>), grid, dim3(kThreads), 0, stream, a, tiles)
  switch (lq) {
    case 1: M3_STEP_LAUNCH(1); break;
    case 2: M3_STEP_LAUNCH(2); break;
    case 4: M3_STEP_LAUNCH(4); break;
    case 8: M3_STEP_LAUNCH(8); break;
    default: M3_STEP_LAUNCH(16);
  }
#undef M3_STEP_LAUNCH
  return hipGetLastError();
}

}  // namespace

// A wave holds four channels; with fewer than 512 of them on the 1024 SIMDs (127 tiles
// of 16 channels) the tokens are cut so that there are about 2048, into segments of four
// tiles at least.  Cutting does two thirds of the work twice.  Measured, bfloat16 with the
// gate, us by the number of segments, * what the rule takes:
//
//   T16384 N16   D256:  1: 351   8: 84    16: 48    32: 43*   64: 50
//                D512:  1: 348   8: 85    16: 72*   32: 72    64: 83
//                D1024: 1: 346   4: 162    8: 135*  16: 128   32: 130
//                D1536: 1: 376   3: 310    5*       6: 230     8: 200
//                D2032: 1: 357   3: 317    4: 269*   8: 252
//                D2048: 1: 373*  3: 322    4: 272    8: 255
//                D2560: 1: 404*  2: 496    4: 345    8: 311
//                D4096: 1: 385*  2: 486    4: 453
//   T16384 N64   D1024: 1: 1030  4: 453    8: 436*  16: 439
//                D2032: 1: 1031  3: 952    4: 857*   8: 853
//                D2560: 1: 1029* 2: 1405   4: 1117   8: 1059
//   T512         D256:  1: 14.6* 2: 16.0  (fewer than three: not cut)
//   T768         D256:  1: 20.2  3: 16.1*  6: 11.9
//   T2048        D64:   1: 46.4  8: 16.1* 16: 12.1
//
// So what the rule cuts is worth cutting and what has the chip's 256 CUs full is not; it
// leaves uncut from 128 tiles on what would still gain in four segments with 16 states
// (up to 160 tiles; with 64 states not), and segments of two tiles would serve short
// sequences of few channels better than four.
int select_segments(int64_t B, int64_t T, int64_t D) {
  const int64_t waves = B * channel_tiles(D) * kWaves;
  if (waves < 1 || waves >= 512) return 1;
  int64_t segs = 2048 / waves;
  if (segs > T / (4 * kTile)) segs = T / (4 * kTile);
  if (segs < 3) return 1;
  const int64_t len = segment_tokens(T, (int)segs);
  return (int)((T + len - 1) / len);
}

size_t select_workspace(int64_t B, int64_t T, int64_t D, int N) {
  const int segs = select_segments(B, T, D);
  return (size_t)B * (segs - 1) * D * (N + 1) * sizeof(float);
}

double select_groups(int64_t B, int64_t T, int64_t D) {
  return (double)B * (double)channel_tiles(D) * select_segments(B, T, D);
}
double select_step_groups(int64_t B, int64_t D, int N) {
  const int each = kThreads / lanes_of(N) * kSteps;
  return (double)B * (double)((D + each - 1) / each);
}

hipError_t launch_select(const SelectArgs& a, m3_dtype dtype, hipStream_t stream) {
  return dtype == M3_BF16 ? launch_select_t<bf16>(a, stream) : launch_select_t<float>(a, stream);
}
hipError_t launch_select_step(const SelectArgs& a, m3_dtype dtype, hipStream_t stream) {
  return dtype == M3_BF16 ? launch_select_step_t<bf16>(a, stream) : launch_select_step_t<float>(a, stream);
}

}  // namespace m3
