// causal_conv.hip -- the short causal convolution in front of a selective scan
//
//   y_t = act(bias + sum_k weight[k] x_{t-(W-1)+k}),  W = 2, 3 or 4 taps a channel
//
// over prompts and for one token.  Bound by memory: a prompt's x is read and its
// y written once, a token moves its W - 1 kept inputs both ways.
//
// A thread owns one vector of 16 bytes of channels over a run of tokens, kept in
// registers as a window that slides by four tokens (27 us for B4 T2048 D4096
// bfloat16, 5.0 TB/s, where plain copies of large arrays reach 4.2 to 6.2 by their kind;
// by eight it takes more registers and leaves fewer waves, 3 us more):
// only the W - 1 inputs before its run are read twice, from the caches.  Runs are
// four such windows, fewer where that leaves the chip short of threads.
#include "gate.h"
#include "layer_internal.h"
#include "slots.h"
#include "vec_io.h"

namespace m3 {
namespace {

constexpr int kThreads = 256, kRun = 4;

template <int V, int W>
struct Taps {
  float w[V][W], bias[V];
};
template <int V, int W>
__device__ __forceinline__ Taps<V, W> load_taps(const ConvArgs& a, int64_t d, int n) {
  Taps<V, W> t = {};
  const float *w = a.weight + d * W, *bias = a.bias + d;
  if (n >= V) {  // (16 bytes a load: element by element they take 5 us of 32)
    __builtin_memcpy(t.w, w, sizeof t.w);
    if (a.bias) __builtin_memcpy(t.bias, bias, sizeof t.bias);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (e < n) {
        __builtin_memcpy(t.w[e], w + e * W, sizeof t.w[e]);
        if (a.bias) t.bias[e] = bias[e];
      }
  }
  return t;
}

// One output vector from the W inputs that end with its token.
template <typename T, int V, int W>
__device__ __forceinline__ Raw<T, V> filter(const Taps<V, W>& t, const Raw<T, V>* win, bool silu) {
  float v[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    v[e] = t.bias[e];
#pragma unroll
    for (int k = 0; k < W; ++k) v[e] = __builtin_fmaf(t.w[e][k], run_at(win[k], e), v[e]);
    if (silu) v[e] = v[e] * sigmoid_of(v[e]);
  }
  return to_run<T, V>(v);
}

// Input t of a sequence (t >= -(W-1)): from x, or from the inputs kept before it.
template <typename T, int V, int W>
__device__ __forceinline__ Raw<T, V> input_at(const ConvArgs& a, const T* x, int64_t b, int64_t t,
                                              int64_t d, int n) {
  if (t >= 0) return load_run<T, V>(x + t * a.ld_x, n);
  if (!a.state_in) return no_run<T, V>();
  return load_run<T, V>(static_cast<const T*>(a.state_in) + (b * (W - 1) + (W - 1 + t)) * a.D + d, n);
}

template <typename T, int W>
__global__ void __launch_bounds__(kThreads) conv_kernel(ConvArgs a, int nVec, int nRun, int run) {
  constexpr int V = 16 / (int)sizeof(T);
  const int64_t item = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t r = item / nVec;
  const int64_t d = (item - r * nVec) * V;
  const int64_t b = r / (nRun + 1);
  const int64_t k = r - b * (nRun + 1);
  if (b >= a.B) return;
  const int n = (int)min((int64_t)V, a.D - d);
  const int64_t len = a.lengths ? min(max((int64_t)a.lengths[b], (int64_t)0), a.T) : a.T;
  const T* x = static_cast<const T*>(a.x) + b * a.T * a.ld_x + d;
  if (k == nRun) {  // the inputs kept behind the last token
    if (!a.state_out) return;
    T* out = static_cast<T*>(a.state_out) + b * (W - 1) * a.D + d;
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      store_run<T, V>(out + j * a.D, n, input_at<T, V, W>(a, x, b, len - (W - 1) + j, d, n));
    return;
  }
  T* y = static_cast<T*>(a.y) + b * a.T * a.ld_y + d;
  const int64_t t0 = k * run, t1 = min(t0 + run, a.T);
  if (t0 < len) {
    const Taps<V, W> taps = load_taps<V, W>(a, d, n);
    Raw<T, V> win[kRun + W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) win[j] = input_at<T, V, W>(a, x, b, t0 - (W - 1) + j, d, n);
    for (int64_t t = t0; t < t1; t += kRun) {
#pragma unroll
      for (int j = 0; j < kRun; ++j)
        win[W - 1 + j] = t + j < len ? load_run<T, V>(x + (t + j) * a.ld_x, n) : no_run<T, V>();
#pragma unroll
      for (int j = 0; j < kRun; ++j)
        if (t + j < t1) {
          Raw<T, V> o = filter<T, V, W>(taps, win + j, a.silu);
          if (t + j >= len) o = no_run<T, V>();
          store_run<T, V>(y + (t + j) * a.ld_y, n, o);
        }
#pragma unroll
      for (int j = 0; j < W - 1; ++j) win[j] = win[kRun + j];
    }
  } else {
    for (int64_t t = t0; t < t1; ++t) store_run<T, V>(y + t * a.ld_y, n, no_run<T, V>());
  }
}

// A workgroup is one row's kThreads vectors; all it reads is requested before
// the rows before it are searched for its slot.
template <typename T, int W>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(ConvArgs a, int tiles) {
  constexpr int V = 16 / (int)sizeof(T);
  const int b = blockIdx.x / tiles, tile = blockIdx.x % tiles;
  const int slot = slot_of(a.slots, a.n_slots, b);
  if (slot < 0) return;
  const int64_t d = ((int64_t)tile * kThreads + threadIdx.x) * V;
  const int n = (int)max((int64_t)0, min((int64_t)V, a.D - d));
  T* state = static_cast<T*>(a.state_out) + (int64_t)slot * (W - 1) * a.D + d;
  Raw<T, V> win[W];
  Taps<V, W> taps = {};
  if (n > 0) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) win[j] = load_run<T, V>(state + j * a.D, n);
    win[W - 1] = load_run<T, V>(static_cast<const T*>(a.x) + b * a.ld_x + d, n);
    taps = load_taps<V, W>(a, d, n);
  }
  if (__syncthreads_or(named_before<kThreads>(a.slots, b, slot)) || n == 0) return;
  store_run<T, V>(static_cast<T*>(a.y) + b * a.ld_y + d, n, filter<T, V, W>(taps, win, a.silu));
#pragma unroll
  for (int j = 0; j < W - 1; ++j) store_run<T, V>(state + j * a.D, n, win[j + 1]);
}

int vectors(int64_t D, int esize) { return (int)((D * esize + 15) / 16); }

// Tokens a thread takes: four windows, fewer where that would leave less than 2^17
// threads (two waves a SIMD).
int run_tokens(int64_t B, int64_t T, int64_t D, int esize) {
  int run = 4 * kRun;
  while (run > kRun && (double)B * (double)((T + run - 1) / run) * vectors(D, esize) < 131072.0) run /= 2;
  return run;
}

template <typename T>
hipError_t launch_conv_t(const ConvArgs& a, hipStream_t stream) {
  constexpr int es = (int)sizeof(T);
  const int nVec = vectors(a.D, es), run = run_tokens(a.B, a.T, a.D, es);
  const int nRun = (int)((a.T + run - 1) / run);
  const dim3 grid((unsigned)conv_groups(a.B, a.T, a.D, es));
#define M3_CONV_LAUNCH(W) \
  hipLaunchKernelGGL((conv_kernel<T, W>), grid, dim3(kThreads), 0, stream, a, nVec, nRun, run)
  if (a.W == 2) M3_CONV_LAUNCH(2);
  else if (a.W == 3) M3_CONV_LAUNCH(3);
  else M3_CONV_LAUNCH(4);
#undef M3_CONV_LAUNCH
  return hipGetLastError();
}

template <typename T>
hipError_t launch_conv_step_t(const ConvArgs& a, hipStream_t stream) {
  const int tiles = (vectors(a.D, (int)sizeof(T)) + kThreads - 1) / kThreads;
  const dim3 grid((unsigned)conv_step_groups(a.B, a.D, (int)sizeof(T)));
#define M3_CONV_LAUNCH(W) \
  hipLaunchKernelGGL((conv_step_kernel<T, W>), grid, dim3(kThreads), 0, stream, a, tiles)
  if (a.W == 2) M3_CONV_LAUNCH(2);
  else if (a.W == 3) M3_CONV_LAUNCH(3);
  else M3_CONV_LAUNCH(4);
#undef M3_CONV_LAUNCH
  return hipGetLastError();
}

}  // namespace

double conv_groups(int64_t B, int64_t T, int64_t D, int esize) {
  const int run = run_tokens(B, T, D, esize);
  const double items = (double)B * (double)((T + run - 1) / run + 1) * vectors(D, esize);
  return ceil(items / kThreads);
}
double conv_step_groups(int64_t B, int64_t D, int esize) {
  return (double)B * ((vectors(D, esize) + kThreads - 1) / kThreads);
}

hipError_t launch_conv(const ConvArgs& a, m3_dtype dtype, hipStream_t stream) {
  return dtype == M3_BF16 ? launch_conv_t<bf16>(a, stream) : launch_conv_t<float>(a, stream);
}
hipError_t launch_conv_step(const ConvArgs& a, m3_dtype dtype, hipStream_t stream) {
  return dtype == M3_BF16 ? launch_conv_step_t<bf16>(a, stream) : launch_conv_step_t<float>(a, stream);
}

}  // namespace m3
