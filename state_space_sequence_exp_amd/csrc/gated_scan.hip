// gated_scan.hip -- the gated linear recurrence, per channel
//
//   h_t = a_t h_{t-1} + (1 - a_t) x_t,  a = sigmoid(f),  y = h * silu(g)
//
// and its gradients: with G_t = dL/dh_t = dy_t silu(g_t) + a_{t+1} G_{t+1},
//   dx = G w,  df = G (h_{t-1} - x) a w,  dg = dy h silu'(g),  dh0 = a_0 G_0.
//
// One lane per channel walks the tokens.  The backward pass goes from the
// last chunk to the first: it walks a chunk forward from its kept entry
// state, its states in the LDS, then back.
#include "gate.h"
#include "layer_internal.h"

namespace m3 {
namespace {

constexpr int kLanes = 64;

template <typename T, bool kGate>
__global__ void __launch_bounds__(kLanes) scan_kernel(ScanArgs a) {
  const int64_t d = (int64_t)blockIdx.x * kLanes + threadIdx.x, b = blockIdx.y;
  if (d >= a.D) return;
  float h = a.h0 ? a.h0[b * a.D + d] : 0.f;
  for (int64_t t = 0; t < a.T; ++t) {
    const int64_t row = b * a.T + t;
    if (a.states && t % M3_SCAN_CHUNK == 0)
      a.states[(b * a.nC + t / M3_SCAN_CHUNK) * a.D + d] = h;
    const float x = to_f32(static_cast<const T*>(a.x)[row * a.ld_x + d]);
    const Gate q = gate_of(to_f32(static_cast<const T*>(a.f)[row * a.ld_f + d]));
    h = gate_step(q, h, x);
    float y = h;
    if constexpr (kGate) {
      const float g = to_f32(static_cast<const T*>(a.g)[row * a.ld_g + d]);
      y = h * (g * sigmoid_of(g));
    }
    static_cast<T*>(a.y)[row * a.ld_y + d] = from_f32<T>(y);
  }
  if (a.h_last) a.h_last[b * a.D + d] = h;
}

template <typename T, bool kGate>
__global__ void __launch_bounds__(kLanes) scan_backward_kernel(ScanArgs a) {
  __shared__ float s_h[M3_SCAN_CHUNK][kLanes];  // the state before each token
  const int lane = threadIdx.x;
  const int64_t d = (int64_t)blockIdx.x * kLanes + lane, b = blockIdx.y;
  if (d >= a.D) return;
  float u = a.dh_last ? a.dh_last[b * a.D + d] : 0.f;  // a_{t+1} G_{t+1}
  for (int64_t c = a.nC - 1; c >= 0; --c) {
    const int64_t t0 = c * M3_SCAN_CHUNK;
    const int n = (int)(a.T - t0 < M3_SCAN_CHUNK ? a.T - t0 : M3_SCAN_CHUNK);
    float h = a.states[(b * a.nC + c) * a.D + d];
    for (int i = 0; i < n; ++i) {
      const int64_t row = b * a.T + t0 + i;
      s_h[i][lane] = h;
      h = gate_step(gate_of(to_f32(static_cast<const T*>(a.f)[row * a.ld_f + d])), h,
                    to_f32(static_cast<const T*>(a.x)[row * a.ld_x + d]));
    }
    for (int i = n - 1; i >= 0; --i) {
      const int64_t row = b * a.T + t0 + i;
      const float x = to_f32(static_cast<const T*>(a.x)[row * a.ld_x + d]);
      const Gate q = gate_of(to_f32(static_cast<const T*>(a.f)[row * a.ld_f + d]));
      const float dy = to_f32(static_cast<const T*>(a.dy)[row * a.ld_y + d]);
      const float before = s_h[i][lane];
      float dh = dy;
      if constexpr (kGate) {
        const float g = to_f32(static_cast<const T*>(a.g)[row * a.ld_g + d]);
        const float sg = sigmoid_of(g), after = gate_step(q, before, x);
        static_cast<T*>(a.dg)[row * a.ld_dg + d] =
            from_f32<T>(dy * after * (sg * __builtin_fmaf(g, 1.f - sg, 1.f)));
        dh = dy * (g * sg);
      }
      const float G = dh + u, slope = q.a * q.w;
      static_cast<T*>(a.dx)[row * a.ld_dx + d] = from_f32<T>(q.w == 0.f ? 0.f : G * q.w);
      static_cast<T*>(a.df)[row * a.ld_df + d] =
          from_f32<T>(slope == 0.f ? 0.f : G * (before - x) * slope);
      u = gate_decay(q, G);
    }
  }
  if (a.dh0) a.dh0[b * a.D + d] = u;
}

template <typename T, bool kGate>
__global__ void __launch_bounds__(256) scan_step_kernel(ScanStepArgs a) {
  const int64_t d = (int64_t)blockIdx.x * 256 + threadIdx.x, b = blockIdx.y;
  if (d >= a.D) return;
  const float x = to_f32(static_cast<const T*>(a.x)[b * a.ld_x + d]);
  const Gate q = gate_of(to_f32(static_cast<const T*>(a.f)[b * a.ld_f + d]));
  const float h = gate_step(q, a.h_in[b * a.D + d], x);
  a.h_out[b * a.D + d] = h;
  float y = h;
  if constexpr (kGate) {
    const float g = to_f32(static_cast<const T*>(a.g)[b * a.ld_g + d]);
    y = h * (g * sigmoid_of(g));
  }
  static_cast<T*>(a.y)[b * a.ld_y + d] = from_f32<T>(y);
}

}  // namespace

hipError_t launch_scan(const ScanArgs& a, m3_dtype dtype, hipStream_t stream) {
  const dim3 grid((unsigned)((a.D + kLanes - 1) / kLanes), (unsigned)a.B);
  if (dtype == M3_BF16) {
    if (a.g) hipLaunchKernelGGL((scan_kernel<bf16, true>), grid, dim3(kLanes), 0, stream, a);
    else hipLaunchKernelGGL((scan_kernel<bf16, false>), grid, dim3(kLanes), 0, stream, a);
  } else {
    if (a.g) hipLaunchKernelGGL((scan_kernel<float, true>), grid, dim3(kLanes), 0, stream, a);
    else hipLaunchKernelGGL((scan_kernel<float, false>), grid, dim3(kLanes), 0, stream, a);
  }
  return hipGetLastError();
}

hipError_t launch_scan_backward(const ScanArgs& a, m3_dtype dtype, hipStream_t stream) {
  const dim3 grid((unsigned)((a.D + kLanes - 1) / kLanes), (unsigned)a.B);
  if (dtype == M3_BF16) {
    if (a.g) hipLaunchKernelGGL((scan_backward_kernel<bf16, true>), grid, dim3(kLanes), 0, stream, a);
    else hipLaunchKernelGGL((scan_backward_kernel<bf16, false>), grid, dim3(kLanes), 0, stream, a);
  } else {
    if (a.g) hipLaunchKernelGGL((scan_backward_kernel<float, true>), grid, dim3(kLanes), 0, stream, a);
    else hipLaunchKernelGGL((scan_backward_kernel<float, false>), grid, dim3(kLanes), 0, stream, a);
  }
  return hipGetLastError();
}

hipError_t launch_scan_step(const ScanStepArgs& a, m3_dtype dtype, hipStream_t stream) {
  const dim3 grid((unsigned)((a.D + 255) / 256), (unsigned)a.B);
  if (dtype == M3_BF16) {
    if (a.g) hipLaunchKernelGGL((scan_step_kernel<bf16, true>), grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((scan_step_kernel<bf16, false>), grid, dim3(256), 0, stream, a);
  } else {
    if (a.g) hipLaunchKernelGGL((scan_step_kernel<float, true>), grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((scan_step_kernel<float, false>), grid, dim3(256), 0, stream, a);
  }
  return hipGetLastError();
}

}  // namespace m3
