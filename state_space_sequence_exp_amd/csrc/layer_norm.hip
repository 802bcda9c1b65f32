// layer_norm.hip -- layer norm with the residual sum, and its gradients:
//
//   s = x + residual,  q = (s - mean) rstd,  y = q weight + bias
//   dx = rstd (p - mean(p) - q mean(p q)) + dsum,  p = dy weight
//   dweight = sum_rows dy q,  dbias = sum_rows dy
//
// One workgroup a row; the row stays in the LDS as floats between the passes
// (sum, centred squares, output).  The weight gradients are summed by row
// groups into the workspace, then over the groups, in a fixed order.
#include <algorithm>

#include "layer_internal.h"
#include "m3_device.h"

namespace m3 {
namespace {

constexpr int kThreads = 256;

// Sum over the workgroup, the same in every thread.
__device__ __forceinline__ float block_sum(float v, float* s_part) {
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s_part[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.f;
  for (int i = 0; i < kThreads / kWave; ++i) v += s_part[i];
  return v;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) norm_kernel(NormArgs a) {
  extern __shared__ float s_row[];
  __shared__ float s_part[kThreads / kWave];
  const int64_t r = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + r * a.ld_x;
  const T* res = static_cast<const T*>(a.residual) + r * a.ld_res;
  float sum = 0.f;
  for (int d = threadIdx.x; d < a.D; d += kThreads) {
    float v = to_f32(x[d]);
    if (a.residual) v = to_f32(from_f32<T>(v + to_f32(res[d])));
    if (a.sum) static_cast<T*>(a.sum)[r * a.ld_sum + d] = from_f32<T>(v);
    s_row[d] = v;
    sum += v;
  }
  const float mean = block_sum(sum, s_part) / (float)a.D;
  float sq = 0.f;
  for (int d = threadIdx.x; d < a.D; d += kThreads) {
    const float c = s_row[d] - mean;
    sq = __builtin_fmaf(c, c, sq);
  }
  const float rstd = 1.f / sqrtf(block_sum(sq, s_part) / (float)a.D + a.eps);
  for (int d = threadIdx.x; d < a.D; d += kThreads) {
    const float q = (s_row[d] - mean) * rstd;
    static_cast<T*>(a.y)[r * a.ld_y + d] =
        from_f32<T>(__builtin_fmaf(q, a.weight[d], a.bias ? a.bias[d] : 0.f));
  }
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[r] = mean;
    if (a.rstd) a.rstd[r] = rstd;
  }
}

// Workgroup i: the rows of group i, one after another.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_backward_kernel(NormArgs a) {
  extern __shared__ float s_acc[];  // this group's dweight and dbias
  __shared__ float s_part[kThreads / kWave];
  float *s_dw = s_acc, *s_db = s_acc + a.D;
  for (int d = threadIdx.x; d < a.D; d += kThreads) s_dw[d] = s_db[d] = 0.f;
  const int64_t per = (a.rows + gridDim.x - 1) / gridDim.x;
  const int64_t r0 = blockIdx.x * per, r1 = r0 + per < a.rows ? r0 + per : a.rows;
  for (int64_t r = r0; r < r1; ++r) {
    const T* s = static_cast<const T*>(a.sum) + r * a.ld_sum;
    const T* dy = static_cast<const T*>(a.dy) + r * a.ld_dy;
    const float mean = a.mean[r], rstd = a.rstd[r];
    float sp = 0.f, spq = 0.f;
    for (int d = threadIdx.x; d < a.D; d += kThreads) {
      const float q = (to_f32(s[d]) - mean) * rstd, g = to_f32(dy[d]), p = g * a.weight[d];
      sp += p;
      spq = __builtin_fmaf(p, q, spq);
      s_dw[d] = __builtin_fmaf(g, q, s_dw[d]);
      s_db[d] += g;
    }
    const float mp = block_sum(sp, s_part) / (float)a.D;
    const float mpq = block_sum(spq, s_part) / (float)a.D;
    for (int d = threadIdx.x; d < a.D; d += kThreads) {
      const float q = (to_f32(s[d]) - mean) * rstd, p = to_f32(dy[d]) * a.weight[d];
      float v = rstd * (p - mp - q * mpq);
      if (a.dsum) v += to_f32(static_cast<const T*>(a.dsum)[r * a.ld_dsum + d]);
      static_cast<T*>(a.dx)[r * a.ld_dx + d] = from_f32<T>(v);
    }
  }
  for (int d = threadIdx.x; d < a.D; d += kThreads) {
    a.partial[((int64_t)blockIdx.x * 2) * a.D + d] = s_dw[d];
    a.partial[((int64_t)blockIdx.x * 2 + 1) * a.D + d] = s_db[d];
  }
}

__global__ void __launch_bounds__(kThreads) norm_weights_kernel(NormArgs a, int groups) {
  const int d = (int)(blockIdx.x * kThreads + threadIdx.x);
  if (d >= a.D) return;
  float dw = 0.f, db = 0.f;
  for (int i = 0; i < groups; ++i) {
    dw += a.partial[((int64_t)i * 2) * a.D + d];
    db += a.partial[((int64_t)i * 2 + 1) * a.D + d];
  }
  a.dweight[d] = dw;
  if (a.dbias) a.dbias[d] = db;
}

}  // namespace

int norm_backward_groups(int64_t rows, int) { return (int)std::min<int64_t>(rows, 256); }

hipError_t launch_norm(const NormArgs& a, m3_dtype dtype, hipStream_t stream) {
  const size_t lds = sizeof(float) * (size_t)a.D;
  const dim3 grid((unsigned)a.rows);
  const void* k = dtype == M3_BF16 ? reinterpret_cast<const void*>(&norm_kernel<bf16>)
                                   : reinterpret_cast<const void*>(&norm_kernel<float>);
  const hipError_t e = lds_limit(k, lds);
  if (e != hipSuccess) return e;
  if (dtype == M3_BF16)
    hipLaunchKernelGGL(norm_kernel<bf16>, grid, dim3(kThreads), lds, stream, a);
  else
    hipLaunchKernelGGL(norm_kernel<float>, grid, dim3(kThreads), lds, stream, a);
  return hipGetLastError();
}

hipError_t launch_norm_backward(const NormArgs& a, m3_dtype dtype, hipStream_t stream) {
  const int groups = norm_backward_groups(a.rows, a.D);
  if (groups > 0) {
    const size_t lds = 2 * sizeof(float) * (size_t)a.D;
    const void* k = dtype == M3_BF16 ? reinterpret_cast<const void*>(&norm_backward_kernel<bf16>)
                                     : reinterpret_cast<const void*>(&norm_backward_kernel<float>);
    const hipError_t e = lds_limit(k, lds);
    if (e != hipSuccess) return e;
    if (dtype == M3_BF16)
      hipLaunchKernelGGL(norm_backward_kernel<bf16>, dim3(groups), dim3(kThreads), lds, stream, a);
    else
      hipLaunchKernelGGL(norm_backward_kernel<float>, dim3(groups), dim3(kThreads), lds, stream, a);
  }
  hipLaunchKernelGGL(norm_weights_kernel, dim3((a.D + kThreads - 1) / kThreads), dim3(kThreads), 0,
                     stream, a, groups);
  return hipGetLastError();
}

}  // namespace m3
