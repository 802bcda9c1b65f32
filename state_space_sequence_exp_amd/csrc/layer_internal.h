// layer_internal.h -- host-side interface between the C ABI of the layer
// operators (layer_api.hip: gated recurrence, layer norm, 8-bit state cache;
// selective_api.hip: short convolution, selective scan, gated feed-forward) and
// their kernel launchers.  Not installed; not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "m3_internal.h"
#include "m3ssm.h"

namespace m3 {

// One gated-recurrence call (all validated; ld in elements, never 0).
struct ScanArgs {
  int64_t B, T, D, nC;
  int64_t ld_x, ld_f, ld_g, ld_y, ld_dx, ld_df, ld_dg;
  const void *x, *f, *g;   // g may be null
  const float* h0;         // may be null (zeros)
  void* y;
  float* h_last;           // may be null
  float* states;           // forward: out, may be null; backward: in
  const void* dy;
  const float* dh_last;    // may be null
  void *dx, *df, *dg;
  float* dh0;              // may be null
  void* workspace;         // the chain's counters and words; null where none is needed
};
struct ChainWs;            // scan_tile.h
// A workgroup's tile: tokens (forward, backward) x bytes of channels.
constexpr int kScanForwardTile = 128, kScanBackwardTile = M3_SCAN_CHUNK, kScanTileBytes = 256;
static_assert(kScanForwardTile % M3_SCAN_CHUNK == 0, "a tile holds whole chunks");
inline int64_t scan_tiles(int64_t D, int esize) {
  return (D + kScanTileBytes / esize - 1) / (kScanTileBytes / esize);
}
// The chain's workspace: its bytes (0 with one tile) and its parts, for tiles
// of `tile` tokens.
size_t scan_workspace(int64_t B, int64_t T, int64_t D, int tile, int esize);
ChainWs scan_chain(void* workspace, int64_t B, int64_t T, int64_t D, int tile, int esize);
// h_last of sequences without tokens (n states; zeros without h0).
hipError_t launch_scan_empty(const float* h0, float* h_last, int64_t n, hipStream_t stream);
hipError_t launch_scan(const ScanArgs& a, m3_dtype dtype, hipStream_t stream);
hipError_t launch_scan_backward(const ScanArgs& a, m3_dtype dtype, hipStream_t stream);

struct ScanStepArgs {
  int64_t B, D, ld_x, ld_f, ld_g, ld_y;
  const float* h_in;
  float* h_out;
  const void *x, *f, *g;
  void* y;
};
hipError_t launch_scan_step(const ScanStepArgs& a, m3_dtype dtype, hipStream_t stream);

constexpr int64_t kNormMaxChannels = 16384;

struct NormArgs {
  int64_t rows;
  int D;
  int64_t ld_x, ld_res, ld_sum, ld_y, ld_dy, ld_dsum, ld_dx;
  float eps;
  const void *x, *residual;
  const float *weight, *bias;
  void *y, *sum;
  float *mean, *rstd;
  const void *dy, *dsum;
  void* dx;
  float *dweight, *dbias;
  float* partial;  // backward workspace
};
// Row groups whose weight-gradient partials the backward keeps.
int norm_backward_groups(int64_t rows, int D, int esize);
hipError_t launch_norm(const NormArgs& a, m3_dtype dtype, hipStream_t stream);
hipError_t launch_norm_backward(const NormArgs& a, m3_dtype dtype, hipStream_t stream);

struct CacheArgs {
  int S, H, N, P, R;
  int n_slots;
  const int32_t* slots;  // may be null (identity)
  void* codes;
  float* scales;
  const float* h_in;     // store
  void* h_out;           // load
  const void *x_t, *x_prev, *B_t, *B_prev, *C_t;
  const float *dt, *A, *lam, *theta;
  void* y;
};
hipError_t launch_state_store(const CacheArgs& a, m3_code code, hipStream_t stream);
hipError_t launch_state_load(const CacheArgs& a, m3_code code, m3_dtype dtype, hipStream_t stream);
hipError_t launch_decode_cached(const CacheArgs& a, m3_code code, m3_dtype dtype,
                                hipStream_t stream);

// One convolution call (ld in elements, never 0).
struct ConvArgs {
  int64_t B, T, D, ld_x, ld_y;
  int W;
  bool silu;
  const void* x;
  const float *weight, *bias;  // bias may be null
  const void* state_in;        // may be null (zeros)
  const int32_t* lengths;      // may be null (all T)
  void* y;
  void* state_out;             // may be null; the step: the pool
  const int32_t* slots;        // the step: may be null (identity)
  int n_slots;
};
// Workgroups of a call.
double conv_groups(int64_t B, int64_t T, int64_t D, int esize);
double conv_step_groups(int64_t B, int64_t D, int esize);
hipError_t launch_conv(const ConvArgs& a, m3_dtype dtype, hipStream_t stream);
hipError_t launch_conv_step(const ConvArgs& a, m3_dtype dtype, hipStream_t stream);

struct SelectArgs {
  int64_t B, T, D;
  int N;
  int64_t ld_x, ld_dt, ld_z, ld_y, ld_b, ld_c;
  bool softplus;
  const void *x, *dt, *z, *Bt, *Ct;        // z may be null
  const float *A, *skip, *dt_bias, *h0;    // all but A may be null
  const int32_t* lengths;                  // may be null (all T)
  void* y;
  float* h_last;                           // may be null; the step: the pool
  const int32_t* slots;                    // the step: may be null (identity)
  int n_slots;
  void* workspace;
};
// Segments that a scan's tokens are cut into (1: not cut), the workspace that
// takes, and the workgroups of a launch.
int select_segments(int64_t B, int64_t T, int64_t D);
size_t select_workspace(int64_t B, int64_t T, int64_t D, int N);
double select_groups(int64_t B, int64_t T, int64_t D);
double select_step_groups(int64_t B, int64_t D, int N);
hipError_t launch_select(const SelectArgs& a, m3_dtype dtype, hipStream_t stream);
hipError_t launch_select_step(const SelectArgs& a, m3_dtype dtype, hipStream_t stream);

struct FfnArgs {
  int M, K, F;
  int64_t ld_x, ld_wg, ld_wu, ld_h, ld_gate, ld_up, ld_dh, ld_dx, ld_dwg, ld_dwu;
  const void *x, *wg, *wu;
  void* h;
  float *gate, *up;            // forward out (may be null), backward in
  const void* dh;
  void *dx, *dwg, *dwu;        // may be null
  void* workspace;
};
size_t ffn_backward_workspace(int64_t M, int64_t K, int64_t F, int esize);
// Which operands' rows are not whole 16-byte chunks at multiples of 4 bytes (a null
// pointer: by their distance alone), and the workgroups of the first launch, which
// copies these.
struct FfnCopies {
  bool weights, inputs;
};
FfnCopies ffn_copies(const FfnArgs& a, int esize);
double ffn_operand_groups(const FfnArgs& a, int esize);
hipError_t launch_ffn(const FfnArgs& a, m3_dtype dtype, hipStream_t stream);
hipError_t launch_ffn_backward(const FfnArgs& a, m3_dtype dtype, hipStream_t stream);

}  // namespace m3
