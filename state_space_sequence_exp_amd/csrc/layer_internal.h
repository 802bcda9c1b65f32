// layer_internal.h -- host-side interface between the C ABI of the layer
// operators (layer_api.hip: gated recurrence, layer norm, 8-bit state cache)
// and their kernel launchers.  Not installed; not part of the ABI.
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

}  // namespace m3
