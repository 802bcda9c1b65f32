// layer_api.hip -- the C ABI of the operators beside the recurrence (declared
// in include/m3ssm.h): the gated linear recurrence, layer norm and the 8-bit
// state cache.  Arguments are validated on the host before any HIP call, so
// an invalid call enqueues nothing.
#include "layer_check.h"

namespace {

using namespace m3::check;

constexpr int64_t kMaxScanLd = (1 << 22) - 1024;

m3_status check_scan(const m3_scan_dims* d, bool backward) {
  if (!d) return M3_ERR_INVALID_VALUE;
  if (d->batch < 0 || d->seqlen < 0 || d->channels < 1) return M3_ERR_INVALID_VALUE;
  const int64_t lds[] = {d->ld_x, d->ld_f, d->ld_g, d->ld_y, d->ld_dx, d->ld_df, d->ld_dg};
  for (int i = 0; i < (backward ? 7 : 4); ++i) {
    if (!ld_ok(lds[i], d->channels)) return M3_ERR_INVALID_VALUE;
    if ((double)d->batch * (double)d->seqlen * (double)ld_of(lds[i], d->channels) > kMaxElements)
      return M3_ERR_NOT_SUPPORTED;
    // a chunk's rows are addressed by 32-bit byte offsets
    if (d->seqlen > 1 && ld_of(lds[i], d->channels) > kMaxScanLd) return M3_ERR_NOT_SUPPORTED;
  }
  // one workgroup a chunk and channel tile, of 512 threads at most
  if (d->batch > INT_MAX || d->channels > INT_MAX / 2 || d->seqlen > INT_MAX - M3_SCAN_CHUNK ||
      (double)d->batch * (double)m3::scan_tiles(d->channels, 4) *
              (double)(d->seqlen / M3_SCAN_CHUNK + 1) > kMaxGroups512)
    return M3_ERR_NOT_SUPPORTED;
  return M3_SUCCESS;
}

// The workspace of a call: M3_SUCCESS, or why it is refused.
m3_status check_scan_workspace(const m3_scan_dims* d, m3_dtype dtype, const void* workspace,
                               size_t bytes) {
  const size_t need_bytes = m3_gated_scan_workspace_size(d, dtype);
  if (need_bytes == 0) return M3_SUCCESS;
  if (!workspace || bytes < need_bytes) return M3_ERR_WORKSPACE;
  return aligned(workspace, 256) ? M3_SUCCESS : M3_ERR_INVALID_VALUE;
}

m3::ScanArgs scan_args(const m3_scan_dims* d) {
  m3::ScanArgs a = {};
  a.B = d->batch;
  a.T = d->seqlen;
  a.D = d->channels;
  a.nC = (d->seqlen + M3_SCAN_CHUNK - 1) / M3_SCAN_CHUNK;
  a.ld_x = ld_of(d->ld_x, d->channels);
  a.ld_f = ld_of(d->ld_f, d->channels);
  a.ld_g = ld_of(d->ld_g, d->channels);
  a.ld_y = ld_of(d->ld_y, d->channels);
  a.ld_dx = ld_of(d->ld_dx, d->channels);
  a.ld_df = ld_of(d->ld_df, d->channels);
  a.ld_dg = ld_of(d->ld_dg, d->channels);
  return a;
}

// What a call may write of its workspace.
Span workspace_of(const m3_scan_dims* d, m3_dtype dtype, void* workspace) {
  return bytes_of(workspace, m3_gated_scan_workspace_size(d, dtype));
}

}  // namespace

extern "C" {

size_t m3_gated_scan_workspace_size(const m3_scan_dims* dims, m3_dtype dtype) {
  if (!dtype_ok(&dtype) || check_scan(dims, false) != M3_SUCCESS) return 0;
  // the backward pass has the smaller tiles
  return m3::scan_workspace(dims->batch, dims->seqlen, dims->channels, m3::kScanBackwardTile,
                            (int)esize_of(dtype));
}

m3_status m3_gated_scan(const m3_scan_dims* dims, m3_dtype dtype, const void* x, const void* f,
                        const void* g, const float* h0, void* y, float* h_last, float* states,
                        void* workspace, size_t workspace_bytes, void* stream) {
  if (!dtype_ok(&dtype)) return M3_ERR_INVALID_VALUE;
  const m3_status st = check_scan(dims, false);
  if (st != M3_SUCCESS) return st;
  const uintptr_t es = esize_of(dtype);
  if (!maybe(h0, 4) || !maybe(h_last, 4) || !maybe(states, 4)) return M3_ERR_INVALID_VALUE;
  if (dims->batch > 0 && dims->seqlen > 0 &&
      (!need(x, es) || !need(f, es) || !maybe(g, es) || !need(y, es)))
    return M3_ERR_INVALID_VALUE;
  if (dims->batch == 0) return M3_SUCCESS;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const size_t state_bytes = (size_t)dims->batch * dims->channels * sizeof(float);
  if (dims->seqlen == 0) {
    if (h0 && h_last && partial_overlap(h0, h_last, state_bytes)) return M3_ERR_INVALID_VALUE;
    return h_last ? done(m3::launch_scan_empty(h0, h_last, dims->batch * dims->channels, s))
                  : M3_SUCCESS;
  }
  const m3_status wst = check_scan_workspace(dims, dtype, workspace, workspace_bytes);
  if (wst != M3_SUCCESS) return wst;
  m3::ScanArgs a = scan_args(dims);
  a.x = x;
  a.f = f;
  a.g = g;
  a.h0 = h0;
  a.y = y;
  a.h_last = h_last;
  a.states = states;
  a.workspace = workspace;
  // (a sequence's last tile writes h_last while others may still read h0)
  const int64_t rows = a.B * a.T;
  const Span out[] = {rows_of(y, rows, a.D, a.ld_y, es), bytes_of(h_last, state_bytes),
                      bytes_of(states, state_bytes * a.nC), workspace_of(dims, dtype, workspace)};
  const Span in[] = {rows_of(x, rows, a.D, a.ld_x, es), rows_of(f, rows, a.D, a.ld_f, es),
                     rows_of(g, rows, a.D, a.ld_g, es), bytes_of(h0, state_bytes)};
  if (outputs_meet(out, in)) return M3_ERR_INVALID_VALUE;
  return done(m3::launch_scan(a, dtype, s));
}

m3_status m3_gated_scan_backward(const m3_scan_dims* dims, m3_dtype dtype, const void* dy,
                                 const void* x, const void* f, const void* g,
                                 const float* states, const float* dh_last, void* dx, void* df,
                                 void* dg, float* dh0, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  if (!dtype_ok(&dtype)) return M3_ERR_INVALID_VALUE;
  const m3_status st = check_scan(dims, true);
  if (st != M3_SUCCESS) return st;
  const uintptr_t es = esize_of(dtype);
  if (!maybe(dh_last, 4) || !maybe(dh0, 4)) return M3_ERR_INVALID_VALUE;
  if (dims->batch > 0 && dims->seqlen > 0) {
    if (!need(dy, es) || !need(x, es) || !need(f, es) || !maybe(g, es) || !need(states, 4) ||
        !need(dx, es) || !need(df, es) || !maybe(dg, es) || (g == nullptr) != (dg == nullptr))
      return M3_ERR_INVALID_VALUE;
  }
  if (dims->batch == 0) return M3_SUCCESS;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const size_t state_bytes = (size_t)dims->batch * dims->channels * sizeof(float);
  if (dims->seqlen == 0) {
    if (dh_last && dh0 && partial_overlap(dh_last, dh0, state_bytes)) return M3_ERR_INVALID_VALUE;
    return dh0 ? done(m3::launch_scan_empty(dh_last, dh0, dims->batch * dims->channels, s))
               : M3_SUCCESS;
  }
  const m3_status wst = check_scan_workspace(dims, dtype, workspace, workspace_bytes);
  if (wst != M3_SUCCESS) return wst;
  m3::ScanArgs a = scan_args(dims);
  a.dy = dy;
  a.x = x;
  a.f = f;
  a.g = g;
  a.states = const_cast<float*>(states);
  a.dh_last = dh_last;
  a.dx = dx;
  a.df = df;
  a.dg = dg;
  a.dh0 = dh0;
  a.workspace = workspace;
  const int64_t rows = a.B * a.T;
  const Span out[] = {rows_of(dx, rows, a.D, a.ld_dx, es), rows_of(df, rows, a.D, a.ld_df, es),
                      rows_of(dg, rows, a.D, a.ld_dg, es), bytes_of(dh0, state_bytes),
                      workspace_of(dims, dtype, workspace)};
  const Span in[] = {rows_of(dy, rows, a.D, a.ld_y, es), rows_of(x, rows, a.D, a.ld_x, es),
                     rows_of(f, rows, a.D, a.ld_f, es), rows_of(g, rows, a.D, a.ld_g, es),
                     bytes_of(states, state_bytes * a.nC), bytes_of(dh_last, state_bytes)};
  if (outputs_meet(out, in)) return M3_ERR_INVALID_VALUE;
  return done(m3::launch_scan_backward(a, dtype, s));
}

m3_status m3_gated_scan_step(const m3_scan_dims* dims, m3_dtype dtype, const float* h_in,
                             float* h_out, const void* x, const void* f, const void* g, void* y,
                             void* stream) {
  if (!dtype_ok(&dtype) || !dims) return M3_ERR_INVALID_VALUE;
  m3_scan_dims one = *dims;
  one.seqlen = 1;
  const m3_status st = check_scan(&one, false);
  if (st != M3_SUCCESS) return st;
  if (dims->batch == 0) return M3_SUCCESS;
  const uintptr_t es = esize_of(dtype);
  if (!need(h_in, 4) || !need(h_out, 4) || !need(x, es) || !need(f, es) || !maybe(g, es) ||
      !need(y, es))
    return M3_ERR_INVALID_VALUE;
  if (partial_overlap(h_in, h_out, (size_t)dims->batch * dims->channels * sizeof(float)))
    return M3_ERR_INVALID_VALUE;
  m3::ScanStepArgs a = {};
  a.B = dims->batch;
  a.D = dims->channels;
  a.ld_x = ld_of(dims->ld_x, dims->channels);
  a.ld_f = ld_of(dims->ld_f, dims->channels);
  a.ld_g = ld_of(dims->ld_g, dims->channels);
  a.ld_y = ld_of(dims->ld_y, dims->channels);
  a.h_in = h_in;
  a.h_out = h_out;
  a.x = x;
  a.f = f;
  a.g = g;
  a.y = y;
  const size_t state_bytes = (size_t)a.B * a.D * sizeof(float);
  const Span ys = rows_of(y, a.B, a.D, a.ld_y, es), state = bytes_of(h_out, state_bytes);
  const Span out[] = {ys, state};
  const Span in[] = {rows_of(x, a.B, a.D, a.ld_x, es), rows_of(f, a.B, a.D, a.ld_f, es),
                     rows_of(g, a.B, a.D, a.ld_g, es)};
  if (outputs_meet(out, in) || meet(ys, bytes_of(h_in, state_bytes))) return M3_ERR_INVALID_VALUE;
  return done(m3::launch_scan_step(a, dtype, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

// ---- layer norm -----------------------------------------------------------------

namespace {

m3_status check_norm(const m3_norm_dims* d, bool backward) {
  if (!d) return M3_ERR_INVALID_VALUE;
  if (d->rows < 0 || d->channels < 1) return M3_ERR_INVALID_VALUE;
  const int64_t fwd[] = {d->ld_x, d->ld_residual, d->ld_sum, d->ld_y};
  const int64_t bwd[] = {d->ld_sum, d->ld_dy, d->ld_dsum, d->ld_dx};
  for (int i = 0; i < 4; ++i) {
    const int64_t ld = backward ? bwd[i] : fwd[i];
    if (!ld_ok(ld, d->channels)) return M3_ERR_INVALID_VALUE;
    if ((double)d->rows * (double)ld_of(ld, d->channels) > kMaxElements)
      return M3_ERR_NOT_SUPPORTED;
  }
  if (d->channels > m3::kNormMaxChannels || d->rows > INT_MAX) return M3_ERR_NOT_SUPPORTED;
  return M3_SUCCESS;
}

m3::NormArgs norm_args(const m3_norm_dims* d) {
  m3::NormArgs a = {};
  a.rows = d->rows;
  a.D = (int)d->channels;
  a.ld_x = ld_of(d->ld_x, d->channels);
  a.ld_res = ld_of(d->ld_residual, d->channels);
  a.ld_sum = ld_of(d->ld_sum, d->channels);
  a.ld_y = ld_of(d->ld_y, d->channels);
  a.ld_dy = ld_of(d->ld_dy, d->channels);
  a.ld_dsum = ld_of(d->ld_dsum, d->channels);
  a.ld_dx = ld_of(d->ld_dx, d->channels);
  return a;
}

}  // namespace

extern "C" {

m3_status m3_layer_norm(const m3_norm_dims* dims, m3_dtype dtype, const void* x,
                        const void* residual, const float* weight, const float* bias, float eps,
                        void* y, void* sum_out, float* mean, float* rstd, void* stream) {
  if (!dtype_ok(&dtype)) return M3_ERR_INVALID_VALUE;
  const m3_status st = check_norm(dims, false);
  if (st != M3_SUCCESS) return st;
  if (!(eps >= 0.f) || !(eps < 3.0e38f)) return M3_ERR_INVALID_VALUE;  // also rejects NaN
  if (dims->rows == 0) return M3_SUCCESS;
  const uintptr_t es = esize_of(dtype);
  if (!need(x, es) || !maybe(residual, es) || !need(weight, 4) || !maybe(bias, 4) ||
      !need(y, es) || !maybe(sum_out, es) || !maybe(mean, 4) || !maybe(rstd, 4))
    return M3_ERR_INVALID_VALUE;
  m3::NormArgs a = norm_args(dims);
  // an output takes an input's place whole or not at all, and the outputs differ
  const Span xs = rows_of(x, a.rows, a.D, a.ld_x, es), rs = rows_of(residual, a.rows, a.D, a.ld_res, es);
  const Span ys = rows_of(y, a.rows, a.D, a.ld_y, es), ss = rows_of(sum_out, a.rows, a.D, a.ld_sum, es);
  if (cross(ys, xs) || cross(ys, rs) || cross(ss, xs) || cross(ss, rs)) return M3_ERR_INVALID_VALUE;
  const size_t stat = (size_t)a.rows * sizeof(float), cols = (size_t)a.D * sizeof(float);
  const Span means = bytes_of(mean, stat), rstds = bytes_of(rstd, stat);
  const Span out[] = {ys, ss, means, rstds};
  const Span in[] = {bytes_of(weight, cols), bytes_of(bias, cols)};
  if (outputs_meet(out, in) || meet(means, xs) || meet(means, rs) || meet(rstds, xs) || meet(rstds, rs))
    return M3_ERR_INVALID_VALUE;
  a.eps = eps;
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.bias = bias;
  a.y = y;
  a.sum = sum_out;
  a.mean = mean;
  a.rstd = rstd;
  return done(m3::launch_norm(a, dtype, static_cast<hipStream_t>(stream)));
}

size_t m3_layer_norm_backward_workspace_size(const m3_norm_dims* dims, m3_dtype dtype) {
  if (!dtype_ok(&dtype) || check_norm(dims, true) != M3_SUCCESS) return 0;
  return (size_t)m3::norm_backward_groups(dims->rows, (int)dims->channels,
                                          (int)esize_of(dtype)) * 2 *
         (size_t)dims->channels * sizeof(float);
}

m3_status m3_layer_norm_backward(const m3_norm_dims* dims, m3_dtype dtype, const void* dy,
                                 const void* s, const float* weight, const float* mean,
                                 const float* rstd, const void* dsum, void* dx, float* dweight,
                                 float* dbias, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  if (!dtype_ok(&dtype)) return M3_ERR_INVALID_VALUE;
  const m3_status st = check_norm(dims, true);
  if (st != M3_SUCCESS) return st;
  const uintptr_t es = esize_of(dtype);
  if (!need(dweight, 4) || !maybe(dbias, 4)) return M3_ERR_INVALID_VALUE;
  m3::NormArgs a = norm_args(dims);
  const size_t cols = (size_t)a.D * sizeof(float);
  if (dims->rows > 0) {
    if (!need(dy, es) || !need(s, es) || !need(weight, 4) || !need(mean, 4) || !need(rstd, 4) ||
        !maybe(dsum, es) || !need(dx, es))
      return M3_ERR_INVALID_VALUE;
    if (!workspace || workspace_bytes < m3_layer_norm_backward_workspace_size(dims, dtype))
      return M3_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return M3_ERR_INVALID_VALUE;
    const Span dxs = rows_of(dx, a.rows, a.D, a.ld_dx, es), dys = rows_of(dy, a.rows, a.D, a.ld_dy, es);
    const Span dss = rows_of(dsum, a.rows, a.D, a.ld_dsum, es), ss = rows_of(s, a.rows, a.D, a.ld_sum, es);
    if (cross(dxs, dys) || cross(dxs, dss)) return M3_ERR_INVALID_VALUE;
    const size_t stat = (size_t)a.rows * sizeof(float);
    const Span ws = bytes_of(workspace, m3_layer_norm_backward_workspace_size(dims, dtype));
    const Span dws = bytes_of(dweight, cols), dbs = bytes_of(dbias, cols);
    const Span early[] = {dxs, ws};
    const Span in[] = {ss, bytes_of(weight, cols), bytes_of(mean, stat), bytes_of(rstd, stat)};
    // the weights' gradients are written when all else has been read
    if (outputs_meet(early, in) || meet(ws, dys) || meet(ws, dss) || meet(dws, dxs) || meet(dws, ws) ||
        meet(dbs, dxs) || meet(dbs, ws))
      return M3_ERR_INVALID_VALUE;
  }
  if (meet(bytes_of(dweight, cols), bytes_of(dbias, cols))) return M3_ERR_INVALID_VALUE;
  a.dy = dy;
  a.sum = const_cast<void*>(s);
  a.weight = weight;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.dsum = dsum;
  a.dx = dx;
  a.dweight = dweight;
  a.dbias = dbias;
  a.partial = static_cast<float*>(workspace);
  return done(m3::launch_norm_backward(a, dtype, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

// ---- state cache ------------------------------------------------------------------

namespace {

m3_status check_cache(const m3_dims* d, const int32_t* slots, int64_t n_slots) {
  if (!d) return M3_ERR_INVALID_VALUE;
  if (d->batch < 0 || d->nheads < 1 || d->headdim_p < 1 || d->dstate_n < 2 ||
      (d->dstate_n % 2) != 0 || n_slots < 0 || !maybe(slots, 4))
    return M3_ERR_INVALID_VALUE;
  const int64_t P = d->headdim_p;
  if (P != 16 && P != 32 && P != 64 && P != 128) return M3_ERR_NOT_SUPPORTED;
  if (d->dstate_n > 256 || d->dstate_n > m3::decode_max_n((int)P)) return M3_ERR_NOT_SUPPORTED;
  if (d->batch > INT_MAX || d->nheads > INT_MAX || n_slots > INT_MAX ||
      (double)d->batch * (double)d->nheads > kMaxGroups256)
    return M3_ERR_NOT_SUPPORTED;
  if (!slots && d->batch > n_slots) return M3_ERR_INVALID_VALUE;
  return M3_SUCCESS;
}

m3::CacheArgs cache_args(const m3_dims* d, void* codes, float* scales, const int32_t* slots,
                         int64_t n_slots) {
  m3::CacheArgs a = {};
  a.S = (int)d->batch;
  a.H = (int)d->nheads;
  a.N = (int)d->dstate_n;
  a.P = (int)d->headdim_p;
  a.n_slots = (int)n_slots;
  a.slots = slots;
  a.codes = codes;
  a.scales = scales;
  return a;
}

// The memory of a cache's codes and scales (as much as there is of one that no
// memory could hold).
struct CacheSpans {
  Span codes, scales, slots;
};
CacheSpans cache_spans(const m3::CacheArgs& a) {
  const double rows = (double)a.n_slots * (double)a.H * (double)a.N;
  const size_t most = SIZE_MAX / 4;
  const bool fits = rows * a.P < (double)most;
  return {bytes_of(a.codes, fits ? (size_t)a.n_slots * a.H * a.N * a.P : most),
          bytes_of(a.scales, fits ? (size_t)a.n_slots * a.H * a.N * sizeof(float) : most),
          bytes_of(a.slots, (size_t)a.S * sizeof(int32_t))};
}
size_t state_elements(const m3::CacheArgs& a) { return (size_t)a.S * a.H * a.N * a.P; }

}  // namespace

extern "C" {

m3_status m3_state_store(const m3_dims* dims, m3_code code, const float* h, void* codes,
                         float* scales, const int32_t* slots, int64_t n_slots, void* stream) {
  if (!code_ok(&code)) return M3_ERR_INVALID_VALUE;
  const m3_status st = check_cache(dims, slots, n_slots);
  if (st != M3_SUCCESS) return st;
  if (dims->batch == 0 || n_slots == 0) return M3_SUCCESS;
  if (!need(h, 16) || !need(codes, 16) || !need(scales, 4)) return M3_ERR_INVALID_VALUE;
  m3::CacheArgs a = cache_args(dims, codes, scales, slots, n_slots);
  a.h_in = h;
  const CacheSpans c = cache_spans(a);
  const Span out[] = {c.codes, c.scales};
  const Span in[] = {c.slots, bytes_of(h, state_elements(a) * sizeof(float))};
  if (outputs_meet(out, in)) return M3_ERR_INVALID_VALUE;
  return done(m3::launch_state_store(a, code, static_cast<hipStream_t>(stream)));
}

m3_status m3_state_load(const m3_dims* dims, m3_code code, m3_dtype dtype, const void* codes,
                        const float* scales, const int32_t* slots, int64_t n_slots, void* h,
                        void* stream) {
  if (!code_ok(&code) || !dtype_ok(&dtype)) return M3_ERR_INVALID_VALUE;
  const m3_status st = check_cache(dims, slots, n_slots);
  if (st != M3_SUCCESS) return st;
  if (dims->batch == 0) return M3_SUCCESS;
  if (!need(h, 16) || (n_slots > 0 && (!need(codes, 16) || !need(scales, 4))))
    return M3_ERR_INVALID_VALUE;
  m3::CacheArgs a = cache_args(dims, const_cast<void*>(codes), const_cast<float*>(scales), slots,
                               n_slots);
  a.h_out = h;
  const CacheSpans c = cache_spans(a);
  const Span out[] = {bytes_of(h, state_elements(a) * esize_of(dtype))};
  const Span in[] = {c.codes, c.scales, c.slots};
  if (outputs_meet(out, in)) return M3_ERR_INVALID_VALUE;
  return done(m3::launch_state_load(a, code, dtype, static_cast<hipStream_t>(stream)));
}

m3_status m3_decode_step_cached(const m3_dims* dims, m3_dtype dtype, m3_code code, void* codes,
                                float* scales, const int32_t* slots, int64_t n_slots,
                                const void* x_t, const void* x_prev, const void* B_t,
                                const void* B_prev, const void* C_t, const float* dt,
                                const float* A, const float* lam, const float* theta, void* y_t,
                                void* stream) {
  if (!dtype_ok(&dtype) || !code_ok(&code)) return M3_ERR_INVALID_VALUE;
  const m3_status st = check_cache(dims, slots, n_slots);
  if (st != M3_SUCCESS) return st;
  const int64_t R = dims->rank_r;
  if (R < 1) return M3_ERR_INVALID_VALUE;
  if (R != 1 && R != 2 && R != 4) return M3_ERR_NOT_SUPPORTED;
  if (dims->batch == 0 || n_slots == 0) return M3_SUCCESS;
  // without lam x_prev and B_prev are not read
  const uintptr_t es = esize_of(dtype);
  if (!need(codes, 16) || !need(scales, 4) || !need(x_t, 4 * es) || !need(B_t, 2 * es) ||
      !need(C_t, 2 * es) || !need(dt, 4) || !need(A, 4) || !need(y_t, es))
    return M3_ERR_INVALID_VALUE;
  if (!maybe(lam, 4) || !maybe(theta, 4) || !maybe(x_prev, 4 * es) || !maybe(B_prev, 2 * es) ||
      (lam && (!x_prev || !B_prev)))
    return M3_ERR_INVALID_VALUE;
  m3::CacheArgs a = cache_args(dims, codes, scales, slots, n_slots);
  a.R = (int)R;
  a.x_t = x_t;
  a.x_prev = x_prev;
  a.B_t = B_t;
  a.B_prev = B_prev;
  a.C_t = C_t;
  a.dt = dt;
  a.A = A;
  a.lam = lam;
  a.theta = theta;
  a.y = y_t;
  const size_t heads = (size_t)a.S * a.H;
  const size_t xy = heads * R * a.P * es, bc = heads * R * a.N * es, each = heads * sizeof(float);
  const CacheSpans c = cache_spans(a);
  const Span out[] = {c.codes, c.scales, bytes_of(y_t, xy)};
  const Span in[] = {c.slots, bytes_of(x_t, xy), bytes_of(lam ? x_prev : nullptr, xy), bytes_of(B_t, bc),
                     bytes_of(lam ? B_prev : nullptr, bc), bytes_of(C_t, bc), bytes_of(dt, each),
                     bytes_of(A, (size_t)a.H * sizeof(float)), bytes_of(lam, each),
                     bytes_of(theta, each * (a.N / 2))};
  if (outputs_meet(out, in)) return M3_ERR_INVALID_VALUE;
  return done(m3::launch_decode_cached(a, code, dtype, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
