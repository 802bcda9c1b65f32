// selective_api.hip -- the C ABI of the short causal convolution, the selective
// scan and the gated feed-forward projections (declared in include/m3ssm.h).
// Arguments are validated on the host before any HIP call, so an invalid call
// enqueues nothing.
#include "layer_check.h"

namespace {

using namespace m3::check;

// Rows and slots of a pool.
bool pool_ok(int64_t batch, const int32_t* slots, int64_t n_slots) {
  return n_slots >= 0 && maybe(slots, 4) && (slots || batch <= n_slots);
}
// The memory of a pool of n_slots states (as much as there is of one that no
// memory could hold).
Span pool_of(const void* p, int64_t n_slots, double state, size_t es) {
  const double bytes = (double)n_slots * state * (double)es;
  return bytes_of(p, bytes < (double)(SIZE_MAX / 4) ? (size_t)bytes : SIZE_MAX / 4);
}

m3_status check_conv(const m3_conv_dims* d, m3_dtype dtype, bool step) {
  if (!d) return M3_ERR_INVALID_VALUE;
  if (d->batch < 0 || d->channels < 1 || (!step && d->seqlen < 0) || d->width < 1 ||
      !ld_ok(d->ld_x, d->channels) || !ld_ok(d->ld_y, d->channels))
    return M3_ERR_INVALID_VALUE;
  if (d->width < 2 || d->width > 4) return M3_ERR_NOT_SUPPORTED;
  const double rows = (double)d->batch * (step ? 1.0 : (double)d->seqlen + 4.0);
  if (d->batch > INT_MAX || d->channels > INT_MAX || (!step && d->seqlen > INT_MAX) ||
      rows * (double)ld_of(d->ld_x, d->channels) > kMaxElements ||
      rows * (double)ld_of(d->ld_y, d->channels) > kMaxElements)
    return M3_ERR_NOT_SUPPORTED;
  const int es = (int)esize_of(dtype);
  const double groups = step ? m3::conv_step_groups(d->batch, d->channels, es)
                             : m3::conv_groups(d->batch, d->seqlen, d->channels, es);
  return groups > kMaxGroups256 ? M3_ERR_NOT_SUPPORTED : M3_SUCCESS;
}

m3::ConvArgs conv_args(const m3_conv_dims* d) {
  m3::ConvArgs a = {};
  a.B = d->batch;
  a.T = d->seqlen;
  a.D = d->channels;
  a.W = (int)d->width;
  a.ld_x = ld_of(d->ld_x, d->channels);
  a.ld_y = ld_of(d->ld_y, d->channels);
  return a;
}

m3_status check_select(const m3_select_dims* d, bool step) {
  if (!d) return M3_ERR_INVALID_VALUE;
  if (d->batch < 0 || d->channels < 1 || d->dstate_n < 1 || (!step && d->seqlen < 0))
    return M3_ERR_INVALID_VALUE;
  if (d->dstate_n > M3_SELECT_MAX_STATES) return M3_ERR_NOT_SUPPORTED;
  const int64_t wide[] = {d->ld_x, d->ld_dt, d->ld_z, d->ld_y}, thin[] = {d->ld_b, d->ld_c};
  const double rows = (double)d->batch * (step ? 1.0 : (double)d->seqlen);
  for (int64_t ld : wide) {
    if (!ld_ok(ld, d->channels)) return M3_ERR_INVALID_VALUE;
    if (rows * (double)ld_of(ld, d->channels) > kMaxElements) return M3_ERR_NOT_SUPPORTED;
  }
  for (int64_t ld : thin) {
    if (!ld_ok(ld, d->dstate_n)) return M3_ERR_INVALID_VALUE;
    if (rows * (double)ld_of(ld, d->dstate_n) > kMaxElements) return M3_ERR_NOT_SUPPORTED;
  }
  if (d->batch > INT_MAX || d->channels > INT_MAX || (!step && d->seqlen > INT_MAX))
    return M3_ERR_NOT_SUPPORTED;
  const double groups = step ? m3::select_step_groups(d->batch, d->channels, (int)d->dstate_n)
                             : m3::select_groups(d->batch, d->seqlen, d->channels);
  return groups > (step ? kMaxGroups256 : kMaxGroups512) ? M3_ERR_NOT_SUPPORTED : M3_SUCCESS;
}

m3::SelectArgs select_args(const m3_select_dims* d) {
  m3::SelectArgs a = {};
  a.B = d->batch;
  a.T = d->seqlen;
  a.D = d->channels;
  a.N = (int)d->dstate_n;
  a.ld_x = ld_of(d->ld_x, d->channels);
  a.ld_dt = ld_of(d->ld_dt, d->channels);
  a.ld_z = ld_of(d->ld_z, d->channels);
  a.ld_y = ld_of(d->ld_y, d->channels);
  a.ld_b = ld_of(d->ld_b, d->dstate_n);
  a.ld_c = ld_of(d->ld_c, d->dstate_n);
  return a;
}

}  // namespace

extern "C" {

m3_status m3_causal_conv(const m3_conv_dims* dims, m3_dtype dtype, const void* x,
                         const float* weight, const float* bias, int silu, const void* state_in,
                         const int32_t* lengths, void* y, void* state_out, void* stream) {
  if (!dtype_ok(&dtype)) return M3_ERR_INVALID_VALUE;
  const m3_status st = check_conv(dims, dtype, false);
  if (st != M3_SUCCESS) return st;
  if (dims->batch == 0) return M3_SUCCESS;
  const uintptr_t es = esize_of(dtype);
  if (!need(weight, 4) || !maybe(bias, 4) || !maybe(state_in, es) || !maybe(lengths, 4) ||
      !maybe(state_out, es))
    return M3_ERR_INVALID_VALUE;
  if (dims->seqlen > 0 ? !need(x, es) || !need(y, es) : !maybe(x, es) || !maybe(y, es))
    return M3_ERR_INVALID_VALUE;
  m3::ConvArgs a = conv_args(dims);
  a.silu = silu != 0;
  a.x = x;
  a.weight = weight;
  a.bias = bias;
  a.state_in = state_in;
  a.lengths = lengths;
  a.y = y;
  a.state_out = state_out;
  const int64_t rows = a.B * a.T;
  const size_t kept = (size_t)a.B * (a.W - 1) * a.D * es, cols = (size_t)a.D * sizeof(float);
  const Span out[] = {rows_of(y, rows, a.D, a.ld_y, es), bytes_of(state_out, kept)};
  const Span in[] = {rows_of(x, rows, a.D, a.ld_x, es), bytes_of(weight, cols * a.W), bytes_of(bias, cols),
                     bytes_of(state_in, kept), bytes_of(lengths, (size_t)a.B * sizeof(int32_t))};
  if (outputs_meet(out, in)) return M3_ERR_INVALID_VALUE;
  if (a.T == 0 && !state_out) return M3_SUCCESS;
  return done(m3::launch_conv(a, dtype, static_cast<hipStream_t>(stream)));
}

m3_status m3_causal_conv_step(const m3_conv_dims* dims, m3_dtype dtype, void* state,
                              const int32_t* slots, int64_t n_slots, const void* x,
                              const float* weight, const float* bias, int silu, void* y,
                              void* stream) {
  if (!dtype_ok(&dtype)) return M3_ERR_INVALID_VALUE;
  const m3_status st = check_conv(dims, dtype, true);
  if (st != M3_SUCCESS) return st;
  if (!pool_ok(dims->batch, slots, n_slots)) return M3_ERR_INVALID_VALUE;
  if (n_slots > INT_MAX) return M3_ERR_NOT_SUPPORTED;
  if (dims->batch == 0 || n_slots == 0) return M3_SUCCESS;
  const uintptr_t es = esize_of(dtype);
  if (!need(state, es) || !need(x, es) || !need(weight, 4) || !maybe(bias, 4) || !need(y, es))
    return M3_ERR_INVALID_VALUE;
  m3::ConvArgs a = conv_args(dims);
  a.T = 1;
  a.silu = silu != 0;
  a.x = x;
  a.weight = weight;
  a.bias = bias;
  a.y = y;
  a.state_out = state;
  a.slots = slots;
  a.n_slots = (int)n_slots;
  const size_t cols = (size_t)a.D * sizeof(float);
  const Span out[] = {rows_of(y, a.B, a.D, a.ld_y, es), pool_of(state, n_slots, (double)(a.W - 1) * a.D, es)};
  const Span in[] = {rows_of(x, a.B, a.D, a.ld_x, es), bytes_of(weight, cols * a.W), bytes_of(bias, cols),
                     bytes_of(slots, (size_t)a.B * sizeof(int32_t))};
  if (outputs_meet(out, in)) return M3_ERR_INVALID_VALUE;
  return done(m3::launch_conv_step(a, dtype, static_cast<hipStream_t>(stream)));
}

size_t m3_selective_scan_workspace_size(const m3_select_dims* dims, m3_dtype dtype) {
  if (!dtype_ok(&dtype) || check_select(dims, false) != M3_SUCCESS) return 0;
  return m3::select_workspace(dims->batch, dims->seqlen, dims->channels, (int)dims->dstate_n);
}

m3_status m3_selective_scan(const m3_select_dims* dims, m3_dtype dtype, const void* x,
                            const void* dt, const float* A, const void* B, const void* C,
                            const float* skip, const void* z, const float* dt_bias, int softplus,
                            const float* h0, const int32_t* lengths, void* y, float* h_last,
                            void* workspace, size_t workspace_bytes, void* stream) {
  if (!dtype_ok(&dtype)) return M3_ERR_INVALID_VALUE;
  const m3_status st = check_select(dims, false);
  if (st != M3_SUCCESS) return st;
  if (dims->batch == 0) return M3_SUCCESS;
  const uintptr_t es = esize_of(dtype);
  if (!maybe(h0, 4) || !maybe(h_last, 4) || !maybe(skip, 4) || !maybe(dt_bias, 4) || !maybe(z, es) ||
      !maybe(lengths, 4))
    return M3_ERR_INVALID_VALUE;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const size_t cols = (size_t)dims->channels * sizeof(float);
  const size_t states = (size_t)dims->batch * dims->dstate_n * cols;
  if (dims->seqlen == 0) {
    if (h0 && h_last && partial_overlap(h0, h_last, states)) return M3_ERR_INVALID_VALUE;
    return h_last ? done(m3::launch_scan_empty(h0, h_last, (int64_t)(states / sizeof(float)), s)) : M3_SUCCESS;
  }
  if (!need(x, es) || !need(dt, es) || !need(A, 4) || !need(B, es) || !need(C, es) || !need(y, es))
    return M3_ERR_INVALID_VALUE;
  const size_t need_bytes = m3_selective_scan_workspace_size(dims, dtype);
  if (need_bytes > 0) {
    if (!workspace || workspace_bytes < need_bytes) return M3_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return M3_ERR_INVALID_VALUE;
  }
  m3::SelectArgs a = select_args(dims);
  a.softplus = softplus != 0;
  a.x = x;
  a.dt = dt;
  a.z = z;
  a.Bt = B;
  a.Ct = C;
  a.A = A;
  a.skip = skip;
  a.dt_bias = dt_bias;
  a.h0 = h0;
  a.lengths = lengths;
  a.y = y;
  a.h_last = h_last;
  a.workspace = workspace;
  const int64_t rows = a.B * a.T;
  const Span out[] = {rows_of(y, rows, a.D, a.ld_y, es), bytes_of(h_last, states),
                      bytes_of(workspace, need_bytes)};
  const Span in[] = {rows_of(x, rows, a.D, a.ld_x, es), rows_of(dt, rows, a.D, a.ld_dt, es),
                     rows_of(z, rows, a.D, a.ld_z, es), rows_of(B, rows, a.N, a.ld_b, es),
                     rows_of(C, rows, a.N, a.ld_c, es), bytes_of(A, cols * a.N), bytes_of(skip, cols),
                     bytes_of(dt_bias, cols), bytes_of(h0, states),
                     bytes_of(lengths, (size_t)a.B * sizeof(int32_t))};
  if (outputs_meet(out, in)) return M3_ERR_INVALID_VALUE;
  return done(m3::launch_select(a, dtype, s));
}

m3_status m3_selective_scan_step(const m3_select_dims* dims, m3_dtype dtype, float* h,
                                 const int32_t* slots, int64_t n_slots, const void* x,
                                 const void* dt, const float* A, const void* B, const void* C,
                                 const float* skip, const void* z, const float* dt_bias,
                                 int softplus, void* y, void* stream) {
  if (!dtype_ok(&dtype)) return M3_ERR_INVALID_VALUE;
  const m3_status st = check_select(dims, true);
  if (st != M3_SUCCESS) return st;
  if (!pool_ok(dims->batch, slots, n_slots)) return M3_ERR_INVALID_VALUE;
  if (n_slots > INT_MAX) return M3_ERR_NOT_SUPPORTED;
  if (dims->batch == 0 || n_slots == 0) return M3_SUCCESS;
  const uintptr_t es = esize_of(dtype);
  if (!need(h, 4) || !need(x, es) || !need(dt, es) || !need(A, 4) || !need(B, es) || !need(C, es) ||
      !maybe(skip, 4) || !maybe(z, es) || !maybe(dt_bias, 4) || !need(y, es))
    return M3_ERR_INVALID_VALUE;
  m3::SelectArgs a = select_args(dims);
  a.T = 1;
  a.softplus = softplus != 0;
  a.x = x;
  a.dt = dt;
  a.z = z;
  a.Bt = B;
  a.Ct = C;
  a.A = A;
  a.skip = skip;
  a.dt_bias = dt_bias;
  a.y = y;
  a.h_last = h;
  a.slots = slots;
  a.n_slots = (int)n_slots;
  const size_t cols = (size_t)a.D * sizeof(float);
  const Span out[] = {rows_of(y, a.B, a.D, a.ld_y, es),
                      pool_of(h, n_slots, (double)a.D * (double)a.N, sizeof(float))};
  const Span in[] = {rows_of(x, a.B, a.D, a.ld_x, es), rows_of(dt, a.B, a.D, a.ld_dt, es),
                     rows_of(z, a.B, a.D, a.ld_z, es), rows_of(B, a.B, a.N, a.ld_b, es),
                     rows_of(C, a.B, a.N, a.ld_c, es), bytes_of(A, cols * a.N), bytes_of(skip, cols),
                     bytes_of(dt_bias, cols), bytes_of(slots, (size_t)a.B * sizeof(int32_t))};
  if (outputs_meet(out, in)) return M3_ERR_INVALID_VALUE;
  return done(m3::launch_select_step(a, dtype, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

// ---- gated feed-forward ---------------------------------------------------------

namespace {

// Leading dimensions whose rows a tile's 32-bit offsets reach (256 of them, in bytes),
// and grids of tiles that a launch takes.
constexpr int64_t kMaxFfnLd = (1 << 22) - 1;
constexpr double kMaxFfnTiles = 8.0e6;  // of 64 x 64, of up to 512 threads

m3_status check_ffn(const m3_ffn_dims* d, m3_dtype dtype, bool backward) {
  if (!d) return M3_ERR_INVALID_VALUE;
  if (d->rows < 0 || d->channels < 1 || d->hidden < 1) return M3_ERR_INVALID_VALUE;
  const struct {
    int64_t ld, row;
    bool here;
  } arrays[] = {{d->ld_x, d->channels, true},        {d->ld_wgate, d->channels, true},
                {d->ld_wup, d->channels, true},      {d->ld_gate, d->hidden, true},
                {d->ld_up, d->hidden, true},         {d->ld_h, d->hidden, !backward},
                {d->ld_dh, d->hidden, backward},     {d->ld_dx, d->channels, backward},
                {d->ld_dwgate, d->channels, backward}, {d->ld_dwup, d->channels, backward}};
  for (const auto& a : arrays)
    if (a.here && !ld_ok(a.ld, a.row)) return M3_ERR_INVALID_VALUE;
  for (const auto& a : arrays)
    if (a.here && ld_of(a.ld, a.row) > kMaxFfnLd) return M3_ERR_NOT_SUPPORTED;
  const double M = (double)d->rows + 64, K = (double)d->channels + 64, F = (double)d->hidden + 64;
  // (backward, dg and du lie side by side, whole tiles each)
  if (backward && d->hidden > kMaxFfnLd / 2 - 63) return M3_ERR_NOT_SUPPORTED;
  if (d->rows > INT_MAX - 64 || M * F / 2048 > kMaxFfnTiles || M * K / 4096 > kMaxFfnTiles ||
      F * K / 2048 > kMaxFfnTiles)
    return M3_ERR_NOT_SUPPORTED;
  return M3_SUCCESS;
}

m3::FfnArgs ffn_args(const m3_ffn_dims* d) {
  m3::FfnArgs a = {};
  a.M = (int)d->rows;
  a.K = (int)d->channels;
  a.F = (int)d->hidden;
  a.ld_x = ld_of(d->ld_x, d->channels);
  a.ld_wg = ld_of(d->ld_wgate, d->channels);
  a.ld_wu = ld_of(d->ld_wup, d->channels);
  a.ld_h = ld_of(d->ld_h, d->hidden);
  a.ld_gate = ld_of(d->ld_gate, d->hidden);
  a.ld_up = ld_of(d->ld_up, d->hidden);
  a.ld_dh = ld_of(d->ld_dh, d->hidden);
  a.ld_dx = ld_of(d->ld_dx, d->channels);
  a.ld_dwg = ld_of(d->ld_dwgate, d->channels);
  a.ld_dwu = ld_of(d->ld_dwup, d->channels);
  return a;
}

// The backward's: also whether its first launch holds the copies that have to be made of
// these arrays, or, of null ones, by their rows' distances alone.
m3_status check_ffn_backward(const m3_ffn_dims* d, m3_dtype dtype, const void* x, const void* w_gate,
                             const void* w_up) {
  const m3_status st = check_ffn(d, dtype, true);
  if (st != M3_SUCCESS) return st;
  m3::FfnArgs a = ffn_args(d);
  a.x = x;
  a.wg = w_gate;
  a.wu = w_up;
  return m3::ffn_operand_groups(a, (int)esize_of(dtype)) > kMaxGroups256 ? M3_ERR_NOT_SUPPORTED : M3_SUCCESS;
}

}  // namespace

extern "C" {

m3_status m3_gated_ffn(const m3_ffn_dims* dims, m3_dtype dtype, const void* x,
                       const void* w_gate, const void* w_up, void* h, float* gate, float* up,
                       void* stream) {
  if (!dtype_ok(&dtype)) return M3_ERR_INVALID_VALUE;
  const m3_status st = check_ffn(dims, dtype, false);
  if (st != M3_SUCCESS) return st;
  if (dims->rows == 0) return M3_SUCCESS;
  const uintptr_t es = esize_of(dtype);
  if (!need(x, es) || !need(w_gate, es) || !need(w_up, es) || !need(h, es) || !maybe(gate, 4) ||
      !maybe(up, 4) || (gate == nullptr) != (up == nullptr))
    return M3_ERR_INVALID_VALUE;
  m3::FfnArgs a = ffn_args(dims);
  a.x = x;
  a.wg = w_gate;
  a.wu = w_up;
  a.h = h;
  a.gate = gate;
  a.up = up;
  const Span out[] = {rows_of(h, a.M, a.F, a.ld_h, es), rows_of(gate, a.M, a.F, a.ld_gate, 4),
                      rows_of(up, a.M, a.F, a.ld_up, 4)};
  const Span in[] = {rows_of(x, a.M, a.K, a.ld_x, es), rows_of(w_gate, a.F, a.K, a.ld_wg, es),
                     rows_of(w_up, a.F, a.K, a.ld_wu, es)};
  if (outputs_meet(out, in)) return M3_ERR_INVALID_VALUE;
  return done(m3::launch_ffn(a, dtype, static_cast<hipStream_t>(stream)));
}

size_t m3_gated_ffn_backward_workspace_size(const m3_ffn_dims* dims, m3_dtype dtype) {
  if (!dtype_ok(&dtype) || check_ffn_backward(dims, dtype, nullptr, nullptr, nullptr) != M3_SUCCESS) return 0;
  return m3::ffn_backward_workspace(dims->rows, dims->channels, dims->hidden, (int)esize_of(dtype));
}

m3_status m3_gated_ffn_backward(const m3_ffn_dims* dims, m3_dtype dtype, const void* dh,
                                const void* x, const void* w_gate, const void* w_up,
                                const float* gate, const float* up, void* dx, void* dw_gate,
                                void* dw_up, void* workspace, size_t workspace_bytes,
                                void* stream) {
  if (!dtype_ok(&dtype)) return M3_ERR_INVALID_VALUE;
  const m3_status st = check_ffn_backward(dims, dtype, x, w_gate, w_up);
  if (st != M3_SUCCESS) return st;
  const uintptr_t es = esize_of(dtype);
  if (!maybe(dx, es) || !maybe(dw_gate, es) || !maybe(dw_up, es) ||
      (dw_gate == nullptr) != (dw_up == nullptr))
    return M3_ERR_INVALID_VALUE;
  m3::FfnArgs a = ffn_args(dims);
  size_t bytes = 0;
  if (dims->rows > 0) {
    if (!need(dh, es) || !need(x, es) || !need(w_gate, es) || !need(w_up, es) || !need(gate, 4) ||
        !need(up, 4))
      return M3_ERR_INVALID_VALUE;
    if (!dx && !dw_gate) return M3_SUCCESS;
    bytes = m3_gated_ffn_backward_workspace_size(dims, dtype);
    if (!workspace || workspace_bytes < bytes) return M3_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return M3_ERR_INVALID_VALUE;
  } else if (!dw_gate) {
    return M3_SUCCESS;
  }
  // (without rows the gradients are still written: not over each other or the weights)
  const Span out[] = {rows_of(dx, a.M, a.K, a.ld_dx, es), rows_of(dw_gate, a.F, a.K, a.ld_dwg, es),
                      rows_of(dw_up, a.F, a.K, a.ld_dwu, es), bytes_of(workspace, bytes)};
  const Span in[] = {rows_of(x, a.M, a.K, a.ld_x, es),      rows_of(w_gate, a.F, a.K, a.ld_wg, es),
                     rows_of(w_up, a.F, a.K, a.ld_wu, es),  rows_of(dh, a.M, a.F, a.ld_dh, es),
                     rows_of(gate, a.M, a.F, a.ld_gate, 4), rows_of(up, a.M, a.F, a.ld_up, 4)};
  if (outputs_meet(out, in)) return M3_ERR_INVALID_VALUE;
  a.dh = dh;
  a.x = x;
  a.wg = w_gate;
  a.wu = w_up;
  a.gate = const_cast<float*>(gate);
  a.up = const_cast<float*>(up);
  a.dx = dx;
  a.dwg = dw_gate;
  a.dwu = dw_up;
  a.workspace = workspace;
  return done(m3::launch_ffn_backward(a, dtype, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
